// gsr_adapters.hpp -- low-rank adapters beside a product: row m of
// C = act(alpha * A @ W + bias) uses W = B + s_l La_l^T Lb_l^T with l = ids[m]
// (rows whose id names no adapter: W = B).
//
// The sum over K is taken first, the rank last:
//   1. adapter_shrink_kernel: t[m, r] = s_l * sum_k A[m, k] La_l[r, k], fp32;
//   2. the product's own kernels add sum_r t[m, r] Lb_l[n, r] to their fp32
//      sums, so the adapter costs no pass over C and is scaled, biased and
//      activated with the sum it belongs to.
// Both steps run on the matrix cores with La and Lb as checkpoints hold them
// (rank x K and N x rank: the reduced index is contiguous, so a lane's operand
// is one 16-byte load and needs no LDS).
//
// t is an fp16 operand in step 2 without losing its fp32 value.  Its ranks go
// in chunks of 16; a row's chunk is scaled by the power of two that brings its
// largest |t| into [1, 2), and each value is split into its fp16 rounding and
// the fp16 rounding of the rest, which leaves at most 2^-23 of that largest
// value (hi has 11 bits, lo the 11 bits below, down to fp16's smallest step of
// 2^-24).  The product runs over both halves and the power of two multiplies
// its fp32 result, so no magnitude of t overflows or underflows.  A chunk's
// record is its 16 hi values and then its 16 lo values: 64 bytes, the K = 32
// operand of one 16x16x32 MFMA against the chunk of Lb taken twice.
//
// Rows of one tile may belong to different adapters.  The loops run once per
// distinct adapter of the tile's rows; a lane of the accumulator layout holds
// one row, so a lane adds a result only if the adapter is its row's, and what
// another adapter's weights hold (NaN, infinities) cannot reach it.
#pragma once

#include "gsr_kernels.hpp"

namespace gsr {

constexpr int kAdapterChunk = 16;  // ranks per record of t

// One 8-value operand piece of a matrix behind a buffer: values r .. r + 7 of
// the row that starts at element `row`, zeros from `len` on (and for a row
// that is not `in`).  Without branches, so that the loads of a batch go out
// together.  VEC: rows are 16-byte aligned and `len` is a multiple of 8.
template <bool VEC>
__device__ __forceinline__ half8 piece8(__amdgpu_buffer_rsrc_t rs, uint32_t row, int r, int len, bool in)
{
    if constexpr (VEC) {
        return __builtin_bit_cast(half8, __builtin_amdgcn_raw_buffer_load_b128(
                                             rs, (in && r < len) ? (row + (uint32_t)r) * 2u : kOutOfRange, 0, 0));
    } else {
        uint32_t h[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            h[i] = __builtin_amdgcn_raw_buffer_load_b16(rs, (in && r + i < len) ? (row + (uint32_t)(r + i)) * 2u : kOutOfRange, 0, 0);
        return __builtin_bit_cast(half8, u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16});
    }
}

__device__ __forceinline__ int adapter_of(const int32_t* ids, int m, int M, int adapters)
{
    const int l = ids[min(m, M - 1)];
    return (m < M && (uint32_t)l < (uint32_t)adapters) ? l : -1;
}

// ---- step 1 ---------------------------------------------------------------------
struct ShrinkArgs {
    const uint16_t* A;      // M x K
    const uint16_t* la;     // adapters x rank x K
    const int32_t* ids;     // M
    const float* scales;    // adapters, or null (ones)
    uint16_t* t;            // M x chunks records
    float* t_scale;         // M x chunks
    int M, K, adapters, rank, chunks;
    int slots;              // workgroups that share a row block's adapters
};

constexpr int kShrinkWaves = 16;
constexpr int kShrinkRows = 16;  // rows per workgroup

// f(l) for each distinct adapter among 16 rows, as the lanes hold their ids,
// in order of the lowest row.
template <class F>
__device__ __forceinline__ void for_each_adapter(int id, F&& f)
{
    uint64_t todo = __ballot(id >= 0);
    while (todo) {
        const int l = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)todo) - 1);
        f(l);
        todo &= ~__ballot(id == l);
    }
}

// A workgroup takes 16 rows, NB chunks of ranks and every slots-th distinct
// adapter of the rows; its 16 waves cut K into runs of 32-value steps, walked
// STEPS at a time so that their loads are in flight together, and the waves'
// sums meet in LDS and are added in wave order.  A row's chunk is finished by
// one workgroup, so nothing is shared between workgroups and no order depends
// on timing.  Bound by the bytes of A and La (a decode step reads each
// adapter once; prompts read A once and La from the caches), which is why few
// rows get a workgroup per adapter and chunk, and many rows one per row block
// that reads A once for four chunks.
template <bool VEC, int NB>
__global__ void __launch_bounds__(64 * kShrinkWaves) adapter_shrink_kernel(ShrinkArgs s)
{
    constexpr int STEPS = NB == 1 ? 8 : 4;
    __shared__ float sums[kShrinkWaves][kShrinkRows][kAdapterChunk * NB + 4];
    __shared__ int done[kShrinkRows];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lrow = lane & 15, lq = lane >> 4;
    const int m0 = blockIdx.x * kShrinkRows, c0 = blockIdx.y * NB, r0 = c0 * kAdapterChunk;

    const int id = adapter_of(s.ids, m0 + lrow, s.M, s.adapters);
    const int steps = (s.K + 31) / 32;
    const int ks0 = steps * wave / kShrinkWaves, ks1 = steps * (wave + 1) / kShrinkWaves;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(s.A, (uint32_t)s.M * (uint32_t)s.K * 2u);
    const uint32_t arow = (uint32_t)(m0 + lrow) * (uint32_t)s.K;
    const bool ain = m0 + lrow < s.M;

    f32x4 out[NB] = {};
    bool mine = false;
    int at = 0;
    for_each_adapter(id, [&](int l) {
        if (at++ % s.slots != (int)blockIdx.z) return;
        mine |= id == l;
        const __amdgpu_buffer_rsrc_t rl = make_rsrc(s.la + (int64_t)l * s.rank * s.K, (uint32_t)s.rank * (uint32_t)s.K * 2u);
        f32x4 d[NB] = {};
        for (int ks = ks0; ks < ks1; ks += STEPS) {
            half8 x[STEPS], w[STEPS][NB];
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int k = 32 * (ks + i) + 8 * lq;
                const int len = ks + i < ks1 ? s.K : 0;
                x[i] = piece8<VEC>(ra, arow, k, len, ain);
#pragma unroll
                for (int q = 0; q < NB; ++q) {
                    const int r = r0 + 16 * q + lrow;
                    w[i][q] = piece8<VEC>(rl, (uint32_t)r * (uint32_t)s.K, k, len, r < s.rank);
                }
            }
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
#pragma unroll
                for (int q = 0; q < NB; ++q) d[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[i][q], x[i], d[q], 0, 0, 0);
        }
#pragma unroll
        for (int q = 0; q < NB; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i) out[q][i] = id == l ? out[q][i] + d[q][i] : out[q][i];
    });
    if (__ballot(mine) == 0) return;  // the same in every wave
#pragma unroll
    for (int q = 0; q < NB; ++q) *(f32x4*)&sums[wave][lrow][16 * q + 4 * lq] = out[q];
    if (wave == 0 && lq == 0) done[lrow] = mine ? id : -1;
    __syncthreads();

    // thread t: row t / 16 % 16 and rank t % 16 of chunk t / 256
    const int row = (tid >> 4) & 15, c = tid & 15, q = tid >> 8;
    if (q >= NB || c0 + q >= s.chunks) return;  // whole waves
    const int l = done[row];
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < kShrinkWaves; ++w) t += sums[w][row][16 * q + c];
    t *= (l >= 0 && s.scales != nullptr) ? s.scales[l] : 1.0f;
    bool odd = !(fabsf(t) <= 3.0e38f);
    float big = fabsf(t);
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) {
        big = fmaxf(big, __shfl_xor(big, x));
        odd |= (bool)__shfl_xor((int)odd, x);
    }
    if (l < 0) return;
    // 2^e <= big < 2^(e + 1); zeros, and rows with an infinity or a NaN, keep 2^0
    int e = 0;
    if (!odd && big > 0.0f) e = max(__builtin_amdgcn_frexp_expf(big) - 1, -100);
    const int64_t rec = (int64_t)(m0 + row) * s.chunks + c0 + q;
    const float v = t * ldexpf(1.0f, -e);
    const _Float16 hi = (_Float16)v;
    const _Float16 lo = odd ? (_Float16)0.0f : (_Float16)(v - (float)hi);
    s.t[rec * 32 + c] = __builtin_bit_cast(uint16_t, hi);
    s.t[rec * 32 + 16 + c] = __builtin_bit_cast(uint16_t, lo);
    if (c == 0) s.t_scale[rec] = ldexpf(1.0f, e);
}

// ---- step 2 ---------------------------------------------------------------------
__device__ __forceinline__ __amdgpu_buffer_rsrc_t lb_rsrc(const Problem& p, int l)
{
    return make_rsrc(p.lb + (int64_t)l * p.N * p.rank, (uint32_t)p.N * (uint32_t)p.rank * 2u);
}

// Values r .. r + 7 of Lb's row n.
__device__ __forceinline__ half8 lb_piece(const Problem& p, __amdgpu_buffer_rsrc_t rl, int n, int r)
{
    const uint32_t row = (uint32_t)n * (uint32_t)p.rank;
    return p.lb_vec ? piece8<true>(rl, row, r, p.rank, n < p.N) : piece8<false>(rl, row, r, p.rank, n < p.N);
}

// acc += t @ Lb^T on the 16x16x32 MFMA for FN x FM blocks (n, m) of 16x16 at
// column n0, row m0 of the problem: lane l holds row 16 b + l % 16 and columns
// 16 a + 4 (l / 16) + 0..3.  One MFMA per block and chunk: lanes 0-31 hold hi,
// lanes 32-63 lo.  Nothing hides behind these loads, so they go out early and
// together: the ids of all row blocks first, a row block's records while the
// block before it is worked on, and Lb's fragments of CB chunks at a time,
// which stay in registers from row block to row block while the adapter does
// not change (as in a batch of prompts) and its rank needs no more of them.
// The adapters of a row block are looped over with the column blocks'
// contribution in registers of its own, and every accumulator is then changed
// once, in straight-line code: changing accumulators inside a loop made the
// register allocator spill them (756 registers on the 128x256 tile).  GN of
// the FN column blocks are worked on at a time; GN and CB are what the wave's
// registers hold.
template <int GN, int CB, int FN, int FM>
__device__ __forceinline__ void adapter_add16(const Problem& p, f32x4 (&acc)[FN][FM], int m0, int n0)
{
    static_assert(FN % GN == 0, "whole groups of column blocks");
    const int lane = threadIdx.x & 63, lrow = lane & 15, lq = lane >> 4;
    int id[FM];
#pragma unroll
    for (int b = 0; b < FM; ++b) id[b] = adapter_of(p.ids, m0 + 16 * b + lrow, p.M, p.adapters);
    auto records = [&](int b, int c0, half8 (&t)[CB], float (&sc)[CB]) {
#pragma unroll
        for (int j = 0; j < CB; ++j) {
            const int64_t rec = (int64_t)min(m0 + 16 * b + lrow, p.M - 1) * p.chunks + min(c0 + j, p.chunks - 1);
            t[j] = __builtin_bit_cast(half8, *(const u32x4*)(p.t + rec * 32 + 8 * lq));
            sc[j] = p.t_scale[rec];
        }
    };
#pragma unroll
    for (int g = 0; g < FN; g += GN) {
        half8 x[CB][GN], t0[CB];
        float s0[CB];
        records(0, 0, t0, s0);
#pragma unroll
        for (int j = 0; j < CB; ++j)
#pragma unroll
            for (int a = 0; a < GN; ++a) x[j][a] = (half8)(_Float16)0.0f;
        int held = -1;  // the adapter whose first CB chunks x holds
#pragma unroll
        for (int b = 0; b < FM; ++b) {
            half8 t1[CB];
            float s1[CB];
            if (b + 1 < FM) records(b + 1, 0, t1, s1);
            f32x4 delta[GN] = {};
            uint64_t todo = __ballot(id[b] >= 0);
            while (todo) {
                const int l = __builtin_amdgcn_readlane(id[b], __ffsll((unsigned long long)todo) - 1);
                todo &= ~__ballot(id[b] == l);
                for (int c0 = 0; c0 < p.chunks; c0 += CB) {
                    if (held != l || p.chunks > CB) {
                        held = l;
                        const __amdgpu_buffer_rsrc_t rl = lb_rsrc(p, l);
#pragma unroll
                        for (int j = 0; j < CB; ++j)
#pragma unroll
                            for (int a = 0; a < GN; ++a)
                                x[j][a] = lb_piece(p, rl, n0 + 16 * (g + a) + lrow, kAdapterChunk * (c0 + j) + 8 * (lq & 1));
                        if (c0 > 0 || p.chunks > CB) records(b, c0, t0, s0);
                    }
#pragma unroll
                    for (int j = 0; j < CB; ++j) {
                        if (c0 + j >= p.chunks) break;
#pragma unroll
                        for (int a = 0; a < GN; ++a) {
                            const f32x4 d = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[j][a], t0[j], f32x4{}, 0, 0, 0);
#pragma unroll
                            for (int i = 0; i < 4; ++i) delta[a][i] += id[b] == l ? s0[j] * d[i] : 0.0f;
                        }
                    }
                }
            }
#pragma unroll
            for (int a = 0; a < GN; ++a) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[g + a][b][i] += delta[a][i];
                asm volatile("" : "+a"(acc[g + a][b]));  // back where the products left it
            }
            if (b + 1 < FM) {
#pragma unroll
                for (int j = 0; j < CB; ++j) t0[j] = t1[j], s0[j] = s1[j];
            }
        }
    }
}

// The same on the 32x32x16 MFMA for TN x TM blocks of 32x32: lane l holds row
// 32 b + l % 32 and columns 32 a + 8 g + 4 (l / 32) + i in register 4 g + i.
// The work items (adapter, chunk) are numbered; a wave takes items first,
// first + stride, ... (waves that each hold a share of the sum share them
// out), BATCH at a time: load() requests a batch, apply() adds it, so a batch
// can be in flight behind the product.
template <int TN, int TM, int BATCH>
struct AdapterItems {
    int m0, n0, first, stride;
    int id[TM], todo = 0;
    int item = 0, l = -1, c;  // the next item: adapter l's chunk c
    int ls[BATCH], n = 0;     // the batch: its adapters and its size
    half8 x[BATCH][TN], hi[BATCH][TM], lo[BATCH][TM];
    float sc[BATCH][TM];

    __device__ __forceinline__ AdapterItems(const Problem& p, int m0_, int n0_, int first_, int stride_)
        : m0(m0_), n0(n0_), first(first_), stride(stride_), c(p.chunks)
    {
#pragma unroll
        for (int b = 0; b < TM; ++b) {
            id[b] = adapter_of(p.ids, m0 + 32 * b + (int)(threadIdx.x & 31), p.M, p.adapters);
            todo |= (id[b] >= 0 ? 1 : 0) << b;
        }
    }

    // the wave's next item, or false
    __device__ __forceinline__ bool next(const Problem& p, int& ol, int& oc)
    {
        for (;;) {
            if (c == p.chunks) {
                const uint64_t any = __ballot(todo != 0);
                if (any == 0) return false;
                const int src = __ffsll((unsigned long long)any) - 1;
                const int tb = __ffs(__builtin_amdgcn_readlane(todo, src)) - 1;
                int v = id[0];
#pragma unroll
                for (int b = 1; b < TM; ++b) v = tb == b ? id[b] : v;
                l = __builtin_amdgcn_readlane(v, src);
#pragma unroll
                for (int b = 0; b < TM; ++b)
                    if (id[b] == l) todo &= ~(1 << b);
                c = 0;
            }
            const bool mine = item % stride == first;
            ol = l, oc = c;
            ++item, ++c;
            if (mine) return true;
        }
    }

    __device__ __forceinline__ void load(const Problem& p)
    {
        const int lane = threadIdx.x & 63, frow = lane & 31, fhi = lane >> 5;
        n = 0;
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            int ch = 0;
            ls[j] = -1;
            if (n == j && next(p, ls[j], ch)) ++n;
            if (n <= j) continue;
            const __amdgpu_buffer_rsrc_t rl = lb_rsrc(p, ls[j]);
#pragma unroll
            for (int a = 0; a < TN; ++a) x[j][a] = lb_piece(p, rl, n0 + 32 * a + frow, kAdapterChunk * ch + 8 * fhi);
#pragma unroll
            for (int b = 0; b < TM; ++b) {
                const int64_t rec = (int64_t)min(m0 + 32 * b + frow, p.M - 1) * p.chunks + ch;
                hi[j][b] = __builtin_bit_cast(half8, *(const u32x4*)(p.t + rec * 32 + 8 * fhi));
                lo[j][b] = __builtin_bit_cast(half8, *(const u32x4*)(p.t + rec * 32 + 16 + 8 * fhi));
                sc[j][b] = p.t_scale[rec];
            }
        }
    }

    __device__ __forceinline__ void apply(f32x16 (&acc)[TN][TM])
    {
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            if (j >= n) break;
#pragma unroll
            for (int b = 0; b < TM; ++b) {
                if (__ballot(id[b] == ls[j]) == 0) continue;
#pragma unroll
                for (int a = 0; a < TN; ++a) {
                    f32x16 d = {};
                    d = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[j][a], lo[j][b], d, 0, 0, 0);
                    d = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[j][a], hi[j][b], d, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[a][b][i] = id[b] == ls[j] ? acc[a][b][i] + sc[j][b] * d[i] : acc[a][b][i];
                }
            }
        }
    }

    // the batch in flight and all that follow it
    __device__ __forceinline__ void finish(const Problem& p, f32x16 (&acc)[TN][TM])
    {
        while (n > 0) {
            apply(acc);
            if (n < BATCH) break;
            load(p);
        }
    }
};

}  // namespace gsr
