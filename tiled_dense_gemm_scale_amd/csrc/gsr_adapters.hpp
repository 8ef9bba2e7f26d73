// gsr_adapters.hpp -- low-rank adapters beside a product: row m of
// C = act(alpha * A @ W + bias) uses W = B + s_l La_l^T Lb_l^T with l = ids[m]
// (rows whose id names no adapter: W = B).
//
// The sum over K is taken first, the rank last:
//   1. adapter_shrink_kernel: t[m, r] = s_l * sum_k A[m, k] La_l[r, k], fp32;
//   2. the product's own kernels add sum_r t[m, r] Lb_l[n, r] to their fp32
//      accumulators, so the adapter costs no pass over C and is scaled, biased
//      and activated with the sum it belongs to.
// Both steps run on the matrix cores with La and Lb as checkpoints hold them
// (rank x K and N x rank: the reduced index is contiguous, so a lane's operand
// is one 16-byte load and needs no LDS).
//
// t is an fp16 operand in step 2 without losing its fp32 value: a row is
// scaled by the power of two that brings its largest |t| into [1, 2), and each
// value is split into its fp16 rounding and the fp16 rounding of the rest,
// which leaves at most 2^-23 of the row's largest value (hi has 11 bits, lo
// the 11 bits below, down to fp16's smallest step of 2^-24).  The product
// runs over both halves and the power of two multiplies its fp32 result, so
// no magnitude of t overflows or underflows.
//
// Rows of one tile may belong to different adapters.  The loops run once per
// distinct adapter of the tile's rows; a lane of the accumulator layout holds
// one row, so a lane adds a result only if the adapter is its row's, and what
// another adapter's weights hold (NaN, infinities) cannot reach it.
#pragma once

#include "gsr_kernels.hpp"

namespace gsr {

// One 8-value operand piece: values r .. r + 7 of a row of `len` values at
// `row`; zeros past the row's end.  VEC: the row is 16-byte aligned and `len`
// a multiple of 8.
template <bool VEC>
__device__ __forceinline__ half8 piece8(const uint16_t* row, int r, int len)
{
    if constexpr (VEC) {
        return r < len ? __builtin_bit_cast(half8, *(const u32x4*)(row + r)) : (half8)(_Float16)0.0f;
    } else {
        half8 h = (half8)(_Float16)0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (r + i < len) h[i] = __builtin_bit_cast(_Float16, row[r + i]);
        return h;
    }
}

__device__ __forceinline__ int adapter_of(const int32_t* ids, int m, int M, int adapters)
{
    const int l = m < M ? ids[m] : -1;
    return (uint32_t)l < (uint32_t)adapters ? l : -1;
}

// ---- step 1 ---------------------------------------------------------------------
struct ShrinkArgs {
    const uint16_t* A;      // M x K
    const uint16_t* la;     // adapters x rank x K
    const int32_t* ids;     // M
    const float* scales;    // adapters, or null (ones)
    uint16_t* hi;           // M x rank_pad
    uint16_t* lo;
    float* row_scale;       // M
    float* partial;         // parts > 1: parts x (16 row_blocks) x rank_pad
    uint32_t* count;        // parts > 1: row_blocks
    int M, K, adapters, rank, rank_pad;
    int parts, kchunk;      // parts of kchunk values of K (a multiple of 32)
};

constexpr int kShrinkWaves = 8;
constexpr int kShrinkRows = 16;    // rows per workgroup
constexpr int kShrinkRanks = 64;   // ranks per pass over its part of K
constexpr int kShrinkMaxRank = 256;

// The distinct adapters among 16 rows, as the lanes hold their ids: f(l) for
// each, in order of the lowest row.
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

// A workgroup takes 16 rows and one part of K, 64 ranks at a time.  Its work
// items are (adapter, 32 values of K) pairs in that order, cut evenly over
// eight waves: one adapter's K range is shared when the rows agree, and
// adapters run side by side when they do not.  The waves' sums meet in LDS and
// are added in wave order; parts meet in the workspace, and the workgroup that
// arrives last adds them in part order (device-scope accesses and the arrival
// counter as in KsSum::split_sum_store), so no order depends on timing.
template <bool VEC>
__global__ void __launch_bounds__(64 * kShrinkWaves) adapter_shrink_kernel(ShrinkArgs s)
{
    __shared__ float sums[kShrinkWaves][kShrinkRows][kShrinkRanks];
    __shared__ int last;
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int lrow = lane & 15, lq = lane >> 4;
    const int block = blockIdx.x / s.parts, part = blockIdx.x - block * s.parts;
    const int m0 = block * kShrinkRows;
    const int kbeg = part * s.kchunk, kend = min(s.K, kbeg + s.kchunk);
    const int steps = (kend - kbeg + 31) / 32;

    const int id = adapter_of(s.ids, m0 + lrow, s.M, s.adapters);
    int distinct = 0;
    for_each_adapter(id, [&](int) { ++distinct; });
    if (distinct == 0) return;  // in every part of these rows
    const int items = distinct * steps;
    const int first = (int)((int64_t)items * wave / kShrinkWaves), end = (int)((int64_t)items * (wave + 1) / kShrinkWaves);
    const uint16_t* arow = s.A + (int64_t)min(m0 + lrow, s.M - 1) * s.K;

    // thread t ends with row t / 32 of the block, ranks t % 32, + 32, ...
    const int row = tid >> 5, c = tid & 31;
    float t[kShrinkMaxRank / 32];
#pragma unroll
    for (int rt = 0; rt < kShrinkMaxRank / kShrinkRanks; ++rt) {
        const int r0 = rt * kShrinkRanks;
        t[2 * rt] = t[2 * rt + 1] = 0.0f;
        if (r0 >= s.rank_pad) continue;
        const int nb = min(kShrinkRanks, s.rank_pad - r0) / 16;  // 2 or 4 blocks of 16 ranks
        f32x4 out[4] = {};
        int at = 0;  // the current adapter's first item
        for_each_adapter(id, [&](int l) {
            const int ks0 = max(first - at, 0), ks1 = min(end - at, steps);
            at += steps;
            if (ks0 >= ks1) return;
            const uint16_t* rrow[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                rrow[q] = s.la + ((int64_t)l * s.rank + min(r0 + 16 * q + lrow, s.rank - 1)) * s.K;
            f32x4 d[4] = {};
#pragma unroll 4
            for (int ks = ks0; ks < ks1; ++ks) {
                const int k = kbeg + 32 * ks + 8 * lq;
                const half8 x = piece8<VEC>(arow, k, kend);
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (q < nb) d[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(piece8<VEC>(rrow[q], k, kend), x, d[q], 0, 0, 0);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) out[q][i] = id == l ? out[q][i] + d[q][i] : out[q][i];
        });
        if (rt > 0) __syncthreads();  // the sums of the ranks before have been read
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q < nb) *(f32x4*)&sums[wave][lrow][16 * q + 4 * lq] = out[q];
        __syncthreads();
#pragma unroll
        for (int h = 0; h < 2; ++h)
            if (c + 32 * h < 16 * nb)
#pragma unroll
                for (int w = 0; w < kShrinkWaves; ++w) t[2 * rt + h] += sums[w][row][c + 32 * h];
    }
    if (s.parts > 1) {
        const int64_t stride = (int64_t)(gridDim.x / s.parts) * kShrinkRows * s.rank_pad;  // one part
        float* const slot = s.partial + (int64_t)(m0 + row) * s.rank_pad;
#pragma unroll
        for (int h = 0; h < kShrinkMaxRank / 32; ++h)
            if (c + 32 * h < s.rank_pad)
                __hip_atomic_store(slot + part * stride + c + 32 * h, t[h], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's sums have reached device scope
        __syncthreads();
        if (tid == 0) {
            const uint32_t before = __hip_atomic_fetch_add(s.count + block, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            last = before == (uint32_t)s.parts - 1u;
        }
        __syncthreads();
        if (!last) return;
        if (tid == 0) __hip_atomic_store(s.count + block, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
        for (int h = 0; h < kShrinkMaxRank / 32; ++h) {
            t[h] = 0.0f;
            if (c + 32 * h < s.rank_pad)
                for (int g = 0; g < s.parts; ++g)
                    t[h] += __hip_atomic_load(slot + g * stride + c + 32 * h, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    // the finished row
    const int m = m0 + row;
    const int l = adapter_of(s.ids, m, s.M, s.adapters);
    const float scale = (l >= 0 && s.scales != nullptr) ? s.scales[l] : 1.0f;
    float big = 0.0f;
    bool odd = false;
#pragma unroll
    for (int h = 0; h < kShrinkMaxRank / 32; ++h) {
        t[h] = c + 32 * h < s.rank ? t[h] * scale : 0.0f;
        odd |= !(fabsf(t[h]) <= 3.0e38f);
        big = fmaxf(big, fabsf(t[h]));
    }
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) {
        big = fmaxf(big, __shfl_xor(big, x));
        odd |= (bool)__shfl_xor((int)odd, x);
    }
    if (l < 0) return;
    // 2^e <= big < 2^(e + 1); rows of zeros, and rows with an infinity or a NaN, keep 2^0
    int e = 0;
    if (!odd && big > 0.0f) e = max(__builtin_amdgcn_frexp_expf(big) - 1, -100);
    const float down = ldexpf(1.0f, -e);
    if (c == 0) s.row_scale[m] = ldexpf(1.0f, e);
#pragma unroll
    for (int h = 0; h < kShrinkMaxRank / 32; ++h) {
        const float v = t[h] * down;
        const _Float16 hv = (_Float16)v;
        const _Float16 lv = odd ? (_Float16)0.0f : (_Float16)(v - (float)hv);
        const int64_t o = (int64_t)m * s.rank_pad + c + 32 * h;
        if (c + 32 * h < s.rank_pad) {
            s.hi[o] = __builtin_bit_cast(uint16_t, hv);
            s.lo[o] = __builtin_bit_cast(uint16_t, lv);
        }
    }
}

// ---- step 2 ---------------------------------------------------------------------
// acc += t @ Lb^T on the 16x16x32 MFMA for FN x FM blocks (n, m) of 16x16 at
// column n0, row m0 of the problem: lane l holds row 16 b + l % 16 and columns
// 16 a + 4 (l / 16) + 0..3.  The adapters of a row block are looped over with
// the FN blocks' contribution in registers of its own, and every accumulator
// is then changed once, in straight-line code: changing accumulators inside
// the loop made the register allocator spill them (756 registers on the
// 128x256 tile).  The Lb fragments stay in registers from row block to row
// block while the adapter does not change and the rank needs no more than one
// of them, as in a batch of prompts.
// GN of the FN column blocks are worked on at a time (8 with a 256-register
// wave, 4 where a copy wave shares the SIMD).
template <int GN, int FN, int FM>
__device__ __forceinline__ void adapter_add16(const Problem& p, f32x4 (&acc)[FN][FM], int m0, int n0)
{
    static_assert(FN % GN == 0, "whole groups of column blocks");
    const int lane = threadIdx.x & 63, lrow = lane & 15, lq = lane >> 4;
#pragma unroll
    for (int g = 0; g < FN; g += GN) {
        uint32_t nrow[GN];
        half8 x[GN];
#pragma unroll
        for (int a = 0; a < GN; ++a) {
            nrow[a] = (uint32_t)min(n0 + 16 * (g + a) + lrow, p.N - 1) * (uint32_t)p.rank;
            x[a] = (half8)(_Float16)0.0f;
        }
        int held = -1;  // the adapter whose first 32 ranks x holds
#pragma unroll
        for (int b = 0; b < FM; ++b) {
            const int m = m0 + 16 * b + lrow;
            const int id = adapter_of(p.ids, m, p.M, p.adapters);
            uint64_t todo = __ballot(id >= 0);
            const float sc = id >= 0 ? p.row_scale[m] : 0.0f;
            const int64_t trow = (int64_t)min(m, p.M - 1) * p.rank_pad + 8 * lq;
            f32x4 delta[GN] = {};
            while (todo) {
                const int l = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)todo) - 1);
                todo &= ~__ballot(id == l);
                const uint16_t* lb = p.lb + (int64_t)l * p.N * p.rank;
                for (int r = 0; r < p.rank_pad; r += 32) {
                    const half8 th = __builtin_bit_cast(half8, *(const u32x4*)(p.t_hi + trow + r));
                    const half8 tl = __builtin_bit_cast(half8, *(const u32x4*)(p.t_lo + trow + r));
                    if (held != l || p.rank_pad > 32) {
                        held = l;
#pragma unroll
                        for (int a = 0; a < GN; ++a)
                            x[a] = p.lb_vec ? piece8<true>(lb + nrow[a], r + 8 * lq, p.rank)
                                            : piece8<false>(lb + nrow[a], r + 8 * lq, p.rank);
                    }
#pragma unroll
                    for (int a = 0; a < GN; ++a) {
                        f32x4 d = {};
                        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[a], tl, d, 0, 0, 0);
                        d = __builtin_amdgcn_mfma_f32_16x16x32_f16(x[a], th, d, 0, 0, 0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) delta[a][i] += id == l ? sc * d[i] : 0.0f;
                    }
                }
            }
#pragma unroll
            for (int a = 0; a < GN; ++a) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[g + a][b][i] += delta[a][i];
                asm volatile("" : "+a"(acc[g + a][b]));  // back where the products left it
            }
        }
    }
}

// The same on the 32x32x16 MFMA, into accumulators that start with it, for TN x TM blocks of 32x32: lane l holds row
// 32 b + l % 32 and columns 32 a + 8 g + 4 (l / 32) + i in register 4 g + i.
// The work items (adapter, 16 ranks) are numbered; this wave takes items
// first, first + stride, ... (waves that each hold a share of the sum share
// them out), four at a time, so that their loads are in flight together.
template <int TN, int TM>
__device__ __forceinline__ void adapter_start32(const Problem& p, f32x16 (&acc)[TN][TM], int m0, int n0, int first, int stride)
{
    const int lane = threadIdx.x & 63, frow = lane & 31, fhi = lane >> 5;
    int id[TM], todo = 0;
    float sc[TM];
#pragma unroll
    for (int b = 0; b < TM; ++b) {
        const int m = m0 + 32 * b + frow;
        id[b] = adapter_of(p.ids, m, p.M, p.adapters);
        sc[b] = id[b] >= 0 ? p.row_scale[m] : 0.0f;
        todo |= (id[b] >= 0 ? 1 : 0) << b;
    }
    const int chunks = (p.rank + 15) / 16;
    int item = 0, l = -1, r = chunks;  // the next item: adapter l's ranks 16 r ..
    // the next item of this wave, or false
    auto next = [&](int& ol, int& orank) {
        for (;;) {
            if (r == chunks) {
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
                r = 0;
            }
            const bool mine = item % stride == first;
            ol = l, orank = 16 * r;
            ++item, ++r;
            if (mine) return true;
        }
    };
    constexpr int BATCH = 4;
    for (;;) {
        int ls[BATCH], rs[BATCH], n = 0;
        half8 x[BATCH][TN], th[BATCH][TM], tl[BATCH][TM];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            ls[j] = -1, rs[j] = 0;
            if (n == j && next(ls[j], rs[j])) ++n;
            if (n <= j) continue;
            const uint16_t* lb = p.lb + (int64_t)ls[j] * p.N * p.rank;
#pragma unroll
            for (int a = 0; a < TN; ++a) {
                const uint16_t* row = lb + (uint32_t)min(n0 + 32 * a + frow, p.N - 1) * (uint32_t)p.rank;
                x[j][a] = p.lb_vec ? piece8<true>(row, rs[j] + 8 * fhi, p.rank) : piece8<false>(row, rs[j] + 8 * fhi, p.rank);
            }
#pragma unroll
            for (int b = 0; b < TM; ++b) {
                const int64_t o = (int64_t)min(m0 + 32 * b + frow, p.M - 1) * p.rank_pad + rs[j] + 8 * fhi;
                th[j][b] = __builtin_bit_cast(half8, *(const u32x4*)(p.t_hi + o));
                tl[j][b] = __builtin_bit_cast(half8, *(const u32x4*)(p.t_lo + o));
            }
        }
        if (n == 0) return;
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
            if (j >= n) break;
#pragma unroll
            for (int b = 0; b < TM; ++b) {
                if (__ballot(id[b] == ls[j]) == 0) continue;
#pragma unroll
                for (int a = 0; a < TN; ++a) {
                    f32x16 d = {};
                    d = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[j][a], tl[j][b], d, 0, 0, 0);
                    d = __builtin_amdgcn_mfma_f32_32x32x16_f16(x[j][a], th[j][b], d, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[a][b][i] = id[b] == ls[j] ? acc[a][b][i] + sc[b] * d[i] : acc[a][b][i];
                }
            }
        }
        if (n < BATCH) return;
    }
}

}  // namespace gsr
