// gsr_adapters.hpp -- low-rank adapters beside a product: row m of
// C = act(alpha * A @ W + bias) uses W = B + s_l La_l^T Lb_l^T with l = ids[m]
// (rows whose id names no adapter: W = B).
//
// The sum over K is taken first, the rank last:
//   1. the adapter_shrink kernels: t[m, r] = s_l * sum_k A[m, k] La_l[r, k], fp32;
//   2. the product's own kernels add sum_r t[m, r] Lb_l[n, r] to their fp32
//      sums, so the adapter costs no pass over C and is scaled, biased and
//      activated with the sum it belongs to.
// Both steps run on the matrix cores with La and Lb as checkpoints hold them
// (rank x K and N x rank: the reduced index is contiguous, so a lane's operand
// is one 16-byte load and needs no LDS).
//
// t is an fp16 operand in step 2 without losing its fp32 value.  A row is
// scaled by the power of two that brings its largest |t| into [1, 2), and each
// value is split into its fp16 rounding and the fp16 rounding of the rest,
// which leaves at most 2^-23 of that largest value (hi has 11 bits, lo the 11
// bits below, down to fp16's smallest step of 2^-24).  The product runs over
// both halves and the power of two multiplies its fp32 result, so that holds
// over all of fp32's range.  Ranks go in chunks of 16: a chunk's
// record is its 16 hi values and then its 16 lo values, 64 bytes, the K = 32
// operand of one 16x16x32 MFMA against the chunk of Lb taken twice.
//
// Rows of one tile may belong to different adapters.  The loops run once per
// distinct adapter of the tile's rows; a lane of the accumulator layout holds
// one row, so a lane adds a result only if the adapter is its row's, and what
// another adapter's weights hold (NaN, infinities) cannot reach it.
#pragma once

#include "gsr_pipeline.hpp"

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
    float* t_scale;         // M
    float* partial;         // parts > 1: parts x (16 blocks) x (16 chunks)
    uint32_t* count;        // parts > 1: blocks
    int M, K, adapters, rank, chunks;
    int blocks;             // of 16 rows
    int parts, kchunk;      // K in parts of kchunk values (a multiple of 32)
    int slots;              // workgroups that share a block's adapters
    // one launch for both steps (gsr_kspec.hpp): the blocks' records are there
    // (flags), who is past looking (done), how often to look
    uint32_t* flags;
    uint32_t* done;
    int looks;
};

constexpr int kShrinkRows = 16;  // rows per workgroup
constexpr int kShrinkMaxRank = 256;

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

// The sums of 16 rows over this workgroup's part of K for NB chunks of ranks
// from chunk c0.  The W waves cut the part into runs of 32-value steps; a wave
// walks its run of every slots-th adapter of the rows (from `slot` on) and
// leaves what it has in sums[wave][row][rank].
//
// An MFMA operand has a row per lane, and a load in that layout touches 16
// rows with every 16 lanes: it ran at 10-12 bytes per clock and CU.  The
// 128-bit path so copies into LDS with neighbouring lanes on neighbouring
// bytes of a row (G 16-byte pieces of each of 16 rows per operand and batch),
// piece c of row r at place c ^ shrink_swz(r), from where the operand reads
// are free of bank conflicts.  A wave's LDS is its own: it waits for its
// copies, no barrier, with DEPTH batches in flight across the ends of
// adapters.
template <int NB_, int W_, int G_, int DEPTH_>
struct ShrinkCfg {
    static constexpr int NB = NB_, W = W_, G = G_, DEPTH = DEPTH_;
    static constexpr int OPER = 16 * G * 16;           // bytes of one operand's batch
    static constexpr int BATCH = (1 + NB) * OPER;
    static constexpr int COPIES = (1 + NB) * OPER / 1024;
    static constexpr int RANKS = kAdapterChunk * NB + 4;  // row of the sums, padded
    static constexpr int SUM_BYTES = W * kShrinkRows * RANKS * 4;
    static constexpr int LDS_BYTES = W * DEPTH * BATCH > SUM_BYTES ? W * DEPTH * BATCH : SUM_BYTES;
    static_assert(G == 8 || G == 16, "pieces per row");
    static_assert(SUM_BYTES + kShrinkRows * 8 <= LDS_BYTES, "the rows' maxima fit behind the sums");
    static_assert(LDS_BYTES <= 160 * 1024 && COPIES * DEPTH < 64, "LDS of a workgroup; the vmcnt field");
};

// Distinct places for one piece of 16 rows in the 256 bytes the LDS serves at
// once: rows of 256 bytes (G = 16) or pairs of rows of 128 (G = 8).
template <int G>
__device__ __forceinline__ int shrink_swz(int r) { return G == 16 ? (r & 15) : ((r >> 1) & 7); }

template <bool VEC, class T>
__device__ __forceinline__ void shrink_sums(const ShrinkArgs& s, uint8_t* smem, int id, int m0, int c0, int kbeg, int kend, int slot,
                                            int slots)
{
    constexpr int NB = T::NB, W = T::W, G = T::G, STEPS = G / 4;
    const int lane = threadIdx.x & 63, lrow = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int steps = (kend - kbeg + 31) / 32;
    const int ks0 = steps * wave / W, ks1 = steps * (wave + 1) / W;
    f32x4 out[NB] = {};
    if constexpr (VEC) {
        const i32x4 ra = raw_rsrc(s.A, (uint32_t)s.M * (uint32_t)s.K * 2u);
        const uint32_t lds0 = lds_address(smem) + (uint32_t)(wave * T::DEPTH * T::BATCH);
        const uint8_t* const base = smem + wave * T::DEPTH * T::BATCH;
        const int batches = (ks1 - ks0 + STEPS - 1) / STEPS, klim = min(kend, kbeg + 32 * ks1);
        // a walk over (adapter, batch): the copies' walk runs DEPTH - 1 ahead of the products'
        struct Walk {
            uint64_t todo;
            int at, l, b;
        };
        auto advance = [&](Walk& w) {  // to the next unit of this workgroup's; l = -1 at the end
            if (++w.b < batches && w.l >= 0) return;
            w.b = 0;
            w.l = -1;
            while (w.todo != 0) {
                const int l = __builtin_amdgcn_readlane(id, __ffsll((unsigned long long)w.todo) - 1);
                w.todo &= ~__ballot(id == l);
                if (w.at++ % slots == slot) {
                    w.l = l;
                    return;
                }
            }
        };
        auto copy = [&](const Walk& w, int buf) {
            const i32x4 rl = raw_rsrc(s.la + (int64_t)w.l * s.rank * s.K, (uint32_t)s.rank * (uint32_t)s.K * 2u);
            const int k0 = kbeg + 32 * (ks0 + w.b * STEPS);
#pragma unroll
            for (int o = 0; o < 1 + NB; ++o)
#pragma unroll
                for (int j = 0; j < T::OPER / 1024; ++j) {
                    const int r = (64 / G) * j + lane / G;  // of the operand's 16 rows
                    const int k = k0 + 8 * ((lane % G) ^ shrink_swz<G>(r));
                    const int row = o == 0 ? m0 + r : kAdapterChunk * (c0 + o - 1) + r;
                    const bool in = k < klim && row < (o == 0 ? s.M : s.rank);
                    copy16_to_lds(o == 0 ? ra : rl, in ? ((uint32_t)row * (uint32_t)s.K + (uint32_t)k) * 2u : kOutOfRange,
                                  lds0 + (uint32_t)(buf * T::BATCH + o * T::OPER + j * 1024));
                }
        };
        Walk ahead{__ballot(id >= 0), 0, -1, 0}, here;
        if (batches <= 0) ahead.todo = 0;
        advance(ahead);
        here = ahead;
        int flying = 0, put = 0, get = 0;
        f32x4 d[NB] = {};
        while (here.l >= 0) {
            while (flying < T::DEPTH && ahead.l >= 0) {
                copy(ahead, put);
                put = put + 1 == T::DEPTH ? 0 : put + 1;
                ++flying;
                advance(ahead);
            }
            if (flying == T::DEPTH) wait_vmcnt<T::COPIES * (T::DEPTH - 1)>();
            else wait_vmcnt<0>();
            const uint8_t* buf = base + get * T::BATCH;
#pragma unroll
            for (int i = 0; i < STEPS; ++i) {
                const int place = lrow * (G * 16) + ((4 * i + lq) ^ shrink_swz<G>(lrow)) * 16;
                const half8 x = __builtin_bit_cast(half8, *(const u32x4*)(buf + place));
#pragma unroll
                for (int q = 0; q < NB; ++q)
                    d[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                        __builtin_bit_cast(half8, *(const u32x4*)(buf + (1 + q) * T::OPER + place)), x, d[q], 0, 0, 0);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next copies land here
            get = get + 1 == T::DEPTH ? 0 : get + 1;
            --flying;
            const int l = here.l;
            advance(here);
            if (here.b == 0) {  // the adapter's run is complete
#pragma unroll
                for (int q = 0; q < NB; ++q)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        out[q][i] = id == l ? out[q][i] + d[q][i] : out[q][i];
                        d[q][i] = 0.0f;
                    }
            }
        }
    } else {
        // Unaligned rows: 16 bytes from the dword at or below a piece and the
        // dword after it, shifted together, BATCH steps at a time; the steps
        // that those could read past the end of K from, value by value.
        // (All value by value, 4662 rows, K 557, rank 128: 118 us.)
        constexpr int BATCH = 2;
        const uint32_t amis = (uint32_t)(uintptr_t)s.A & 2u;
        const __amdgpu_buffer_rsrc_t ra = make_rsrc((const uint8_t*)s.A - amis, (uint32_t)s.M * (uint32_t)s.K * 2u + amis);
        const uint32_t arow = (uint32_t)(m0 + lrow) * (uint32_t)s.K + amis / 2u;
        const bool ain = m0 + lrow < s.M;
        const int whole = min(max((min(kend, s.K - 2) - kbeg) / 32, ks0), ks1);  // steps before this one end before that
        int at = 0;
        for_each_adapter(id, [&](int l) {
            if (at++ % slots != slot) return;
            const uint16_t* la = s.la + (int64_t)l * s.rank * s.K;
            const uint32_t lmis = (uint32_t)(uintptr_t)la & 2u;
            const __amdgpu_buffer_rsrc_t rl = make_rsrc((const uint8_t*)la - lmis, (uint32_t)s.rank * (uint32_t)s.K * 2u + lmis);
            f32x4 d[NB] = {};
            auto steps_of = [&](auto count, int ks, auto&& piece) {
                constexpr int N = decltype(count)::value;
                half8 x[N], w[N][NB];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int k = kbeg + 32 * (ks + i) + 8 * lq;
                    x[i] = piece(ra, arow, k, ain);
#pragma unroll
                    for (int q = 0; q < NB; ++q) {
                        const int r = kAdapterChunk * (c0 + q) + lrow;
                        w[i][q] = piece(rl, (uint32_t)r * (uint32_t)s.K + lmis / 2u, k, r < s.rank);
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i)
#pragma unroll
                    for (int q = 0; q < NB; ++q) d[q] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[i][q], x[i], d[q], 0, 0, 0);
            };
            auto wide = [&](__amdgpu_buffer_rsrc_t rs, uint32_t row, int k, bool in) {
                return __builtin_bit_cast(half8, load8_whole<2>(rs, (row + (uint32_t)k) * 2u, in));
            };
            auto narrow = [&](__amdgpu_buffer_rsrc_t rs, uint32_t row, int k, bool in) {
                return piece8<false>(rs, row, k, kend, in);
            };
            int ks = ks0;
            for (; ks + BATCH <= whole; ks += BATCH) steps_of(std::integral_constant<int, BATCH>{}, ks, wide);
            for (; ks < whole; ++ks) steps_of(std::integral_constant<int, 1>{}, ks, wide);
            for (; ks < ks1; ++ks) steps_of(std::integral_constant<int, 1>{}, ks, narrow);
#pragma unroll
            for (int q = 0; q < NB; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) out[q][i] = id == l ? out[q][i] + d[q][i] : out[q][i];
        });
    }
    __syncthreads();  // the sums take the place of every wave's batches
    float* const sums = (float*)smem;
#pragma unroll
    for (int q = 0; q < NB; ++q) *(f32x4*)(sums + (wave * kShrinkRows + lrow) * T::RANKS + 16 * q + 4 * lq) = out[q];
    __syncthreads();
}

// Row `row`, rank c of chunk q, summed over the waves.
template <class T>
__device__ __forceinline__ float shrink_sum(const uint8_t* smem, int row, int q, int c)
{
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < T::W; ++w) v += ((const float*)smem)[(w * kShrinkRows + row) * T::RANKS + 16 * q + c];
    return v;
}

// The scaled sum of rank c of chunk j: 0 past the last rank, where zeros in La's
// place met whatever A and the scale hold (NaN for an infinity or a NaN).
__device__ __forceinline__ float shrink_rank(const ShrinkArgs& s, int j, int c, float sum)
{
    return kAdapterChunk * j + c < s.rank ? sum : 0.0f;
}

// Writes the records of row `row` of t and t_scale: this thread holds ranks
// c + 16 j of the row for j in v[], the 16 lanes around it the rest.  With
// device-scope stores, for readers in the same launch.
template <int N>
__device__ __forceinline__ void shrink_store(const ShrinkArgs& s, uint16_t* t, float* t_scale, int64_t row, int l, int c,
                                             int j0, int stride, const float (&v)[N], float big)
{
    if (l < 0) return;
    const bool odd = !(big < __builtin_inff());
    // 2^e <= big < 2^(e + 1), or the least normal number's 2^e; zeros keep 2^0
    int e = 0;
    if (!odd && big > 0.0f) e = max(__builtin_amdgcn_frexp_expf(big) - 1, -126);
    // the power of two, negative for a row with an infinity or a NaN
    if (c == 0 && j0 == 0)
        __hip_atomic_store(t_scale + row, odd ? -1.0f : ldexpf(1.0f, e), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int j = j0 + i * stride;
        if (j >= s.chunks) break;
        const float x = ldexpf(v[i], -e);
        // The hi half has the value's sign, for the products with infinities of Lb:
        // fp16's smallest step where it would be zero.  In a row with an infinity
        // or a NaN, which makes one of every sum, the other values are their signs
        // alone (they may be past fp16's range).
        const float sign = v[i] > 0.0f ? 1.0f : v[i] < 0.0f ? -1.0f : 0.0f;
        _Float16 hi = (_Float16)x, lo = (_Float16)0.0f;
        if (!odd) {
            if (hi == (_Float16)0.0f) hi = (_Float16)(sign * 0x1p-24f);
            lo = (_Float16)(x - (float)hi);
        } else if (fabsf(v[i]) < __builtin_inff()) {
            hi = (_Float16)sign;
        }
        uint16_t* rec = t + (row * s.chunks + j) * 32;
        __hip_atomic_store(rec + c, __builtin_bit_cast(uint16_t, hi), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __hip_atomic_store(rec + 16 + c, __builtin_bit_cast(uint16_t, lo), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}

// Many rows: a workgroup takes 16 rows, every slots-th of their adapters and
// all ranks, T::NB chunks at a time, with eight waves on K.  A is read once
// (from the caches for further chunks) and an adapter's La once per 16 rows
// from the caches, so the copies into LDS bound it: 4096 rows of 8 adapters,
// K 4096 (34 MB of A: 6.6 us at the rate of a copy), rank 16 14.8 us, 64 19.5,
// 128 27.5 (operands read in their MFMA layout: 16.3, 28.6 and 47.5).
typedef ShrinkCfg<1, 8, 16, 2> ShrinkRows1;
typedef ShrinkCfg<4, 8, 8, 2> ShrinkRows4;

template <bool VEC, class T>
__global__ void __launch_bounds__(512) adapter_shrink_rows_kernel(ShrinkArgs s)
{
    constexpr int NB = T::NB, QT = 2, PER = (NB + QT - 1) / QT;        // chunks at a time per thread
    constexpr int ROUNDS = NB == 1 ? 1 : kShrinkMaxRank / kAdapterChunk / NB;
    static_assert(T::W == 8, "512 threads");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[T::LDS_BYTES];
    const int tid = threadIdx.x, m0 = blockIdx.x * kShrinkRows;
    const int id = adapter_of(s.ids, m0 + (tid & 15), s.M, s.adapters);

    // thread t: row t / 16 % 16 and rank t % 16 of chunks t / 256, + 2, ...
    const int row = (tid >> 4) & 15, c = tid & 15, q = tid >> 8;
    int l = adapter_of(s.ids, m0 + row, s.M, s.adapters), at = 0;
    bool mine = false;
    for_each_adapter(id, [&](int a) { mine |= at++ % s.slots == (int)blockIdx.z && l == a; });
    if (at <= (int)blockIdx.z) return;  // no adapter for this workgroup
    l = mine ? l : -1;
    const float scale = (l >= 0 && s.scales != nullptr) ? s.scales[l] : 1.0f;
    float v[ROUNDS * PER], big = 0.0f;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < ROUNDS; ++i) {
#pragma unroll
        for (int j = 0; j < PER; ++j) v[i * PER + j] = 0.0f;
        if (i * NB >= s.chunks) continue;
        if (i > 0) __syncthreads();  // the sums of the chunks before have been read
        shrink_sums<VEC, T>(s, smem, id, m0, i * NB, 0, s.K, blockIdx.z, s.slots);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int cq = q + QT * j;
            if (cq >= NB || i * NB + cq >= s.chunks) continue;
            const float u = shrink_rank(s, i * NB + cq, c, shrink_sum<T>(smem, row, cq, c) * scale);
            v[i * PER + j] = u;
            odd |= !(fabsf(u) < __builtin_inff());
            big = fmaxf(big, fabsf(u));
        }
    }
    big = odd ? __builtin_inff() : big;
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) big = fmaxf(big, __shfl_xor(big, x));
    if (NB > 1) {
        float* const bigs = (float*)(smem + T::SUM_BYTES) + row * QT;  // behind the sums others still read
        if (c == 0) bigs[q] = big;
        __syncthreads();
        big = fmaxf(bigs[0], bigs[1]);
    }
    if (q < NB) shrink_store(s, s.t, s.t_scale, m0 + row, l, c, q, QT, v, big);
}

// Few rows (a decode step): the adapters' La is most of the bytes, so a block
// of 16 rows spreads over workgroups of four waves, one per part of K, chunk
// and every slots-th adapter, which meet in the workspace: the workgroup of a
// block that arrives last adds the parts in part order and writes the records
// (device-scope accesses and the arrival counter as in KsSum::split_sum_store,
// so no order depends on timing and no workgroup waits).  Bound by latency (a
// launch, a walk of K / parts, the meeting): 12.6 us for 16 rows of 16
// adapters of rank 64, K 4096 (8.4 MB of La).
typedef ShrinkCfg<1, 8, 8, 2> ShrinkParts;

// The finished row of a block: `at` gives the thread's rank c of chunk j summed
// over the parts; scaled, with the row's largest value.
template <int N, class F>
__device__ __forceinline__ float shrink_row(const ShrinkArgs& s, int l, int c, float (&v)[N], F&& at)
{
    const float scale = (l >= 0 && s.scales != nullptr) ? s.scales[l] : 1.0f;
    float big = 0.0f;
    bool odd = false;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        v[j] = j < s.chunks ? shrink_rank(s, j, c, at(j) * scale) : 0.0f;
        odd |= !(fabsf(v[j]) < __builtin_inff());
        big = fmaxf(big, fabsf(v[j]));
    }
    big = odd ? __builtin_inff() : big;
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) big = fmaxf(big, __shfl_xor(big, x));
    return big;
}

constexpr int kShrinkRounds = kShrinkMaxRank / kAdapterChunk;

// Workgroup `wg` of blocks x parts x chunks x slots, all 512 threads; true in
// every thread of the one that wrote its block's records.
template <bool VEC>
__device__ __forceinline__ bool shrink_part(const ShrinkArgs& s, uint8_t* smem, int* last, int wg)
{
    using T = ShrinkParts;
    static_assert(T::W == 8 && T::NB == 1, "512 threads, one chunk");
    const int tid = threadIdx.x;
    const int block = wg % s.blocks, part = wg / s.blocks % s.parts, chunk = wg / (s.blocks * s.parts) % s.chunks;
    const int slot = wg / (s.blocks * s.parts * s.chunks);
    const int m0 = block * kShrinkRows;
    const int id = adapter_of(s.ids, m0 + (tid & 15), s.M, s.adapters);
    if (__ballot(id >= 0) == 0) return false;  // in every workgroup of the block
    const int row = (tid >> 4) & 15, c = tid & 15;  // threads 0..255: row t / 16, rank t % 16 of a chunk
    const int l = tid < 256 ? adapter_of(s.ids, m0 + row, s.M, s.adapters) : -1;
    // the adapter's place among the block's decides whose it is
    bool mine = false;
    int at = 0;
    for_each_adapter(id, [&](int a) { mine |= at++ % s.slots == slot && l == a; });

    const int64_t stride = (int64_t)s.blocks * kShrinkRows * s.chunks * kAdapterChunk;  // one part
    float* const mine0 = s.partial + (int64_t)(m0 + row) * s.chunks * kAdapterChunk + c;
    if (at > slot) {  // there is an adapter for this workgroup
        const int kbeg = part * s.kchunk, kend = min(s.K, kbeg + s.kchunk);
        shrink_sums<VEC, T>(s, smem, id, m0, chunk, kbeg, kend, slot, s.slots);
        if (mine)
            __hip_atomic_store(mine0 + part * stride + chunk * kAdapterChunk, shrink_sum<T>(smem, row, 0, c),
                               __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's sums have reached device scope
        __syncthreads();
    }
    if (tid == 0) {
        const uint32_t before = __hip_atomic_fetch_add(s.count + block, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *last = before == (uint32_t)(s.parts * s.chunks * s.slots) - 1u;
    }
    __syncthreads();
    if (!__builtin_amdgcn_readfirstlane(*last)) return false;
    if (tid == 0) __hip_atomic_store(s.count + block, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (tid < 256) {
        float v[kShrinkRounds];
        const float big = shrink_row(s, l, c, v, [&](int j) {
            float sum = 0.0f;
            for (int g = 0; g < s.parts; g += 8) {
                float u[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)  // parts past the last read its sums again and add nothing
                    u[i] = __hip_atomic_load(mine0 + min(g + i, s.parts - 1) * stride + j * kAdapterChunk, __ATOMIC_RELAXED,
                                             __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
                for (int i = 0; i < 8; ++i) sum += g + i < s.parts ? u[i] : 0.0f;
            }
            return sum;
        });
        shrink_store(s, s.t, s.t_scale, m0 + row, l, c, 0, 1, v, big);
    }
    return true;
}

template <bool VEC>
__global__ void __launch_bounds__(512) adapter_shrink_parts_kernel(ShrinkArgs s)
{
    __shared__ __attribute__((aligned(1024))) uint8_t smem[ShrinkParts::LDS_BYTES];
    __shared__ int last;
    shrink_part<VEC>(s, smem, &last, blockIdx.x);
}

// ---- both steps in one launch (few rows) -------------------------------------------
// The workgroups of step 1 come first in the grid; a tile's workgroup needs
// their records only after its loop over K, when they have usually been there
// for long.  It looks for them a limited number of times and, not having found
// them, makes them itself in LDS, with the same sums in the same order: no
// workgroup depends on another one's running, and the bits are the same either
// way.  A decode step saves a launch and hides the sums behind the weights'
// bytes: 1 x 4096 x 11008, rank 64, 28 -> 21 us, 16 x 11008 x 4096 with 16
// adapters of rank 16 30 -> 26 us, where reading B alone at the rate of a copy
// is 18.  A block's records are announced by its flag.  Who writes a flag, and
// every workgroup that is past looking, counts in `done`; the last of them all
// puts flags and count back to zero.
//
// Bit b: block b (of at most four, M <= 64) has rows with an adapter.
__device__ __forceinline__ uint32_t active_blocks(const ShrinkArgs& s)
{
    const uint64_t rows = __ballot(adapter_of(s.ids, threadIdx.x & 63, s.M, s.adapters) >= 0);
    uint32_t m = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) m |= ((rows >> (16 * b)) & 0xffffull) ? 1u << b : 0u;
    return m;
}

// One arrival at `done`; the last of tiles + active blocks clears.  One lane.
__device__ __forceinline__ void shrink_done(const ShrinkArgs& s, int tiles, uint32_t active)
{
    const uint32_t before = __hip_atomic_fetch_add(s.done, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (before != (uint32_t)(tiles + __popc(active)) - 1u) return;
#pragma unroll
    for (int b = 0; b < 4; ++b) __hip_atomic_store(s.flags + b, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(s.done, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// A workgroup of step 1 in the common grid.
template <bool VEC>
__device__ __forceinline__ void shrink_announce(const ShrinkArgs& s, uint8_t* smem, int* last, int wg, int tiles)
{
    if (!shrink_part<VEC>(s, smem, last, wg)) return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's records have reached device scope
    __syncthreads();
    const uint32_t active = active_blocks(s);
    if (threadIdx.x == 0) {
        __hip_atomic_store(s.flags + wg % s.blocks, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the flag is set before whoever counts last clears it
        shrink_done(s, tiles, active);
    }
}

// One wave of a tile's workgroup, whose rows have adapters in the blocks of
// `want`: looks until their records are there, at most s.looks times.  True:
// they are.
__device__ __forceinline__ bool shrink_look(const ShrinkArgs& s, uint32_t want)
{
    const int lane = threadIdx.x & 63;
    const bool ask = lane < 4 && ((want >> lane) & 1u);
    bool there = __ballot(ask) == 0;
    for (int i = 0; i < s.looks && !there; ++i) {
        const uint32_t f = ask ? __hip_atomic_load(s.flags + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 1u;
        there = __ballot(f == 0u) == 0;
    }
    return there;
}

// The records of rows m0 .. m0 + rows - 1 (a multiple of 16 of them) made by
// the tile's own workgroup of 512 threads, into t and t_scale in LDS behind the
// ShrinkParts::LDS_BYTES that the sums take.
template <bool VEC>
__device__ __forceinline__ void shrink_here(const ShrinkArgs& s, uint8_t* smem, uint16_t* t, float* t_scale, int m0, int rows)
{
    using T = ShrinkParts;
    const int tid = threadIdx.x, row = (tid >> 4) & 15, c = tid & 15;
    for (int b0 = 0; b0 < rows; b0 += kShrinkRows) {
        const int id = adapter_of(s.ids, m0 + b0 + (tid & 15), s.M, s.adapters);
        if (__ballot(id >= 0) == 0) continue;
        const int l = tid < 256 ? adapter_of(s.ids, m0 + b0 + row, s.M, s.adapters) : -1;
        const float scale = (l >= 0 && s.scales != nullptr) ? s.scales[l] : 1.0f;
        // the row's fp32 values wait in the place of its records
        uint8_t* const wait = (uint8_t*)(t + (int64_t)(b0 + row) * s.chunks * 32) + 4 * c;
        float big = 0.0f;
        bool odd = false;
        for (int j = 0; j < s.chunks; ++j) {
            float v[1] = {0.0f};
            for (int g = 0; g < s.parts; ++g) {
                __syncthreads();  // the sums before have been read
                shrink_sums<VEC, T>(s, smem, id, m0 + b0, j, g * s.kchunk, min(s.K, (g + 1) * s.kchunk), 0, 1);
                v[0] += shrink_sum<T>(smem, row, 0, c);
            }
            v[0] = shrink_rank(s, j, c, v[0] * scale);
            odd |= !(fabsf(v[0]) < __builtin_inff());
            big = fmaxf(big, fabsf(v[0]));
            if (tid < 256) *(volatile float*)(wait + 64 * j) = v[0];
        }
        big = odd ? __builtin_inff() : big;
#pragma unroll
        for (int x = 8; x > 0; x >>= 1) big = fmaxf(big, __shfl_xor(big, x));
        if (tid < 256)
            for (int j = 0; j < s.chunks; ++j) {
                const float v[1] = {*(volatile float*)(wait + 64 * j)};  // the row's 16 lanes read before one writes
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                shrink_store(s, t, t_scale, b0 + row, l, c, j, 1, v, big);
            }
    }
    __syncthreads();
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

// acc += x^T-block * y-block with the accumulator in AGPRs before and after.
// Not mfma16_inplace: its operands come from vector instructions and the
// accumulators around it may be moved, so the compiler has to see a matrix
// instruction to keep the wait states these need.
__device__ __forceinline__ void mfma16_pinned(f32x4& acc, const half8& x, const half8& y)
{
    acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, acc, 0, 0, 0);
    asm volatile("" : "+a"(acc));
}

// Bits 15 and 31 set where a half of `d` is an infinity or a NaN.
__device__ __forceinline__ uint32_t nonfinite2(uint32_t d) { return ((d & 0x7c007c00u) + 0x04000400u) & 0x80008000u; }

// `seen`, all zeros at first, gets a NaN where v has an infinity or a NaN (one
// packed instruction per two values); any_odd tells whether it has any.
__device__ __forceinline__ half8 look_odd(half8 v, half8 seen) { return __builtin_elementwise_fma(v, (half8)(_Float16)0.0f, seen); }
__device__ __forceinline__ bool any_odd(half8 seen)
{
    const u32x4 w = __builtin_bit_cast(u32x4, seen);
    return (w[0] | w[1] | w[2] | w[3]) != 0u;
}

// v with zeros in the place of infinities and NaN.
__device__ __forceinline__ half8 finite8(half8 v)
{
    u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] &= ~((nonfinite2(w[i]) >> 15) * 0xffffu);
    return __builtin_bit_cast(half8, w);
}

// acc, all zeros, becomes t @ Lb^T on the 16x16x32 MFMA for FN x FM blocks
// (n, m) of 16x16 at column n0, row m0 of the problem: lane l holds row
// 16 b + l % 16 and columns 16 a + 4 (l / 16) + 0..3.  One MFMA per block and
// chunk: lanes 0-31 hold hi, lanes 32-63 lo.
//
// It runs before the product's loop, behind the first operand copies, because
// the registers of the loop's operands are free then: the records of all row
// blocks and an adapter's fragments for all column blocks (CB chunks of each)
// are requested together, so a tile whose rows share an adapter waits once per
// CB chunks.  Accumulators are changed by matrix instructions alone inside the
// loop over adapters (changing them with vector instructions there made the
// register allocator spill them), so the rows of other adapters take part with
// t = 0, and the rows' scales multiply all accumulators once at the end.
// (4097 x 11008 x 4096 with 9 runs of rank 16 takes 318 us in all beside 294
// with no row's id an adapter's, 14 of them the inner sums'; rank 64 350, 22.)
// 0 * infinity and 0 * NaN would then reach those rows: infinities and NaN of Lb
// have zeros in their place, rows of t with such values take no part, and the
// caller, told so by the returned true, runs adapter_nonfinite16 before its
// epilogue.
template <int CB, bool VEC, int FN, int FM>
__device__ __forceinline__ bool adapter_start16(const Problem& p, f32x4 (&acc)[FN][FM], int m0, int n0)
{
    const int lane = threadIdx.x & 63, lrow = lane & 15, lq = lane >> 4;
    // buffers that start at this wave's first row: 32-bit offsets, and zeros past the last row
    const uint32_t rows = (uint32_t)max(min(p.M - m0, 16 * FM), 0), rec_bytes = (uint32_t)p.chunks * 64u;
    const __amdgpu_buffer_rsrc_t rid = make_rsrc(p.ids + m0, rows * 4u);
    const __amdgpu_buffer_rsrc_t rsc = make_rsrc(p.t_scale + m0, rows * 4u);
    const __amdgpu_buffer_rsrc_t rt = make_rsrc(p.t + (int64_t)m0 * p.chunks * 32, rows * rec_bytes);
    int id[FM], all = 0;
    bool odd = false;
    float sc[FM];
#pragma unroll
    for (int b = 0; b < FM; ++b) id[b] = (int)__builtin_amdgcn_raw_buffer_load_b32(rid, (uint32_t)(16 * b + lrow) * 4u, 0, 0);
#pragma unroll
    for (int b = 0; b < FM; ++b) sc[b] = __builtin_bit_cast(float, __builtin_amdgcn_raw_buffer_load_b32(rsc, (uint32_t)(16 * b + lrow) * 4u, 0, 0));
#pragma unroll
    for (int b = 0; b < FM; ++b) {
        if ((uint32_t)(16 * b + lrow) >= rows || (uint32_t)id[b] >= (uint32_t)p.adapters) id[b] = -1, sc[b] = 1.0f;
        odd |= sc[b] < 0.0f;
        if (sc[b] < 0.0f) id[b] = -1, sc[b] = 1.0f;  // all of such a row is adapter_nonfinite16's
        all |= (id[b] >= 0 ? 1 : 0) << b;
    }
    odd = __ballot(odd) != 0;
    if (__ballot(all != 0) == 0) return odd;
    for (int c = 0; c < p.chunks; c += CB) {
        half8 t[CB][FM];
#pragma unroll
        for (int j = 0; j < CB; ++j)
#pragma unroll
            for (int b = 0; b < FM; ++b)
                t[j][b] = __builtin_bit_cast(half8, __builtin_amdgcn_raw_buffer_load_b128(  // zeros past the last chunk
                    rt, c + j < p.chunks ? (uint32_t)(16 * b + lrow) * rec_bytes + (uint32_t)(c + j) * 64u + 16u * (uint32_t)lq
                                         : kOutOfRange, 0, 0));
        int todo = all;
        while (const uint64_t any = __ballot(todo != 0)) {
            const int src = __ffsll((unsigned long long)any) - 1;
            const int tb = __ffs(__builtin_amdgcn_readlane(todo, src)) - 1;
            int v = id[0];
#pragma unroll
            for (int b = 1; b < FM; ++b) v = tb == b ? id[b] : v;
            const int l = __builtin_amdgcn_readlane(v, src);
            const __amdgpu_buffer_rsrc_t rl = lb_rsrc(p, l);
            half8 x[CB][FN];  // chunks past the last are zeros
#pragma unroll
            for (int j = 0; j < CB; ++j)
#pragma unroll
                for (int a = 0; a < FN; ++a) {
                    const int n = n0 + 16 * a + lrow;
                    x[j][a] = piece8<VEC>(rl, (uint32_t)n * (uint32_t)p.rank, kAdapterChunk * (c + j) + 8 * (lq & 1),
                                          p.rank, n < p.N);
                    // value by value: one fragment at a time, for the registers' sake
                    if constexpr (!VEC) asm volatile("" : "+v"(x[j][a]));
                }
            half8 seen = (half8)(_Float16)0.0f;
#pragma unroll
            for (int j = 0; j < CB; ++j)
#pragma unroll
                for (int a = 0; a < FN; ++a) seen = look_odd(x[j][a], seen);
            if (__ballot(any_odd(seen)) != 0) {
                odd = true;
#pragma unroll
                for (int j = 0; j < CB; ++j)
#pragma unroll
                    for (int a = 0; a < FN; ++a) x[j][a] = finite8(x[j][a]);
            }
#pragma unroll
            for (int b = 0; b < FM; ++b) {
                if (__ballot(id[b] == l) == 0) continue;
                if (id[b] == l) todo &= ~(1 << b);
#pragma unroll
                for (int j = 0; j < CB; ++j) {
                    const half8 y = id[b] == l ? t[j][b] : (half8)(_Float16)0.0f;
#pragma unroll
                    for (int a = 0; a < FN; ++a) mfma16_pinned(acc[a][b], x[j][a], y);
                }
            }
        }
    }
    // a matrix result may be read by other instructions after 18 wait states
    asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < FM; ++b)
#pragma unroll
        for (int a = 0; a < FN; ++a) {
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[a][b][i] *= sc[b];
            asm volatile("" : "+a"(acc[a][b]));  // where the product's loop wants them
        }
    return odd;
}

// What adapter_start16 left out: acc += what the infinities and NaN of t and Lb
// make of each sum.  A sum with one is an infinity or a NaN, and which is
// told by the hi half of t alone, which has the sign of t; finite sums are
// left alone, and so are the rows of other adapters, which share the matrix
// instructions.  Four blocks of columns at a time, for the registers' sake, and
// behind the product's loop: in front of it the 256x256 tile spilled 55 registers
// instead of 29.
template <bool VEC, int FN, int FM>
__device__ __forceinline__ void adapter_nonfinite16(const Problem& p, f32x4 (&acc)[FN][FM], int m0, int n0)
{
    int lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane), "+s"(m0), "+s"(n0));  // nothing of this is made before the product's loop and kept across it
    const int lrow = lane & 15, lq = lane >> 4;
    constexpr int GROUP = 4;
    static_assert(FN % GROUP == 0, "blocks of columns");
#pragma unroll
    for (int b = 0; b < FM; ++b) {
        const int id = adapter_of(p.ids, m0 + 16 * b + lrow, p.M, p.adapters);
        const uint16_t* const rec = p.t + (int64_t)(id >= 0 ? m0 + 16 * b + lrow : 0) * p.chunks * 32 + 8 * (lq & 1);
#pragma unroll
        for (int a0 = 0; a0 < FN; a0 += GROUP) {
            f32x4 sum[GROUP] = {};
            for_each_adapter(id, [&](int l) {
                const __amdgpu_buffer_rsrc_t rl = lb_rsrc(p, l);
#pragma unroll 1
                for (int c = 0; c < p.chunks; ++c) {
                    const bool hi = lq < 2;  // the MFMA's other half of K is zeros
                    const half8 y = hi ? __builtin_bit_cast(half8, *(const u32x4*)(rec + 32 * c)) : (half8)(_Float16)0.0f;
#pragma unroll
                    for (int a = 0; a < GROUP; ++a) {
                        const int n = n0 + 16 * (a0 + a) + lrow;
                        const half8 x = piece8<VEC>(rl, (uint32_t)n * (uint32_t)p.rank, kAdapterChunk * c + 8 * (lq & 1), p.rank,
                                                    hi && n < p.N);
                        const f32x4 d = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, y, f32x4{}, 0, 0, 0);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            sum[a][i] += (id == l && !(fabsf(d[i]) < __builtin_inff())) ? d[i] : 0.0f;
                    }
                }
            });
#pragma unroll
            for (int a = 0; a < GROUP; ++a) {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[a0 + a][b][i] += sum[a][i];
                asm volatile("" : "+a"(acc[a0 + a][b]));
            }
        }
    }
}

// The same on the 32x32x16 MFMA for TN x TM blocks of 32x32: lane l holds row
// 32 b + l % 32 and columns 32 a + 8 g + 4 (l / 32) + i in register 4 g + i.
// The work items (adapter, chunk) are numbered; a wave takes items first,
// first + stride, ... (waves that each hold a share of the sum share them
// out) in batches whose loads are in flight together: load() requests one,
// apply() adds it, so one can be in flight behind the product.
//
// SHARED: the records come from workgroups of the same launch (device-scope
// loads) or from LDS, and are there only once records() has been told where;
// until then a batch holds Lb's side alone.
template <int TN, int TM, bool SHARED>
struct AdapterItems {
    int m0, n0, first, stride;
    const uint16_t* t;        // records, of the problem's rows from row t_row on
    const float* t_scale;
    int t_row;
    int id[TM], todo = 0;
    float sc[TM];             // the rows' scales
    int item = 0, l = -1, c;  // the next item: adapter l's chunk c

    template <int B>
    struct Batch {
        int n = 0, ls[B], ch[B];  // its size, its adapters and their chunks
        half8 x[B][TN], hi[B][TM], lo[B][TM];
    };

    __device__ __forceinline__ AdapterItems(const Problem& p, int m0_, int n0_, int first_, int stride_)
        : m0(m0_), n0(n0_), first(first_), stride(stride_), t(p.t), t_scale(p.t_scale), t_row(0), c(p.chunks)
    {
#pragma unroll
        for (int b = 0; b < TM; ++b) id[b] = adapter_of(p.ids, row_of(b), p.M, p.adapters);
    }

    // once the ids have come
    __device__ __forceinline__ void start()
    {
#pragma unroll
        for (int b = 0; b < TM; ++b) todo |= (id[b] >= 0 ? 1 : 0) << b;
        if constexpr (!SHARED) scales();
    }

    __device__ __forceinline__ int row_of(int b) const { return m0 + 32 * b + (int)(threadIdx.x & 31); }

    __device__ __forceinline__ void scales()
    {
#pragma unroll
        for (int b = 0; b < TM; ++b) {
            const float* at = t_scale + (id[b] >= 0 ? row_of(b) - t_row : 0);
            sc[b] = SHARED ? __hip_atomic_load(at, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : *at;
        }
    }

    // SHARED: the records, and where the first of them belongs
    __device__ __forceinline__ void records(const uint16_t* t_, const float* t_scale_, int t_row_)
    {
        t = t_, t_scale = t_scale_, t_row = t_row_;
        scales();
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

    // the next batch's adapters and Lb
    template <int B>
    __device__ __forceinline__ void load_lb(const Problem& p, Batch<B>& w)
    {
        const int lane = threadIdx.x & 63, frow = lane & 31, fhi = lane >> 5;
        w.n = 0;
#pragma unroll
        for (int j = 0; j < B; ++j) {
            w.ls[j] = -1, w.ch[j] = 0;
            if (w.n == j && next(p, w.ls[j], w.ch[j])) ++w.n;
            if (w.n <= j) continue;
            const __amdgpu_buffer_rsrc_t rl = lb_rsrc(p, w.ls[j]);
#pragma unroll
            for (int a = 0; a < TN; ++a) w.x[j][a] = lb_piece(p, rl, n0 + 32 * a + frow, kAdapterChunk * w.ch[j] + 8 * fhi);
        }
    }

    __device__ __forceinline__ half8 piece(const uint16_t* at) const
    {
        if constexpr (SHARED) {
            const uint64_t* q = (const uint64_t*)at;
            const uint64_t u = __hip_atomic_load(q, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            const uint64_t v = __hip_atomic_load(q + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            return __builtin_bit_cast(half8, u32x4{(uint32_t)u, (uint32_t)(u >> 32), (uint32_t)v, (uint32_t)(v >> 32)});
        } else {
            return __builtin_bit_cast(half8, *(const u32x4*)at);
        }
    }

    // its records (rows without an adapter read some other row's, or what lies there)
    template <int B>
    __device__ __forceinline__ void load_t(const Problem& p, Batch<B>& w) const
    {
        const int fhi = (threadIdx.x >> 5) & 1;
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (w.n <= j) break;
#pragma unroll
            for (int b = 0; b < TM; ++b) {
                const int r = id[b] >= 0 ? row_of(b) - t_row : 0;
                const uint16_t* rec = t + ((int64_t)r * p.chunks + w.ch[j]) * 32 + 8 * fhi;
                w.hi[j][b] = piece(rec);
                w.lo[j][b] = piece(rec + 16);
            }
        }
    }

    // Lb's infinities and NaN must not meet both halves of t: 0 * infinity, or
    // halves of two signs, would make a NaN of what is an infinity.  A batch with
    // such values has zeros in their place, and in t's, and nonfinite() adds what
    // they make of the sums.  One look per batch costs 1 % of 256x4096x4096 with
    // 64 mixed adapters of rank 64 (84.9 us); a look, and Lb's fragments twice, per
    // item cost 3 %.
    template <int B>
    __device__ __forceinline__ void apply(const Problem& p, Batch<B>& w, f32x16 (&acc)[TN][TM]) const
    {
        half8 seen = (half8)(_Float16)0.0f;
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (j >= w.n) break;
#pragma unroll
            for (int a = 0; a < TN; ++a) seen = look_odd(w.x[j][a], seen);
        }
        const bool odd = __ballot(any_odd(seen)) != 0;
        if (odd) {
#pragma unroll
            for (int j = 0; j < B; ++j) {
#pragma unroll
                for (int a = 0; a < TN; ++a) w.x[j][a] = finite8(w.x[j][a]);
#pragma unroll
                for (int b = 0; b < TM; ++b) w.hi[j][b] = finite8(w.hi[j][b]);
            }
        }
#pragma unroll
        for (int j = 0; j < B; ++j) {
            if (j >= w.n) break;
#pragma unroll
            for (int b = 0; b < TM; ++b) {
                if (__ballot(id[b] == w.ls[j]) == 0) continue;
#pragma unroll
                for (int a = 0; a < TN; ++a) {
                    f32x16 d = {};
                    d = __builtin_amdgcn_mfma_f32_32x32x16_f16(w.x[j][a], w.lo[j][b], d, 0, 0, 0);
                    d = __builtin_amdgcn_mfma_f32_32x32x16_f16(w.x[j][a], w.hi[j][b], d, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        acc[a][b][i] = id[b] == w.ls[j] ? acc[a][b][i] + fabsf(sc[b]) * d[i] : acc[a][b][i];
                }
            }
        }
        if (odd) {
#pragma unroll 1
            for (int j = 0; j < w.n; ++j) {
                int ol = w.ls[0], oc = w.ch[0];
#pragma unroll
                for (int i = 1; i < B; ++i) ol = j == i ? w.ls[i] : ol, oc = j == i ? w.ch[i] : oc;
                nonfinite(p, ol, oc, acc);
            }
        }
    }

    // Adds the sums of adapter ol's chunk oc that are an infinity or a NaN, in the
    // lanes whose row is the adapter's; the hi half of t alone, which has the sign
    // of t, tells which.
    __device__ __forceinline__ void nonfinite(const Problem& p, int ol, int oc, f32x16 (&acc)[TN][TM]) const
    {
        const int lane = threadIdx.x & 63, frow = lane & 31, fhi = lane >> 5;
        const __amdgpu_buffer_rsrc_t rl = lb_rsrc(p, ol);
#pragma unroll
        for (int b = 0; b < TM; ++b) {
            const int r = id[b] >= 0 ? row_of(b) - t_row : 0;
            half8 y = piece(t + ((int64_t)r * p.chunks + oc) * 32 + 8 * fhi);
#pragma unroll
            for (int a = 0; a < TN; ++a) {
                half8 x = lb_piece(p, rl, n0 + 32 * a + frow, kAdapterChunk * oc + 8 * fhi);
                asm volatile("" : "+v"(x), "+v"(y));  // a block at a time, for the registers' sake
                const f32x16 d = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, y, f32x16{}, 0, 0, 0);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[a][b][i] += (id[b] == ol && !(fabsf(d[i]) < __builtin_inff())) ? d[i] : 0.0f;
            }
        }
    }

    // every item that is left, B at a time
    template <int B>
    __device__ __forceinline__ void rest(const Problem& p, f32x16 (&acc)[TN][TM])
    {
        Batch<B> w;
        do {
            load_lb(p, w);
            load_t(p, w);
            apply(p, w, acc);
        } while (w.n == B);
    }
};

}  // namespace gsr
