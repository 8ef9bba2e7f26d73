// gsr_stream.hpp -- products of a few rows with weights read once: a wave's
// share of C (16 MT rows x CB columns) over a run of K, operands from memory
// straight into registers.
//
// Such products are bound by the weights' bytes, so nothing stands between the
// loads and the matrix cores: no LDS, no barrier.  A wave's 64 lanes hold an
// MFMA 16x16x32 operand as 16 columns x 4 runs of 8 values of k.  With weights
// in rows of N (k-major) lane (l, g) = (lane % 16, lane / 16) reads the CPL
// columns c .. c + CPL - 1 of the rows 8g .. 8g + 7 of a step of 32 rows, which
// is one operand for each of its columns once the 8 x CPL block is transposed
// in registers (byte permutes, half an instruction per value); the 16 lanes of
// a group so read 16 CPL consecutive columns of a row.  4-bit codes hold 8
// values of k in a word and need no transpose (gsr_w4.hpp).
//
// Waves of a workgroup take runs of K of their own and add their sums through
// LDS in wave order.
//
// Columns past N: a lane whose columns would pass N is moved back to end at N,
// so its sums are those of columns that its neighbour has too, the same bits,
// and no load needs a mask; matrices of fewer than CPL columns are read value
// by value.  Rows past K read as zeros on both sides, so whatever lies behind
// the matrix adds nothing.  Rows of C are independent of one another in the
// matrix cores (infinities and NaN stay in their row and column).
#pragma once

#include "gsr_kernels.hpp"

namespace gsr {

// Vectors at addresses of any even (words: any 4-byte, bytes: any) alignment;
// the hardware takes global loads at every address.
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
typedef uint32_t u32_at1 __attribute__((aligned(1)));

__device__ __forceinline__ uint32_t join16(uint16_t lo, uint16_t hi) { return (uint32_t)lo | ((uint32_t)hi << 16); }

// eight fp16 values at p of which `n` exist (zeros for the others)
__device__ __forceinline__ u32x4 load8_first(const uint16_t* p, int n)
{
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t lo = 2 * i < n ? p[2 * i] : (uint16_t)0, hi = 2 * i + 1 < n ? p[2 * i + 1] : (uint16_t)0;
        v[i] = join16(lo, hi);
    }
    return v;
}

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

constexpr int kStep = 32;  // k per MFMA

// The rows of A that a lane reads: row l of each of MT tiles of 16.  Rows past
// the last are that one again, whose sums nobody takes: no load is masked, and
// lanes with one address are one access.
template <int MT>
struct StreamRows {
    const uint16_t* p[MT];
    __device__ __forceinline__ u32x4 full(int t, int k) const { return *(const u32x4_at2*)(p[t] + k); }
    __device__ __forceinline__ u32x4 part(int t, int k, int K) const { return load8_first(p[t] + k, K - k); }
};

// A descriptor of the rows k0 and on of a matrix of `rows` rows of `pitch` bytes
// (whole dwords): loads behind the last row are zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* base, int rows, int k0, uint32_t pitch)
{
    const uint64_t left = (uint64_t)max(rows - k0, 0) * pitch;  // none: nothing is read
    return make_rsrc((const uint8_t*)base + (size_t)k0 * pitch, (uint32_t)min(left, (uint64_t)0x7fffffffu));
}

// The column where lane l's CPL columns of the block from n0 start.
template <int CPL>
__device__ __forceinline__ int stream_column(int n0, int l, int N)
{
    const int c = n0 + CPL * l;
    return N >= CPL ? min(c, N - CPL) : c;
}

// acc[j][t]: columns c + j of lane l (its 16 lanes' columns), rows 16 t + 4 g + r.
template <int CT, int MT>
struct StreamSums {
    f32x4 v[CT][MT];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < CT; ++j)
#pragma unroll
            for (int t = 0; t < MT; ++t) v[j][t] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
};

// multiply(b[i]) for n > 0 units in turn, DEPTH - 1 units' loads in flight: load(b,
// i) is called for units past the last too, and has to be one that reads nothing
// new there, so that no wait depends on which way a branch went.
template <int DEPTH, class Batch, class Load, class Multiply>
__device__ __forceinline__ void stream_ring(int n, Load&& load, Multiply&& multiply)
{
    Batch b[DEPTH];
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i) load(b[i], i);
    for (int i = 0;; i += DEPTH) {
#pragma unroll
        for (int j = 0; j < DEPTH; ++j) {
            load(b[(j + DEPTH - 1) % DEPTH], i + j + DEPTH - 1);
            multiply(b[j]);
            if (i + j + 1 >= n) return;
        }
    }
}

// ---- fp16 weights ------------------------------------------------------------
struct HalfMatrix {
    const uint16_t* b;  // K x N
};

// DW: every row starts on a dword (N even, b on one).
template <int MT, bool DW>
struct HalfStream {
    static constexpr int CPL = 8, CB = 16 * CPL, UNIT = kStep, DEPTH = 2;  // UNIT: k of the smallest run
    typedef StreamSums<CPL, MT> Sums;

    struct Step {
        u32x4 b[8];
        u32x4 a[MT];
    };
    struct Place {
        const uint16_t* b;
        int K, N, c, g;
        uint32_t off[DW ? 8 : 1];  // bytes from a step's first row
    };

    // Unit u of a run of units before `end` (from there on nothing is read anew).
    template <bool TAIL>
    __device__ static __forceinline__ void load(Step& s, const Place& p, const StreamRows<MT>& rows, int u, int end)
    {
        const int k0 = min(u, end - 1) * kStep;
        if (TAIL && p.N < CPL) {
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {  // one row in flight, for the registers' sake
                const int k = k0 + 8 * p.g + i;
                const u32x4 v = load8_first(p.b + (size_t)min(k, p.K - 1) * p.N + p.c, k < p.K ? p.N - p.c : 0);
#pragma unroll
                for (int x = 0; x < 8; ++x) s.b[x] = x == i ? v : s.b[x];
            }
        } else if constexpr (DW) {
            const __amdgpu_buffer_rsrc_t rs = rows_rsrc(p.b, u < end ? p.K : 0, k0, 2u * (uint32_t)p.N);
#pragma unroll
            for (int i = 0; i < 8; ++i) s.b[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, p.off[i], 0, 0);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int k = k0 + 8 * p.g + i;
                s.b[i] = *(const u32x4_at2*)(p.b + (size_t)(TAIL ? min(k, p.K - 1) : k) * p.N + p.c);
                if (TAIL && k >= p.K) s.b[i] = u32x4{0u, 0u, 0u, 0u};
            }
        }
#pragma unroll
        for (int t = 0; t < MT; ++t) s.a[t] = TAIL ? rows.part(t, k0 + 8 * p.g, p.K) : rows.full(t, k0 + 8 * p.g);
        __builtin_amdgcn_sched_barrier(0);
    }

    __device__ static __forceinline__ void multiply(const Step& s, Sums& acc)
    {
#pragma unroll
        for (int d = 0; d < 4; ++d) {  // columns 2d and 2d + 1
            u32x4 even, odd;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                even[e] = pack_lo(s.b[2 * e][d], s.b[2 * e + 1][d]);
                odd[e] = pack_hi(s.b[2 * e][d], s.b[2 * e + 1][d]);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                acc.v[2 * d][t] = mfma16(s.a[t], even, acc.v[2 * d][t]);
                acc.v[2 * d + 1][t] = mfma16(s.a[t], odd, acc.v[2 * d + 1][t]);
            }
            __builtin_amdgcn_sched_barrier(0);  // a pair's values live no longer than it
        }
    }

    // acc += A[:, k] B[k, :] over the units u0 <= u < u1 of 32 k
    __device__ static __forceinline__ void run(const HalfMatrix& m, int K, int N, int n0, const StreamRows<MT>& rows,
                                               int u0, int u1, Sums& acc)
    {
        const int lane = threadIdx.x & 63;
        Place p;
        p.b = m.b;
        p.K = K;
        p.N = N;
        p.g = lane >> 4;
        p.c = stream_column<CPL>(n0, lane & 15, N);
        if constexpr (DW)
#pragma unroll
            for (int i = 0; i < 8; ++i) p.off[i] = 2u * ((uint32_t)(8 * p.g + i) * (uint32_t)N + (uint32_t)p.c);
        const int full = N >= CPL ? max(u0, min(u1, K / kStep)) : u0;
        if (u0 < full)
            stream_ring<DEPTH, Step>(
                full - u0, [&](Step& s, int i) { load<false>(s, p, rows, u0 + i, full); }, [&](const Step& s) { multiply(s, acc); });
        for (int u = full; u < u1; ++u) {
            Step s{};
            load<true>(s, p, rows, u, u1);
            multiply(s, acc);
        }
    }
};

// ---- the sum over waves ---------------------------------------------------------
// Each of a workgroup's waves has a slice of LDS for one tile (16 rows x CB
// columns) of its sums, row-major.
constexpr int kStreamWaves = 8, kStreamThreads = kWave * kStreamWaves;

template <int CPL, int MT>
__device__ __forceinline__ void stream_put(float* slice, const StreamSums<CPL, MT>& acc, int t)
{
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        f32x4* to = (f32x4*)(slice + (4 * g + r) * 16 * CPL + CPL * l);
#pragma unroll
        for (int j = 0; j < CPL / 4; ++j)
            to[j] = f32x4{acc.v[4 * j][t][r], acc.v[4 * j + 1][t][r], acc.v[4 * j + 2][t][r], acc.v[4 * j + 3][t][r]};
    }
}

// Positions 4q .. 4q + 3 of row m, summed over `waves` slices in order from +0.
template <int CPL>
__device__ __forceinline__ f32x4 stream_sum(const float* slices, int waves, int m, int q)
{
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    for (int w = 0; w < waves; ++w) {
        const f32x4 v = *(const f32x4*)(slices + (size_t)(w * 16 + m) * 16 * CPL + 4 * q);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += v[i];
    }
    return s;
}

// The column of position 4q of the block from n0 (the first of four), or -1
// where the position's lane lies past N.
template <int CPL>
__device__ __forceinline__ int stream_position(int n0, int q, int N)
{
    const int l = 4 * q / CPL;
    return n0 + CPL * l < N ? stream_column<CPL>(n0, l, N) + 4 * q % CPL : -1;
}

// ---- sums that meet in a workspace ---------------------------------------------------
// Written and read at device scope (the L2 of an XCD is not coherent with the
// others'): relaxed atomics at agent scope write through and do not take a
// stale line.  Whoever counts last has every other's sums: each wave waits for
// its stores before the barrier in front of the count, and reads only after the
// count has returned.
__device__ __forceinline__ void meet_store(float* to, f32x4 v)
{
    const u32x4 w = __builtin_bit_cast(u32x4, v);
    uint64_t* d = (uint64_t*)to;
    __hip_atomic_store(d, w[0] | (uint64_t)w[1] << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(d + 1, w[2] | (uint64_t)w[3] << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ f32x4 meet_load(const float* from)
{
    const uint64_t* s = (const uint64_t*)from;
    const uint64_t a = __hip_atomic_load(s, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint64_t b = __hip_atomic_load(s + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    return __builtin_bit_cast(f32x4, u32x4{(uint32_t)a, (uint32_t)(a >> 32), (uint32_t)b, (uint32_t)(b >> 32)});
}

// Counts this workgroup in; true in the one that completes `all`, whose counter
// it puts back to zero.
__device__ __forceinline__ bool meet_last(uint32_t* count, uint32_t all, int* flag)
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's sums have reached device scope
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *flag = (int)(before == all - 1u);
        if (before == all - 1u) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    return *flag != 0;
}

// Column blocks share the 128 counters that every workspace starts with: block
// b counts in b / per, per blocks to a counter.
constexpr int kMeetCounters = 128;
constexpr int64_t kMeetBytes = 4 * kMeetCounters;

// act(y), SiLU = y / (1 + exp(-y)) too
enum : int { kActSilu = 3 };
__device__ __forceinline__ float stream_activate(float y, int act)
{
    if (act == kActSilu) return y * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * y));
    return activate(y, act);
}

__device__ __forceinline__ float half_at(const uint16_t* p) { return (float)__builtin_bit_cast(_Float16, *p); }
__device__ __forceinline__ uint16_t to_half(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

}  // namespace gsr
