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

// The rows of A that a lane reads: row l of each of MT tiles of 16 (null: none,
// zeros).
template <int MT>
struct StreamRows {
    const uint16_t* p[MT];
    __device__ __forceinline__ u32x4 full(int mt, int k) const
    {
        u32x4 v = {0u, 0u, 0u, 0u};
        if (p[mt] != nullptr) v = *(const u32x4_at2*)(p[mt] + k);
        return v;
    }
    __device__ __forceinline__ u32x4 part(int mt, int k, int K) const
    {
        return p[mt] != nullptr ? load8_first(p[mt] + k, K - k) : u32x4{0u, 0u, 0u, 0u};
    }
};

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

// ---- fp16 weights ------------------------------------------------------------
struct HalfMatrix {
    const uint16_t* b;  // K x N
};

template <int MT>
struct HalfStream {
    static constexpr int CPL = 8, CB = 16 * CPL, UNIT = kStep;  // UNIT: k of the smallest run
    typedef StreamSums<CPL, MT> Sums;

    struct Step {
        u32x4 b[8];
        u32x4 a[MT];
    };

    __device__ static __forceinline__ void load(Step& s, const uint16_t* B, int N, uint32_t voff, const StreamRows<MT>& rows,
                                                int tiles, int k0, int g)
    {
        const uint16_t* base = B + (size_t)k0 * N;
#pragma unroll
        for (int i = 0; i < 8; ++i) s.b[i] = *(const u32x4_at2*)(base + (size_t)i * N + voff);
#pragma unroll
        for (int t = 0; t < MT; ++t)
            if (t < tiles) s.a[t] = rows.full(t, k0 + 8 * g);
    }

    __device__ static __forceinline__ void load_part(Step& s, const uint16_t* B, int N, int K, int c,
                                                     const StreamRows<MT>& rows, int tiles, int k0, int g)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int k = k0 + 8 * g + i;
            s.b[i] = load8_first(B + (size_t)min(k, K - 1) * N + c, k < K ? N - c : 0);
        }
#pragma unroll
        for (int t = 0; t < MT; ++t)
            if (t < tiles) s.a[t] = rows.part(t, k0 + 8 * g, K);
    }

    __device__ static __forceinline__ void multiply(const Step& s, int tiles, Sums& acc)
    {
        u32x4 o[8];
        transpose8x8(s.b, o);
#pragma unroll
        for (int t = 0; t < MT; ++t)
            if (t < tiles) {
#pragma unroll
                for (int j = 0; j < 8; ++j) acc.v[j][t] = mfma16(s.a[t], o[j], acc.v[j][t]);
            }
    }

    // acc += A[:, k] B[k, :] over the units u0 <= u < u1 of 32 k
    __device__ static __forceinline__ void run(const HalfMatrix& m, int K, int N, int n0, const StreamRows<MT>& rows,
                                               int tiles, int u0, int u1, Sums& acc)
    {
        const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
        const int c = stream_column<CPL>(n0, l, N);
        const uint32_t voff = (uint32_t)(8 * g) * (uint32_t)N + (uint32_t)c;
        const int full = N >= CPL ? min(u1, K / kStep) : u0;
        Step s0, s1;
        int u = u0;
        if (u < full) {
            load(s0, m.b, N, voff, rows, tiles, u * kStep, g);
            for (; u + 2 < full; u += 2) {
                load(s1, m.b, N, voff, rows, tiles, (u + 1) * kStep, g);
                multiply(s0, tiles, acc);
                load(s0, m.b, N, voff, rows, tiles, (u + 2) * kStep, g);
                multiply(s1, tiles, acc);
            }
            if (u + 1 < full) {
                load(s1, m.b, N, voff, rows, tiles, (u + 1) * kStep, g);
                multiply(s0, tiles, acc);
                multiply(s1, tiles, acc);
                u += 2;
            } else {
                multiply(s0, tiles, acc);
                u += 1;
            }
        }
        for (u = max(u, u0); u < u1; ++u) {
            load_part(s0, m.b, N, K, c, rows, tiles, u * kStep, g);
            multiply(s0, tiles, acc);
        }
    }
};

// ---- the sum over waves ---------------------------------------------------------
// Tile t (16 rows x CB columns) of every wave's sums goes to LDS; f(row, q, sum,
// sum of the second set) is called for every four consecutive positions 4q of
// a row, in wave order from +0.  With SETS = 2 the first half of the waves
// is one sum and the second half another.
constexpr int kStreamWaves = 8, kStreamThreads = kWave * kStreamWaves;

template <int CPL, int MT, int SETS, class F>
__device__ __forceinline__ void stream_reduce(float* lds, const StreamSums<CPL, MT>& acc, int tiles, F&& f)
{
    constexpr int CB = 16 * CPL, QUADS = CB / 4, W = kStreamWaves / SETS;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l = lane & 15, g = lane >> 4;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        if (t >= tiles) break;
        __syncthreads();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            f32x4* to = (f32x4*)(lds + (size_t)(wave * 16 + 4 * g + r) * CB + CPL * l);
#pragma unroll
            for (int j = 0; j < CPL / 4; ++j)
                to[j] = f32x4{acc.v[4 * j][t][r], acc.v[4 * j + 1][t][r], acc.v[4 * j + 2][t][r], acc.v[4 * j + 3][t][r]};
        }
        __syncthreads();
        for (int u = tid; u < 16 * QUADS; u += kStreamThreads) {
            const int m = u / QUADS, q = u % QUADS;
            f32x4 s[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
            for (int w = 0; w < kStreamWaves; ++w) {
                const f32x4 v = *(const f32x4*)(lds + (size_t)(w * 16 + m) * CB + 4 * q);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[w / W][i] += v[i];
            }
            f(16 * t + m, q, s[0], s[1]);
        }
    }
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
