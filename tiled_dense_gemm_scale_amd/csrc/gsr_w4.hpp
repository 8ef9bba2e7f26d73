// gsr_w4.hpp -- weights held in 4 bits: w[k, n] = (q[k, n] - z) s with codes
// q in 0..15, eight of consecutive k in a word (bits 4i .. 4i + 3 are row
// 8r + i; ceil(K / 8) x N words), and a scale (fp16) and zero point (8 bits; 8
// everywhere without any) per column and group of `group` rows, a power of two
// from 32 on; and a wave's share of a product with them.
#pragma once

#include "gsr_stream.hpp"

namespace gsr {

struct W4Matrix {
    const uint32_t* codes;   // ceil(K / 8) x N
    const uint16_t* scales;  // ceil(K / group) x N
    const uint8_t* zeros;    // like scales, or null
    int glog2;               // group = 1 << glog2
};

typedef _Float16 half2v __attribute__((ext_vector_type(2)));

// (w & mask) | base in one instruction: the mask in a scalar register, the base
// in a vector one, as the encoding has room for one constant of neither.
__device__ __forceinline__ half2v and_or(uint32_t w, uint32_t mask, uint32_t base)
{
    uint32_t d;
    asm("v_and_or_b32 %0, %1, %2, %3" : "=v"(d) : "v"(w), "s"(mask), "v"(base));
    return __builtin_bit_cast(half2v, d);
}

// The eight values q - z of a word as an MFMA operand: dword i holds rows i and
// i + 4.  The conversion by a fixed exponent is a published one (Kim, Henry, Fahim and
// Awadalla, "Who Says Elephants Can't Run", 2022); this form is for zero points of 8
// bits.  A code behind the bits of 1024 in fp16 is 1024 + q, four bits higher
// 1024 + 16 q, and the differences below are whole numbers of at most 9 bits,
// so every value is exact.  lo: -(1024 + z), hi: -(64 + z), twice each.  Nine
// instructions for eight weights; the loop is bound by them where the weights'
// bytes come fast enough.
__device__ __forceinline__ u32x4 w4_values(uint32_t w, half2v lo, half2v hi)
{
    constexpr uint32_t kBase = 0x64006400u;
    const half2v sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t t = w >> 8;
    const half2v a = and_or(w, 0x000f000fu, kBase) + lo;
    const half2v b = __builtin_elementwise_fma(and_or(w, 0x00f000f0u, kBase), sixteenth, hi);
    const half2v c = and_or(t, 0x000f000fu, kBase) + lo;
    const half2v d = __builtin_elementwise_fma(and_or(t, 0x00f000f0u, kBase), sixteenth, hi);
    return u32x4{__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), __builtin_bit_cast(uint32_t, c),
                 __builtin_bit_cast(uint32_t, d)};
}

// The same order of eight values of A.
__device__ __forceinline__ u32x4 w4_order(u32x4 a)
{
    return u32x4{pack_lo(a[0], a[2]), pack_hi(a[0], a[2]), pack_lo(a[1], a[3]), pack_hi(a[1], a[3])};
}

// A wave's share: 64 columns, four per lane, one word of each per step.  Runs
// are cut at multiples of 128 rows; a group's sum of products is kept apart and
// scaled in fp32 when the group (or, of larger ones, 128 rows of it) ends, so
// the weights are never rounded.  FL: steps between such ends (1, 2 or 4).  DW:
// every row of A starts on a dword.  SPLIT: A in halves, which lie in the codes'
// order.
template <int FL, bool DW, bool SPLIT>
struct W4Stream {
    static __device__ __forceinline__ int order(int k) { return (k & ~7) | (k & 3) << 1 | (k >> 2 & 1); }
    static __device__ __forceinline__ u32x4 ordered(u32x4 a) { return SPLIT ? a : w4_order(a); }
    static constexpr int CPL = 4, CB = 16 * CPL, STEPS = 4, UNIT = STEPS * kStep, ENDS = STEPS / FL;
    typedef StreamSums<CPL> Sums;
    typedef StreamRows<DW> Rows;

    struct Batch {
        u32x4 w[STEPS];
        u32x4 a[SPLIT ? 2 : 1][STEPS];
        u32x2 s[ENDS];
        uint32_t z[ENDS];
    };
    struct Place {
        W4Matrix m;
        const uint8_t* zeros;  // m.zeros, or any readable bytes of that many
        float* slice;
        int K, N, c, g;
        uint32_t off[STEPS];   // bytes from a unit's first row of words
    };

    // Unit u of a run of units before `end` (from there on nothing is read anew).
    __device__ static __forceinline__ void load(Batch& t, const Place& p, const Rows& rows, int u, int end)
    {
        const int k0 = min(u, end - 1) * UNIT;
        const __amdgpu_buffer_rsrc_t rs = rows_rsrc(p.m.codes, u < end ? (p.K + 7) / 8 : 0, k0 / 8, 4u * (uint32_t)p.N);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) t.w[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, p.off[i], 0, 0);
#pragma unroll
        for (int e = 0; e < ENDS; ++e) {
            const size_t row = (size_t)(min(k0 + e * FL * kStep, p.K - 1) >> p.m.glog2) * p.N;
            t.s[e] = *(const u32x2_at2*)(p.m.scales + row + p.c);
            t.z[e] = *(const u32_at1*)(p.zeros + row + p.c);
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            t.a[0][i] = rows.load(k0 + i * kStep + 8 * rows.run);
            if constexpr (SPLIT) t.a[1][i] = rows.load(rows.wide + k0 + i * kStep + 8 * rows.run);
        }
        __builtin_amdgcn_sched_barrier(0);
    }

    // The scale and the zero point's two forms of a lane's columns.
    struct Scale {
        half2v lo[CPL], hi[CPL];
        float s[CPL];
    };
    __device__ static __forceinline__ void scale_of(Scale& v, u32x2 s, uint32_t zeros, bool have)
    {
        const uint32_t all = have ? zeros : 0x08080808u;
        const half2v shift = {(_Float16)960.0f, (_Float16)960.0f};
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            // the bits of -(1024 + z) are 0xe400 + z
            const uint32_t pick = 0x04000400u | (uint32_t)j * 0x00010001u;
            v.lo[j] = __builtin_bit_cast(half2v, __builtin_amdgcn_perm(0xe4e4e4e4u, all, pick));
            v.hi[j] = v.lo[j] + shift;
            v.s[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(s[j / 2] >> (16 * (j & 1))));
        }
    }

    __device__ static __forceinline__ void multiply(Batch& t, const Place& p, const Rows& rows, int u, Sums& acc)
    {
        const int left = p.K - u * UNIT;
        if (rows.turn)
#pragma unroll
            for (int h = 0; h < (SPLIT ? 2 : 1); ++h) stream_turn(t.a[h], p.slice);
        if (left < UNIT) {  // behind a row of A lies the next one
#pragma unroll
            for (int i = 0; i < STEPS; ++i)
#pragma unroll
                for (int h = 0; h < (SPLIT ? 2 : 1); ++h)
                    t.a[h][i] = first8(t.a[h][i], (SPLIT ? rows.wide - u * UNIT : left) - i * kStep - 8 * p.g);
        }
#pragma unroll
        for (int e = 0; e < ENDS; ++e) {
            if (e * FL * kStep >= left) break;  // no such group
            Scale v;
            scale_of(v, t.s[e], t.z[e], p.m.zeros != nullptr);
            f32x4 sum[CPL], low[CPL];  // low: of the second halves
#pragma unroll
            for (int i = 0; i < FL; ++i) {
                const u32x4 a = ordered(t.a[0][e * FL + i]);
#pragma unroll
                for (int j = 0; j < CPL; ++j) {
                    const u32x4 b = w4_values(t.w[e * FL + i][j], v.lo[j], v.hi[j]);
                    const f32x4 none = {0.f, 0.f, 0.f, 0.f};
                    sum[j] = mfma16(a, b, i == 0 ? none : sum[j]);
                    if constexpr (SPLIT) low[j] = mfma16(t.a[1][e * FL + i], b, i == 0 ? none : low[j]);
                }
                __builtin_amdgcn_sched_barrier(0);  // a step's values live no longer than it
            }
#pragma unroll
            for (int j = 0; j < CPL; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc.v[j][r] = fmaf(v.s[j], SPLIT ? fmaf(low[j][r], 1.0f / kRest, sum[j][r]) : sum[j][r], acc.v[j][r]);
        }
    }

    // One step of 32 rows of a matrix of any width: value by value and scaled by
    // itself.
    __device__ static __forceinline__ void step(const Place& p, const Rows& rows, int k0, Sums& acc)
    {
        const int r = k0 / 8 + p.g, words = (p.K + 7) / 8;
        const size_t row = (size_t)(k0 >> p.m.glog2) * p.N;
        Scale v;
        u32x4 w;
        uint16_t s[CPL];
        uint32_t zeros = 0u;
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const bool in = p.c + j < p.N;
            w[j] = r < words && in ? p.m.codes[(size_t)r * p.N + p.c + j] : 0u;
            s[j] = in ? p.m.scales[row + p.c + j] : (uint16_t)0;
            zeros |= (uint32_t)(in ? p.zeros[row + p.c + j] : (uint8_t)0) << (8 * j);
        }
        scale_of(v, u32x2{join16(s[0], s[1]), join16(s[2], s[3])}, zeros, p.m.zeros != nullptr);
        const int n = (SPLIT ? rows.wide : p.K) - k0 - 8 * p.g;
        u32x4 held[SPLIT ? 2 : 1];
        held[0] = rows.load(k0 + 8 * rows.run);
        if constexpr (SPLIT) held[1] = rows.load(rows.wide + k0 + 8 * rows.run);
        if (rows.turn) stream_turn(held, p.slice);
        const u32x4 a = ordered(first8(held[0], n));
        u32x4 a2 = {0u, 0u, 0u, 0u};
        if constexpr (SPLIT) a2 = first8(held[1], n);
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
            const u32x4 b = w4_values(w[j], v.lo[j], v.hi[j]);
            const f32x4 none = {0.f, 0.f, 0.f, 0.f};
            f32x4 sum = mfma16(a, b, none);
            if constexpr (SPLIT) {
                const f32x4 low = mfma16(a2, b, none);
#pragma unroll
                for (int x = 0; x < 4; ++x) sum[x] = fmaf(low[x], 1.0f / kRest, sum[x]);
            }
#pragma unroll
            for (int x = 0; x < 4; ++x) acc.v[j][x] = fmaf(v.s[j], sum[x], acc.v[j][x]);
        }
    }

    __device__ static __forceinline__ Place place(const W4Matrix& m, int K, int N, int n0, float* slice)
    {
        const int lane = threadIdx.x & 63;
        Place p;
        p.m = m;
        p.zeros = m.zeros ? m.zeros : (const uint8_t*)m.scales;  // without zeros its loads are not looked at
        p.slice = slice;
        p.K = K;
        p.N = N;
        p.g = lane >> 4;
        p.c = stream_column<CPL>(n0, lane & 15, N);
#pragma unroll
        for (int i = 0; i < STEPS; ++i) p.off[i] = 4u * ((uint32_t)(4 * i + p.g) * (uint32_t)N + (uint32_t)p.c);
        return p;
    }

    // acc += A[:, k] w[k, :] over the units u0 <= u < u1 of 128 k; slice: this
    // wave's LDS, 16 x CB floats
    __device__ static __forceinline__ void run(const W4Matrix& m, int K, int N, int n0, const Rows& rows,
                                               int u0, int u1, float* slice, Sums& acc)
    {
        const Place p = place(m, K, N, n0, slice);
        if (u0 >= u1) return;
        if (N >= CPL) {
            stream_ring<Batch>(
                u1 - u0, [&](Batch& t, int i) { load(t, p, rows, u0 + i, u1); },
                [&](Batch& t, int i) { multiply(t, p, rows, u0 + i, acc); });
            return;
        }
#pragma unroll 1
        for (int k0 = u0 * UNIT; k0 < min(K, u1 * UNIT); k0 += kStep) step(p, rows, k0, acc);
    }
};

}  // namespace gsr
