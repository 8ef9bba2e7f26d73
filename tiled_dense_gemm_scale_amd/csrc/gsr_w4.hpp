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

// The eight values q - z of a word as an MFMA operand: dword i holds rows i and
// i + 4.  A code behind the bits of 1024 in fp16 is 1024 + q, four bits higher
// 1024 + 16 q, and the differences below are whole numbers of at most 9 bits,
// so every value is exact.  lo: -(1024 + z), hi: -(64 + z), twice each.
__device__ __forceinline__ u32x4 w4_values(uint32_t w, half2v lo, half2v hi)
{
    constexpr uint32_t kBase = 0x64006400u;
    const half2v sixteenth = {(_Float16)0.0625f, (_Float16)0.0625f};
    const uint32_t t = w >> 8;
    const half2v a = __builtin_bit_cast(half2v, (w & 0x000f000fu) | kBase) + lo;
    const half2v b = __builtin_elementwise_fma(__builtin_bit_cast(half2v, (w & 0x00f000f0u) | kBase), sixteenth, hi);
    const half2v c = __builtin_bit_cast(half2v, (t & 0x000f000fu) | kBase) + lo;
    const half2v d = __builtin_elementwise_fma(__builtin_bit_cast(half2v, (t & 0x00f000f0u) | kBase), sixteenth, hi);
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
// the weights are never rounded.  FL: steps between such ends (1, 2 or 4).
template <int MT, int FL>
struct W4Stream {
    static constexpr int CPL = 4, CB = 16 * CPL, STEPS = 4, UNIT = STEPS * kStep, ENDS = STEPS / FL;
    typedef StreamSums<CPL, MT> Sums;

    struct Batch {
        u32x4 w[STEPS];
        u32x4 a[STEPS][MT];
        u32x2 s[ENDS];
        uint32_t z[ENDS];
    };

    __device__ static __forceinline__ void load(Batch& t, const W4Matrix& m, int N, uint32_t voff, int c,
                                                const StreamRows<MT>& rows, int tiles, int u, int g)
    {
        const int k0 = u * UNIT;
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
            t.w[i] = *(const u32x4_at4*)(m.codes + (size_t)(k0 / 8 + 4 * i) * N + voff);
#pragma unroll
        for (int e = 0; e < ENDS; ++e) {
            const size_t row = (size_t)((k0 + e * FL * kStep) >> m.glog2) * N;
            t.s[e] = *(const u32x2_at2*)(m.scales + row + (uint32_t)c);
            t.z[e] = m.zeros ? *(const u32_at1*)(m.zeros + row + (uint32_t)c) : 0x08080808u;
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
            for (int x = 0; x < MT; ++x)
                if (x < tiles) t.a[i][x] = rows.full(x, k0 + i * kStep + 8 * g);
    }

    __device__ static __forceinline__ void load_part(Batch& t, const W4Matrix& m, int K, int N, int c,
                                                     const StreamRows<MT>& rows, int tiles, int u, int g)
    {
        const int k0 = u * UNIT, words = (K + 7) / 8;
#pragma unroll
        for (int i = 0; i < STEPS; ++i) {
            const int r = k0 / 8 + 4 * i + g;
#pragma unroll
            for (int j = 0; j < CPL; ++j) t.w[i][j] = (r < words && c + j < N) ? m.codes[(size_t)r * N + c + j] : 0u;
        }
#pragma unroll
        for (int e = 0; e < ENDS; ++e) {
            const int k = k0 + e * FL * kStep;
            const size_t row = (size_t)(k >> m.glog2) * N;
            uint16_t s[CPL];
            t.z[e] = 0u;
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const bool in = k < K && c + j < N;
                s[j] = in ? m.scales[row + c + j] : (uint16_t)0;
                t.z[e] |= (uint32_t)(in && m.zeros ? m.zeros[row + c + j] : (uint8_t)8) << (8 * j);
            }
            t.s[e] = u32x2{join16(s[0], s[1]), join16(s[2], s[3])};
        }
#pragma unroll
        for (int i = 0; i < STEPS; ++i)
#pragma unroll
            for (int x = 0; x < MT; ++x)
                if (x < tiles) t.a[i][x] = rows.part(x, k0 + i * kStep + 8 * g, K);
    }

    // `ends`: how many of the batch's ends there are (fewer in the last batch of K)
    __device__ static __forceinline__ void multiply(const Batch& t, int tiles, int ends, Sums& acc)
    {
#pragma unroll
        for (int e = 0; e < ENDS; ++e) {
            if (e >= ends) break;
            half2v lo[CPL], hi[CPL];
            float s[CPL];
#pragma unroll
            for (int j = 0; j < CPL; ++j) {
                const _Float16 z = (_Float16)(float)((t.z[e] >> (8 * j)) & 0xffu);
                const _Float16 l = (_Float16)-1024.0f - z, h = (_Float16)-64.0f - z;
                lo[j] = half2v{l, l};
                hi[j] = half2v{h, h};
                s[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(t.s[e][j / 2] >> (16 * (j & 1))));
            }
            f32x4 sum[CPL][MT];
#pragma unroll
            for (int i = 0; i < FL; ++i) {
                u32x4 b[CPL];
#pragma unroll
                for (int j = 0; j < CPL; ++j) b[j] = w4_values(t.w[e * FL + i][j], lo[j], hi[j]);
#pragma unroll
                for (int x = 0; x < MT; ++x)
                    if (x < tiles) {
                        const u32x4 a = w4_order(t.a[e * FL + i][x]);
#pragma unroll
                        for (int j = 0; j < CPL; ++j)
                            sum[j][x] = mfma16(a, b[j], i == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : sum[j][x]);
                    }
            }
#pragma unroll
            for (int x = 0; x < MT; ++x)
                if (x < tiles) {
#pragma unroll
                    for (int j = 0; j < CPL; ++j)
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc.v[j][x][r] = fmaf(s[j], sum[j][x][r], acc.v[j][x][r]);
                }
        }
    }

    // acc += A[:, k] w[k, :] over the units u0 <= u < u1 of 128 k
    __device__ static __forceinline__ void run(const W4Matrix& m, int K, int N, int n0, const StreamRows<MT>& rows,
                                               int tiles, int u0, int u1, Sums& acc)
    {
        const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
        const int c = stream_column<CPL>(n0, l, N);
        const uint32_t voff = (uint32_t)g * (uint32_t)N + (uint32_t)c;
        const int full = N >= CPL ? min(u1, K / UNIT) : u0;
        Batch b0, b1;
        int u = u0;
        if (u < full) {
            load(b0, m, N, voff, c, rows, tiles, u, g);
            for (; u + 2 < full; u += 2) {
                load(b1, m, N, voff, c, rows, tiles, u + 1, g);
                multiply(b0, tiles, ENDS, acc);
                load(b0, m, N, voff, c, rows, tiles, u + 2, g);
                multiply(b1, tiles, ENDS, acc);
            }
            if (u + 1 < full) {
                load(b1, m, N, voff, c, rows, tiles, u + 1, g);
                multiply(b0, tiles, ENDS, acc);
                multiply(b1, tiles, ENDS, acc);
                u += 2;
            } else {
                multiply(b0, tiles, ENDS, acc);
                u += 1;
            }
        }
        for (u = max(u, u0); u < u1; ++u) {
            load_part(b0, m, K, N, c, rows, tiles, u, g);
            multiply(b0, tiles, min(ENDS, (K - u * UNIT + FL * kStep - 1) / (FL * kStep)), acc);
        }
    }
};

}  // namespace gsr
