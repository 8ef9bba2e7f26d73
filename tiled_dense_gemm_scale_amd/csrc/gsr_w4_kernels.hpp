// gsr_w4_kernels.hpp -- kernels on weights held in 4 bits (gsr_w4.hpp): the
// product of a few rows, quantizing, and the values back.
#pragma once

#include "gsr_w4.hpp"

namespace gsr {

// ---- the product -----------------------------------------------------------------
struct W4Gemm {
    const uint16_t* a;  // M x K
    W4Matrix w;
    const uint16_t* bias;
    uint16_t* c;        // M x N
    int M, N, K, act;
    float alpha;
    int blocks_n, parts, chunk;  // column blocks; parts of K, of `chunk` units each
    int per;                     // column blocks per counter
    float* part;                 // parts x M x (blocks_n CB)
    uint32_t* count;
};

// Workgroup (block of 16 MT rows, column block, part of K), parts fastest.
// With more than one part the sums meet in the workspace and the last workgroup
// of a counter's blocks adds them in part order.
template <int MT, int FL>
__global__ void __launch_bounds__(kStreamThreads, 2) w4_gemm_kernel(W4Gemm p)
{
    using S = W4Stream<MT, FL>;
    constexpr int CPL = S::CPL, CB = S::CB, QUADS = CB / 4;
    __shared__ __attribute__((aligned(16))) float lds[kStreamWaves * 16 * CB];
    __shared__ int flag;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 15;
    const int part = blockIdx.x % p.parts, tile = blockIdx.x / p.parts, nb = tile % p.blocks_n;
    const int m0 = tile / p.blocks_n * 16 * MT, n0 = nb * CB, rows_here = min(16 * MT, p.M - m0);

    StreamRows<MT> rows;
#pragma unroll
    for (int t = 0; t < MT; ++t) rows.p[t] = p.a + (size_t)(m0 + min(16 * t + l, rows_here - 1)) * p.K;
    const int units = (p.K + S::UNIT - 1) / S::UNIT;
    const int first = part * p.chunk, here = max(0, min(p.chunk, units - first));
    const int u0 = first + here * wave / kStreamWaves, u1 = first + here * (wave + 1) / kStreamWaves;
    typename S::Sums acc;
    acc.clear();
    S::run(p.w, p.K, p.N, n0, rows, u0, u1, acc);

    auto finish = [&](int m, int q, int at, f32x4 s) {
        const int col = stream_position<CPL>(at, q, p.N);
        if (col < 0 || m >= p.M) return;
        uint16_t* to = p.c + (size_t)m * p.N + col;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < p.N) to[i] = to_half(activate(s[i] * p.alpha + (p.bias ? half_at(p.bias + col + i) : 0.0f), p.act));
    };
    const size_t wide = (size_t)p.blocks_n * CB;
#pragma unroll
    for (int t = 0; t < MT; ++t) {
        __syncthreads();
        stream_put<CPL, MT>(lds + wave * 16 * CB, acc, t);
        __syncthreads();
        const int m = 16 * t + threadIdx.x / QUADS, q = threadIdx.x % QUADS;
        if (threadIdx.x >= 16 * QUADS || m >= rows_here) continue;
        const f32x4 s = stream_sum<CPL>(lds, kStreamWaves, m - 16 * t, q);
        if (p.parts == 1) finish(m0 + m, q, n0, s);
        else meet_store(p.part + ((size_t)part * p.M + m0 + m) * wide + n0 + 4 * q, s);
    }
    if (p.parts == 1) return;
    const int b0 = nb / p.per * p.per, b1 = min(b0 + p.per, p.blocks_n);
    if (!meet_last(p.count + nb / p.per, (uint32_t)((b1 - b0) * p.parts), &flag)) return;
    for (int b = b0; b < b1; ++b)
        for (int u = threadIdx.x; u < rows_here * QUADS; u += kStreamThreads) {
            const int m = u / QUADS, q = u % QUADS;
            f32x4 s = {0.f, 0.f, 0.f, 0.f};
            for (int g = 0; g < p.parts; ++g) {
                const f32x4 v = meet_load(p.part + ((size_t)g * p.M + m0 + m) * wide + b * CB + 4 * q);
#pragma unroll
                for (int i = 0; i < 4; ++i) s[i] += v[i];
            }
            finish(m0 + m, q, b * CB, s);
        }
}

// ---- quantizing --------------------------------------------------------------------
// One thread per column and group; the group is read twice, the second time
// from the caches.
struct W4Convert {
    const uint16_t* b;    // matrices x K x N
    uint16_t* values;     // the same, written by dequantize
    uint32_t* codes;
    uint16_t* scales;
    uint8_t* zeros;
    int K, N, glog2, groups;
    int64_t matrices;
};

__global__ void __launch_bounds__(256) w4_quantize_kernel(W4Convert p)
{
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= p.N) return;
    const int words = (p.K + 7) / 8;
    const int64_t all = p.matrices * p.groups;
    for (int64_t eg = blockIdx.y; eg < all; eg += gridDim.y) {
        const int64_t e = eg / p.groups;
        const int64_t begin = (eg % p.groups) << p.glog2;
        const int k0 = (int)begin, k1 = (int)min((int64_t)p.K, begin + ((int64_t)1 << p.glog2));
        const uint16_t* b = p.b + (size_t)e * p.K * p.N + n;
        float lo = 0.0f, hi = 0.0f;
        bool odd = false;  // an infinity or a NaN
        for (int k = k0; k < k1; ++k) {
            const float v = half_at(b + (size_t)k * p.N);
            odd |= !(fabsf(v) <= 65504.0f);
            lo = fminf(lo, v);
            hi = fmaxf(hi, v);
        }
        const float step = p.zeros ? (hi - lo) / 15.0f : fmaxf(-lo, hi) / 7.0f;
        const uint16_t sb = odd ? (uint16_t)0x7e00 : to_half(step);
        const float s = (float)__builtin_bit_cast(_Float16, sb);
        const bool live = s > 0.0f;
        const float z = p.zeros && live ? fminf(fmaxf(rintf(-lo / s), 0.0f), 15.0f) : 8.0f;
        const size_t at = (size_t)eg * p.N + n;
        p.scales[at] = sb;
        if (p.zeros) p.zeros[at] = (uint8_t)z;
        for (int k = k0; k < k1; k += 8) {
            uint32_t w = 0;
            for (int i = 0; i < 8; ++i) {
                const float v = k + i < k1 ? half_at(b + (size_t)(k + i) * p.N) : 0.0f;
                const float q = live ? fminf(fmaxf(rintf(v / s) + z, 0.0f), 15.0f) : z;
                w |= (uint32_t)q << (4 * i);
            }
            p.codes[((size_t)e * words + k / 8) * p.N + n] = w;
        }
    }
}

// One thread per word.
__global__ void __launch_bounds__(256) w4_dequantize_kernel(W4Convert p)
{
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= p.N) return;
    const int words = (p.K + 7) / 8;
    const int64_t all = p.matrices * words;
    for (int64_t er = blockIdx.y; er < all; er += gridDim.y) {
        const int64_t e = er / words;
        const int r = (int)(er % words);
        const uint32_t w = p.codes[(size_t)er * p.N + n];
        const size_t at = ((size_t)e * p.groups + ((8 * r) >> p.glog2)) * p.N + n;
        const float s = half_at(p.scales + at), z = p.zeros ? (float)p.zeros[at] : 8.0f;
        for (int i = 0; i < 8 && 8 * r + i < p.K; ++i)
            p.values[((size_t)e * p.K + 8 * r + i) * p.N + n] = to_half(((float)((w >> (4 * i)) & 15u) - z) * s);
    }
}

}  // namespace gsr
