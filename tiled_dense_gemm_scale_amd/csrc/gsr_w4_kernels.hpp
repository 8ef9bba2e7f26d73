// gsr_w4_kernels.hpp -- kernels on weights held in 4 bits (gsr_w4.hpp): the
// product, quantizing, and the values back.
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
    int blocks_m, blocks_n;  // tiles of the launch
    int parts, chunk;        // parts of K, of `chunk` units each
    float* part;             // parts x M x (blocks_n CB)
    uint32_t* count;
};

// The sums of a tile's rows m0 .. m0 + rows_here - 1 and columns from n0 over the
// units first .. first + here - 1 of K, a run of them to each wave, into the waves'
// slices of LDS.
template <class S>
__device__ __forceinline__ void w4_tile(const W4Gemm& p, int64_t m0, int rows_here, int n0, int first, int here, float* lds)
{
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    typename S::Rows rows(p.a + (size_t)m0 * p.K, (uint64_t)rows_here * (uint32_t)p.K * 2u, rows_here);
    rows.row((uint32_t)min(stream_row(), rows_here - 1) * (uint32_t)p.K);
    const int u0 = first + here * wave / kStreamWaves, u1 = first + here * (wave + 1) / kStreamWaves;
    typename S::Sums acc;
    acc.clear();
    S::run(p.w, p.K, p.N, n0, rows, u0, u1, lds + wave * 16 * S::CB, acc);
    stream_put<S::CPL>(lds + wave * 16 * S::CB, acc);
}

// act(alpha s + bias) of four columns of a row of C from `col` on (those from N on
// are none).
__device__ __forceinline__ f32x4 w4_epilogue(const W4Gemm& p, int col, f32x4 s)
{
    const f32x4 b = p.bias ? half4_at(p.bias, col, p.N) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = activate(s[i] * p.alpha + b[i], p.act);
    return s;
}

// A tile of 16 rows and 64 columns, whose workgroup's waves split its K, or a
// part of it: then the tile's sums meet in the workspace and the workgroup that
// comes last adds them.  One block of rows is bound by the codes' bytes and the
// chain of launch, loads and sums; more of them run beside each other and read the
// codes again, from the caches, and unpack them again: from some 100 rows on it is
// slower than fp16 weights (11008 x 4096 with 128 rows 39 us and 31).  4096 x 4096 with
// one row 7.0 us (8.7 MB), 11008 x 4096 with 16 rows 9.8 (25 MB, 2.6 TB/s; in groups of
// 64 with zero points 10.5) and with 64 rows 21.5, 1001 x 4093 in groups of 32 with 61
// rows 10.0.
template <int FL, bool DW>
__global__ void __launch_bounds__(kStreamThreads, 2) w4_rows_kernel(W4Gemm p)
{
    using S = W4Stream<FL, DW, false>;
    constexpr int CPL = S::CPL, CB = S::CB, QUADS = CB / 4;
    __shared__ __attribute__((aligned(16))) float lds[kStreamWaves * 16 * CB];
    __shared__ int flag;
    // neighbouring tiles on one XCD: they share a block of columns
    const int all = p.blocks_m * p.blocks_n * p.parts, per_xcd = (all + 7) / 8;
    const int id = (int)(blockIdx.x & 7) * per_xcd + (int)(blockIdx.x >> 3);
    if (id >= all) return;
    const int part = id % p.parts, tile = id / p.parts;
    const int m0 = tile % p.blocks_m * 16, n0 = tile / p.blocks_m * CB, rows_here = min(16, p.M - m0);

    const int units = (p.K + S::UNIT - 1) / S::UNIT, first = part * p.chunk;
    w4_tile<S>(p, m0, rows_here, n0, first, max(0, min(p.chunk, units - first)), lds);

    const int m = threadIdx.x / QUADS, q = threadIdx.x % QUADS;
    auto finish = [&](f32x4 s) {
        const int col = stream_position<CPL>(n0, q, p.N);
        if (col >= 0) put_half4(p.c + (size_t)(m0 + m) * p.N, col, p.N, w4_epilogue(p, col, s));
    };
    __syncthreads();
    const size_t wide = (size_t)p.blocks_n * CB;
    float* meet = p.part + (size_t)(m0 + m) * wide + n0 + 4 * q;
    if (m < rows_here) {
        const f32x4 s = stream_sum<CPL>(lds, kStreamWaves, m, q);
        if (p.parts > 1) meet_store(meet + (size_t)part * p.M * wide, s);
        else finish(s);
    }
    if (p.parts == 1) return;
    if (!meet_last(p.count + tile, (uint32_t)p.parts, &flag)) return;
    if (m < rows_here) finish(meet_sum(meet, p.parts, (size_t)p.M * wide));
}

// After a product with the weights' values rounded to fp16: the columns of which a
// weight may not fit it (some |scale| times the farthest code from its zero point
// is 65520 or more, the first value that rounds to an infinity), with the weights as
// they are.  A workgroup has 64 columns and looks at their scales (0.7 MB of 11008
// columns of 32 groups, 4.6 us, most of it the launch's); where one is so large it
// walks all rows, its waves each a part of K (1025 x 11008 x 4096 with such a column
// 480 us, with nothing but such columns 500; trained weights have none).  A scale that
// is not finite is left to the product: its column's sums are not finite either way.
template <int FL, bool DW>
__global__ void __launch_bounds__(kStreamThreads, 2) w4_past_kernel(W4Gemm p)
{
    using S = W4Stream<FL, DW, false>;
    constexpr int CPL = S::CPL, CB = S::CB, QUADS = CB / 4, ROWS = kStreamThreads / QUADS;
    __shared__ __attribute__((aligned(16))) float lds[kStreamWaves * 16 * CB];
    __shared__ uint32_t past[QUADS];  // bit i: column i of the quad
    const int n0 = blockIdx.x * CB, m = threadIdx.x / QUADS, q = threadIdx.x % QUADS;
    const int col = stream_position<CPL>(n0, q, p.N), groups = ((p.K - 1) >> p.w.glog2) + 1;
    if (threadIdx.x < QUADS) past[threadIdx.x] = 0u;
    __syncthreads();
    uint32_t mine = 0u;
    if (col >= 0)
        for (int g = m; g < groups; g += ROWS)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (col + i >= p.N) break;
                const size_t at = (size_t)g * p.N + col + i;
                const float s = fabsf(half_at(p.w.scales + at)), z = p.w.zeros ? (float)p.w.zeros[at] : 8.0f;
                if (s <= 65504.0f && s * fmaxf(z, 15.0f - z) >= 65520.0f) mine |= 1u << i;
            }
    if (mine) atomicOr(&past[q], mine);
    __syncthreads();
    bool any = false;
    for (int i = 0; i < QUADS; ++i) any = any || past[i] != 0u;
    if (!any) return;
    for (int64_t m0 = 0; m0 < p.M; m0 += 16) {
        const int rows_here = (int)min((int64_t)16, p.M - m0);
        w4_tile<S>(p, m0, rows_here, n0, 0, (p.K + S::UNIT - 1) / S::UNIT, lds);
        __syncthreads();
        if (m < rows_here && col >= 0) {
            const f32x4 s = w4_epilogue(p, col, stream_sum<CPL>(lds, kStreamWaves, m, q));
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (past[q] >> i & 1u && col + i < p.N) p.c[(size_t)(m0 + m) * p.N + col + i] = to_half(s[i]);
        }
        __syncthreads();  // the next tile's sums
    }
}

// ---- quantizing --------------------------------------------------------------------
struct W4Convert {
    const uint16_t* b;    // matrices x K x N
    uint16_t* values;     // the same, written by dequantize
    uint32_t* codes;
    uint16_t* scales;
    uint8_t* zeros;
    int K, N, glog2, groups;
    int64_t matrices;
};

// What a group's values make of its scale and zero point, and a code of them.
struct W4Step {
    float s, r;
    int z;
    uint16_t bits;
    bool live;
    __device__ __forceinline__ W4Step(float lo, float hi, bool odd, bool zeros)
    {
        const float step = zeros ? (hi - lo) / 15.0f : fmaxf(-lo, hi) / 7.0f;
        bits = odd ? (uint16_t)0x7e00 : to_half(step);
        s = (float)__builtin_bit_cast(_Float16, bits);
        live = s > 0.0f;
        r = live ? 1.0f / s : 0.0f;
        z = zeros && live ? (int)fminf(fmaxf(rintf(quotient(-lo)), 0.0f), 15.0f) : 8;
    }
    // v / s rounded as a division would be wherever that decides a code: from a
    // quotient off by an ulp or two one correction, exact where v / s is half a
    // whole number (then v - t s is the error itself); any other quotient of two
    // fp16 values lies 2^-16 of itself away from those.
    __device__ __forceinline__ float quotient(float v) const
    {
        const float t = v * r;
        return fmaf(fmaf(-t, s, v), r, t);
    }
    // The codes of eight values as a word, each added in by one shift-and-add: the
    // quotient between -z and 15 - z plus 3 2^22 is a float whose bits are
    // 0x4b400000 and the quotient rounded to even; what eight of those bits and
    // zero points make is added at the end.
    template <class Value>
    __device__ __forceinline__ uint32_t word(Value&& value) const
    {
        const float least = (float)-z, most = (float)(15 - z);
        uint32_t w = 0u;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = __builtin_amdgcn_fmed3f(quotient(value(i)), least, most) + 12582912.0f;
            w += __builtin_bit_cast(uint32_t, q) << (4 * i);
        }
        return live ? w + ((uint32_t)z - 0x4b400000u) * 0x11111111u : 0x88888888u;
    }
};

typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));

// Four columns' least and largest values, two to a register, and the largest of
// their bits without the sign: of an infinity or a NaN 0x7c00 or more.
template <bool ZEROS>
struct W4Range {
    half2v lo[2] = {}, hi[2] = {};
    ushort2v top[2] = {};
    // Column j's least and largest value, a NaN as the least for such a one.
    __device__ __forceinline__ void get(int j, float& least, float& most) const
    {
        const uint16_t t = top[j / 2][j & 1];
        const float size = (float)__builtin_bit_cast(_Float16, t);
        least = t >= 0x7c00u ? __builtin_nanf("") : ZEROS ? (float)lo[j / 2][j & 1] : -size;
        most = ZEROS ? (float)hi[j / 2][j & 1] : size;
    }
    __device__ __forceinline__ void take(u32x2 v)
    {
#pragma unroll
        for (int d = 0; d < 2; ++d) {
            const uint32_t w = v[d];
            top[d] = __builtin_elementwise_max(top[d], __builtin_bit_cast(ushort2v, w & 0x7fff7fffu));
            if constexpr (ZEROS) {
                lo[d] = __builtin_elementwise_min(lo[d], __builtin_bit_cast(half2v, w));
                hi[d] = __builtin_elementwise_max(hi[d], __builtin_bit_cast(half2v, w));
            }
        }
    }
};

// A wave has 256 columns, four per lane, and 32 rows of a group, in registers;
// the four waves of a workgroup have 128 rows, one to four groups, and tell each
// other their largest values through LDS.  Larger groups are walked 128 rows at
// a time, twice (LONG).  4096 x 11008: 113 MB in 29 us, 3.9 TB/s, with zero points
// 31: every wave loads before it computes, 1376 workgroups on 1024 places; eight
// waves of 16 rows take the same.  (20 to 40 scalar values live in lanes of vector
// registers.)
template <bool LONG, bool ZEROS>
__global__ void __launch_bounds__(256) w4_quantize_kernel(W4Convert p)
{
    __shared__ u32x4 least[4][64], most[4][64];  // four columns: lo, hi as floats
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int words = (p.K + 7) / 8;
    const bool live = ((int)blockIdx.x * 64 + lane) * 4 < p.N;
    const int c = min(((int)blockIdx.x * 64 + lane) * 4, p.N - 4);
    const int spans = LONG ? p.groups : (p.K + 127) / 128;  // of 128 rows or a longer group
    const int64_t all = p.matrices * spans;
    for (int64_t es = blockIdx.y; es < all; es += gridDim.y) {
        const int64_t e = es / spans, span = es % spans;
        const uint16_t* b = p.b + (size_t)e * p.K * p.N;
        const int64_t k_span = LONG ? span << p.glog2 : span * 128;
        const int64_t k_end = LONG ? min((int64_t)p.K, k_span + ((int64_t)1 << p.glog2)) : min((int64_t)p.K, k_span + 128);
        u32x2 v[32];
        auto load = [&](int64_t k0) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                const int64_t k = k0 + 32 * wave + i;
                v[i] = *(const u32x2_at2*)(b + (size_t)min(k, (int64_t)p.K - 1) * p.N + c);
                if (k >= k_end) v[i] = u32x2{0u, 0u};
            }
        };
        W4Range<ZEROS> range;
        for (int64_t k0 = k_span; k0 < k_end; k0 += 128) {
            load(k0);
#pragma unroll
            for (int i = 0; i < 32; ++i) range.take(v[i]);
        }
        __syncthreads();  // the last span's values are read
        u32x4 put_lo, put_hi;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float lo, hi;
            range.get(j, lo, hi);
            put_lo[j] = __builtin_bit_cast(uint32_t, lo);
            put_hi[j] = __builtin_bit_cast(uint32_t, hi);
        }
        least[wave][lane] = put_lo;
        most[wave][lane] = put_hi;
        __syncthreads();
        // the waves of this wave's group
        const int share = LONG ? 4 : max(1, min(4, (1 << p.glog2) / 32)), w0 = wave / share * share;
        float glo[4] = {}, ghi[4] = {};
        bool godd[4] = {};
        for (int w = w0; w < w0 + share; ++w) {
            const u32x4 a = least[w][lane], d = most[w][lane];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float x = __builtin_bit_cast(float, (uint32_t)a[j]);
                godd[j] |= x != x;
                glo[j] = fminf(glo[j], x);
                ghi[j] = fmaxf(ghi[j], __builtin_bit_cast(float, (uint32_t)d[j]));
            }
        }
        const W4Step st[4] = {{glo[0], ghi[0], godd[0], ZEROS}, {glo[1], ghi[1], godd[1], ZEROS},
                              {glo[2], ghi[2], godd[2], ZEROS}, {glo[3], ghi[3], godd[3], ZEROS}};
        const int64_t group = (LONG ? k_span : k_span + 32 * wave) >> p.glog2;
        if (live && wave == w0 && group < p.groups) {
            const size_t at = ((size_t)e * p.groups + group) * p.N + c;
            *(u32x2_at2*)(p.scales + at) = u32x2{join16(st[0].bits, st[1].bits), join16(st[2].bits, st[3].bits)};
            if (ZEROS)
                *(u32_at1*)(p.zeros + at) = (uint32_t)st[0].z | (uint32_t)st[1].z << 8 | (uint32_t)st[2].z << 16 | (uint32_t)st[3].z << 24;
        }
        for (int64_t k0 = k_span; k0 < k_end; k0 += 128) {
            if (LONG) load(k0);
#pragma unroll
            for (int x = 0; x < 4; ++x) {
                u32x4 w;
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    w[j] = st[j].word([&](int i) {
                        return (float)__builtin_bit_cast(_Float16, (uint16_t)(v[8 * x + i][j / 2] >> (16 * (j & 1))));
                    });
                const int64_t row = k0 / 8 + 4 * wave + x;
                if (live && row < words) *(u32x4_at4*)(p.codes + ((size_t)e * words + row) * p.N + c) = w;
            }
        }
    }
}

// 32 rows of four columns per lane, which are of one group.  4096 x 11008: 113 MB
// in 19 us, 6.0 TB/s.
__global__ void __launch_bounds__(256) w4_dequantize_kernel(W4Convert p)
{
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int words = (p.K + 7) / 8, strips = (p.K + 31) / 32;
    const int c0 = ((int)blockIdx.x * 64 + lane) * 4, c = min(c0, p.N - 4);
    if (c0 >= p.N) return;
    const int64_t all = p.matrices * strips;
    for (int64_t es = (int64_t)blockIdx.y * 4 + wave; es < all; es += (int64_t)gridDim.y * 4) {
        const int64_t e = es / strips;
        const int k0 = (int)(es % strips) * 32;
        const size_t at = ((size_t)e * p.groups + (k0 >> p.glog2)) * p.N + c;
        const u32x2 sb = *(const u32x2_at2*)(p.scales + at);
        const uint32_t zb = p.zeros ? *(const u32_at1*)(p.zeros + at) : 0x08080808u;
        u32x4 w[4];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            w[x] = *(const u32x4_at4*)(p.codes + ((size_t)e * words + min(k0 / 8 + x, words - 1)) * p.N + c);
        float s[4], z[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            s[j] = (float)__builtin_bit_cast(_Float16, (uint16_t)(sb[j / 2] >> (16 * (j & 1))));
            z[j] = (float)((zb >> (8 * j)) & 0xffu);
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) {
            if (k0 + i >= p.K) break;
            uint16_t h[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) h[j] = to_half(((float)((w[i / 8][j] >> (4 * (i % 8))) & 15u) - z[j]) * s[j]);
            *(u32x2_at2*)(p.values + ((size_t)e * p.K + k0 + i) * p.N + c) = u32x2{join16(h[0], h[1]), join16(h[2], h[3])};
        }
    }
}

// Both for fewer than four columns: one thread per column and group, and per
// column and word.
__global__ void __launch_bounds__(256) w4_quantize_narrow_kernel(W4Convert p)
{
    const int words = (p.K + 7) / 8;
    const int64_t all = p.matrices * p.groups * p.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int n = (int)(i % p.N);
        const int64_t eg = i / p.N, e = eg / p.groups, k0 = (eg % p.groups) << p.glog2, k1 = min((int64_t)p.K, k0 + ((int64_t)1 << p.glog2));
        const uint16_t* b = p.b + (size_t)e * p.K * p.N + n;
        float lo = 0.0f, hi = 0.0f;
        bool odd = false;
        for (int64_t k = k0; k < k1; ++k) {
            const float v = half_at(b + (size_t)k * p.N);
            odd |= !(fabsf(v) <= 65504.0f);
            lo = fminf(lo, v);
            hi = fmaxf(hi, v);
        }
        const W4Step st(lo, hi, odd, p.zeros != nullptr);
        p.scales[i] = st.bits;
        if (p.zeros) p.zeros[i] = (uint8_t)st.z;
        for (int64_t k = k0; k < k1; k += 8) {
            p.codes[((size_t)e * words + k / 8) * p.N + n] =
                st.word([&](int x) { return k + x < k1 ? half_at(b + (size_t)(k + x) * p.N) : 0.0f; });
        }
    }
}

__global__ void __launch_bounds__(256) w4_dequantize_narrow_kernel(W4Convert p)
{
    const int words = (p.K + 7) / 8;
    const int64_t all = p.matrices * words * p.N;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)gridDim.x * 256) {
        const int n = (int)(i % p.N);
        const int64_t er = i / p.N, e = er / words;
        const int r = (int)(er % words);
        const uint32_t w = p.codes[i];
        const size_t at = ((size_t)e * p.groups + ((8 * r) >> p.glog2)) * p.N + n;
        const float s = half_at(p.scales + at), z = p.zeros ? (float)p.zeros[at] : 8.0f;
        for (int x = 0; x < 8 && 8 * r + x < p.K; ++x)
            p.values[((size_t)e * p.K + 8 * r + x) * p.N + n] = to_half(((float)((w >> (4 * x)) & 15u) - z) * s);
    }
}

}  // namespace gsr
