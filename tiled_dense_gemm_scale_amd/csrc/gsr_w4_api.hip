// gsr_w4_api.hip -- host side of the 4-bit weights' entry points of
// include/gsr.h: argument checks and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gsr.h"
#include "gsr_few_host.hpp"
#include "gsr_w4_kernels.hpp"

namespace {

using namespace gsr::host;

constexpr int64_t kLimit = (int64_t)1 << 31;

int check_matrix(int64_t matrices, int64_t K, int64_t N, int64_t group)
{
    if (matrices < 0 || K < 0 || N < 0 || group_log2(group) < 0) return GSR_ERROR_INVALID_VALUE;
    if (matrices >= kLimit || K >= gsr::host::kStreamWidth || N >= gsr::host::kStreamWidth ||
        (K > 0 && N > 0 && matrices > ((int64_t)1 << 56) / (K * N)))
        return GSR_ERROR_TOO_LARGE;
    return GSR_SUCCESS;
}

gsr::W4Convert convert_args(int64_t matrices, int64_t K, int64_t N, int64_t group)
{
    gsr::W4Convert p{};
    p.K = (int)K;
    p.N = (int)N;
    p.glog2 = group_log2(group);
    p.groups = (int)cdiv(K, group);
    p.matrices = matrices;
    return p;
}

constexpr int64_t kGridY = 32768;

struct GemmPlan {
    bool dense;  // the weights' values in the workspace, then the dense product
    int parts, chunk;
    int64_t blocks_m, blocks_n, bytes;
};

// Many rows are bound by the matrix cores, whose tiles of 256 rows the stream does
// not have: there the values are written out once, 2.5 bytes to and from memory
// per weight, the dense kernels multiply them, and a third launch looks after the
// columns past fp16.  A matrix of 2^30 weights and more has no such way (the dense
// kernels' are below 2^31 bytes): 1025 rows with 8192 x 131064 3.0 ms, with 8192 x
// 131072 5.7.  That rounds each weight to fp16 (error of C against 64 bits
// 0.00021, its own rounding's, to 0.00027).  In us, the stream, and the three steps:
// 11008 x 4096 with 64 rows 21 and 37, 160 rows 45 and 56, 192 rows 56 and 50, 1025
// rows 271 and 112; 2048 x 2048 with 512 rows 19 and 23, 1025 rows 36 and 30; 1000 x
// 4096 with 1500 rows 45 and 40; 333 x 1001 with 4000 rows 26 and 44.  The stream takes 2 and for each round
// of 256 workgroups 1.4 and 0.16 per unit of K (0.25 where rows of A start at odd
// elements); the values 9 and 7 TB/s (the look at the scales is not counted: a call
// among others sees 0 to 4 of its 4.6 us); the dense products their selector's time,
// off the 128-bit path 34 ns per K or 340 TFLOP/s.
bool dense_pays(int64_t M, int64_t N, int64_t K, bool vec)
{
    const double mnk = 2.0 * (double)M * (double)N * (double)K;
    const double rounds = std::max(1.0, (double)cdiv(M, 16) * (double)cdiv(N, 64) / 256.0);
    const double stream = 2.0 + rounds * (1.4 + (K % 2 == 0 ? 0.16 : 0.25) * (double)cdiv(K, 128));
    const double dense = vec ? dense_time(M, N, K) : std::max(0.034 * (double)K, mnk * 1e-6 / 340.0);
    return 9.0 + 2.5 * (double)K * (double)N * 1e-6 / 7.0 + dense < stream;
}

// Parts of K, of `chunk` units each, so that the tiles make about 256 workgroups of
// a unit per wave at least: tiles of more than one part are at most 128, one to a
// counter.  Meeting costs as much as three units of a wave: in us with parts and
// without, 4096 x 4096 with one row 7.4 (four) and 8.2, 1001 x 4093 6.7 and 8.5,
// 4096 x 11008 with 32 rows 13.6 (two) and 16.4; but 2048 x 2048 6.2 (two) and 5.8,
// 4096 x 4096 with 32 rows 9.2 (two) and 8.7.
struct Parts {
    int parts, chunk;
};
Parts stream_parts(int64_t tiles, int64_t units)
{
    constexpr int64_t W = gsr::kStreamWaves;
    const int64_t want = std::min<int64_t>({16, 256 / std::max<int64_t>(tiles, 1), units / W});
    if (want < 2 || units * (want - 1) < 3 * W * want) return Parts{1, (int)std::max<int64_t>(units, 1)};
    const int64_t chunk = cdiv(units, want);
    return Parts{(int)cdiv(units, chunk), (int)chunk};
}

// aligned: A and the bias let the dense product take its 128-bit path.
GemmPlan gemm_plan(int64_t M, int64_t N, int64_t K, int64_t bytes, bool aligned)
{
    constexpr int CB = gsr::W4Stream<1, true, false>::CB, UNIT = gsr::W4Stream<1, true, false>::UNIT;
    GemmPlan g;
    const int64_t units = cdiv(K, UNIT), values = gsr::kMeetBytes + 2 * K * N;
    g.blocks_m = cdiv(M, 16);
    g.blocks_n = cdiv(N, CB);
    const int64_t tiles = g.blocks_m * g.blocks_n;
    g.dense = M > 16 && K > 0 && values < kLimit && (bytes < 0 || values <= bytes) &&
              dense_pays(M, N, K, aligned && K % 8 == 0 && N % 8 == 0);
    Parts p = stream_parts(tiles, units);
    auto need = [&](int parts) { return parts > 1 ? gsr::kMeetBytes + (int64_t)parts * M * g.blocks_n * CB * 4 : 0; };
    if (bytes >= 0 && need(p.parts) > bytes) p = Parts{1, (int)std::max<int64_t>(units, 1)};
    g.parts = p.parts;
    g.chunk = p.chunk;
    g.bytes = g.dense ? values : need(p.parts);
    return g;
}

typedef void (*gemm_kernel)(gsr::W4Gemm);
struct GemmKernels {
    gemm_kernel rows, past;
};
template <int FL>
GemmKernels gemm_form(bool dwords)
{
    return dwords ? GemmKernels{gsr::w4_rows_kernel<FL, true>, gsr::w4_past_kernel<FL, true>}
                  : GemmKernels{gsr::w4_rows_kernel<FL, false>, gsr::w4_past_kernel<FL, false>};
}
GemmKernels gemm_form(int64_t group, bool dwords)
{
    return group == 32 ? gemm_form<1>(dwords) : group == 64 ? gemm_form<2>(dwords) : gemm_form<4>(dwords);
}

}  // namespace

extern "C" {

int gsr_quantize_w4(int64_t matrices, int64_t K, int64_t N, int64_t group, const void* B, uint32_t* codes, void* scales,
                    uint8_t* zeros, void* stream)
{
    int st = check_matrix(matrices, K, N, group);
    if (st != GSR_SUCCESS) return st;
    const uint64_t sc = w4_scale_count((uint64_t)matrices, K, N, group);
    const Span b{B, (uint64_t)matrices * (uint64_t)K * (uint64_t)N * 2u, 2}, q{codes, w4_code_bytes((uint64_t)matrices, K, N), 4},
        s{scales, 2u * sc, 2}, z{zeros, zeros ? sc : 0u, 1};
    if (b.bytes == 0) return GSR_SUCCESS;
    if (unusable({b, q, s}) || clash(q, {b, s, z}) || clash(s, {b, z}) || clash(z, {b})) return GSR_ERROR_INVALID_VALUE;
    st = check_device();
    if (st != GSR_SUCCESS) return st;
    gsr::W4Convert p = convert_args(matrices, K, N, group);
    p.b = (const uint16_t*)B;
    p.codes = codes;
    p.scales = (uint16_t*)scales;
    p.zeros = zeros;
    if (N < 4)
        return status_of(launch_kernel(gsr::w4_quantize_narrow_kernel, dim3((unsigned)std::min(cdiv(matrices * p.groups * N, 256), kGridY)),
                                       dim3(256), (hipStream_t)stream, p));
    const bool longer = group > 128;
    const dim3 grid((unsigned)cdiv(N, 256), (unsigned)std::min(matrices * (longer ? p.groups : cdiv(K, 128)), kGridY));
    const auto f = zeros ? (longer ? gsr::w4_quantize_kernel<true, true> : gsr::w4_quantize_kernel<false, true>)
                         : (longer ? gsr::w4_quantize_kernel<true, false> : gsr::w4_quantize_kernel<false, false>);
    return status_of(launch_kernel(f, grid, dim3(256), (hipStream_t)stream, p));
}

int gsr_dequantize_w4(int64_t matrices, int64_t K, int64_t N, int64_t group, const uint32_t* codes, const void* scales,
                      const uint8_t* zeros, void* B, void* stream)
{
    int st = check_matrix(matrices, K, N, group);
    if (st != GSR_SUCCESS) return st;
    const uint64_t sc = w4_scale_count((uint64_t)matrices, K, N, group);
    const Span b{B, (uint64_t)matrices * (uint64_t)K * (uint64_t)N * 2u, 2}, q{codes, w4_code_bytes((uint64_t)matrices, K, N), 4},
        s{scales, 2u * sc, 2}, z{zeros, zeros ? sc : 0u, 1};
    if (b.bytes == 0) return GSR_SUCCESS;
    if (unusable({b, q, s}) || clash(b, {q, s, z})) return GSR_ERROR_INVALID_VALUE;
    st = check_device();
    if (st != GSR_SUCCESS) return st;
    gsr::W4Convert p = convert_args(matrices, K, N, group);
    p.values = (uint16_t*)B;
    p.codes = const_cast<uint32_t*>(codes);
    p.scales = (uint16_t*)const_cast<void*>(scales);
    p.zeros = const_cast<uint8_t*>(zeros);
    if (N < 4)
        return status_of(launch_kernel(gsr::w4_dequantize_narrow_kernel, dim3((unsigned)std::min(cdiv(matrices * cdiv(K, 8) * N, 256), kGridY)),
                                       dim3(256), (hipStream_t)stream, p));
    const dim3 grid((unsigned)cdiv(N, 256), (unsigned)std::min(cdiv(matrices * cdiv(K, 32), 4), kGridY));
    return status_of(launch_kernel(gsr::w4_dequantize_kernel, grid, dim3(256), (hipStream_t)stream, p));
}

int64_t gsr_w4_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0 || M >= kLimit || N >= gsr::host::kStreamWidth || K >= gsr::host::kStreamWidth) return -1;
    return M == 0 || N == 0 ? 0 : std::max(gemm_plan(M, N, K, -1, true).bytes, gemm_plan(M, N, K, -1, false).bytes);
}

int gemm_w4_scale_bias_act(int64_t M, int64_t N, int64_t K, const void* A, int64_t group, const uint32_t* codes,
                           const void* scales, const uint8_t* zeros, const void* bias, void* C, float alpha,
                           int32_t activation, void* workspace, int64_t workspace_bytes, void* stream)
{
    int st = check_matrix(1, K, N, group);
    if (st == GSR_ERROR_INVALID_VALUE || M < 0 || workspace_bytes < 0 || !std::isfinite(alpha) ||
        (activation != GSR_ACT_RELU && activation != GSR_ACT_GELU && activation != GSR_ACT_NONE))
        return GSR_ERROR_INVALID_VALUE;
    if (st != GSR_SUCCESS || M >= kLimit) return GSR_ERROR_TOO_LARGE;
    if (M == 0 || N == 0) return GSR_SUCCESS;
    const uint64_t sc = w4_scale_count(1, K, N, group);
    const Span a{A, (uint64_t)M * (uint64_t)K * 2u, 2}, q{codes, w4_code_bytes(1, K, N), 4}, s{scales, 2u * sc, 2},
        z{zeros, zeros ? sc : 0u, 1}, b{bias, bias ? (uint64_t)N * 2u : 0u, 2}, c{C, (uint64_t)M * (uint64_t)N * 2u, 2},
        w{workspace, workspace ? (uint64_t)workspace_bytes : 0u, 16};
    if (unusable({a, q, s, b, c, w}) || clash(c, {a, q, s, z, b, w}) || clash(w, {a, q, s, z, b}))
        return GSR_ERROR_INVALID_VALUE;
    st = check_device();
    if (st != GSR_SUCCESS) return st;
    const GemmPlan g = gemm_plan(M, N, K, (int64_t)w.bytes, !misaligned(A, 16) && !misaligned(bias, 8));
    gsr::W4Gemm p{};
    p.a = (const uint16_t*)A;
    p.w = gsr::W4Matrix{codes, (const uint16_t*)scales, zeros, group_log2(group)};
    p.bias = (const uint16_t*)bias;
    p.c = (uint16_t*)C;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.act = activation;
    p.alpha = alpha;
    p.blocks_m = (int)g.blocks_m;
    p.blocks_n = (int)g.blocks_n;
    const GemmKernels f = gemm_form(group, K % 2 == 0 && !misaligned(A, 4));
    if (g.dense) {
        void* values = (uint8_t*)workspace + gsr::kMeetBytes;
        st = gsr_dequantize_w4(1, K, N, group, codes, scales, zeros, values, stream);
        // the dense product's matrices are below 2^31 bytes
        const int64_t rows = (kLimit - 1) / (2 * std::max(K, N)) / 256 * 256;
        for (int64_t m = 0; m < M && st == GSR_SUCCESS; m += rows)
            st = gemm_scale_bias_act(std::min(rows, M - m), N, K, (const uint8_t*)A + 2 * m * K, values, bias, (uint8_t*)C + 2 * m * N,
                                     alpha, activation, stream);
        if (st != GSR_SUCCESS) return st;
        return status_of(launch_kernel(f.past, dim3((unsigned)g.blocks_n), dim3(gsr::kStreamThreads), (hipStream_t)stream, p));
    }
    p.parts = g.parts;
    p.chunk = g.chunk;
    p.count = (uint32_t*)workspace;
    p.part = (float*)((uint8_t*)workspace + gsr::kMeetBytes);
    // A launch has fewer than 2^32 threads: more rows than that are several, each of
    // whole tiles (with K split there are at most 128 tiles, and one).
    const int64_t most = (((int64_t)1 << 32) / gsr::kStreamThreads - 8) / g.blocks_n / g.parts;
    for (int64_t m = 0; m < M; m += 16 * most) {
        p.M = (int)std::min(16 * most, M - m);
        p.a = (const uint16_t*)A + m * K;
        p.c = (uint16_t*)C + m * N;
        p.blocks_m = (int)cdiv(p.M, 16);
        const int64_t grid = cdiv((int64_t)p.blocks_m * g.blocks_n * g.parts, 8) * 8;
        const hipError_t err = launch_kernel(f.rows, dim3((unsigned)grid), dim3(gsr::kStreamThreads), (hipStream_t)stream, p);
        if (err != hipSuccess) return status_of(err);
    }
    return GSR_SUCCESS;
}

}  // extern "C"
