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
    if (matrices >= kLimit || K >= gsr::host::kStreamWidth || N >= gsr::host::kStreamWidth) return GSR_ERROR_TOO_LARGE;
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
    int mt, parts, chunk, blocks_n, per;
    int64_t row_blocks, bytes;
};

GemmPlan gemm_plan(int64_t M, int64_t N, int64_t K, int64_t bytes)
{
    constexpr int CB = gsr::W4Stream<1, 1>::CB, UNIT = gsr::W4Stream<1, 1>::UNIT;
    GemmPlan g;
    g.mt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
    g.blocks_n = (int)cdiv(N, CB);
    g.row_blocks = cdiv(M, 16 * g.mt);
    const int64_t units = cdiv(K, UNIT);
    Parts p = g.row_blocks == 1 ? stream_parts(g.blocks_n, units, 1) : Parts{1, (int)std::max<int64_t>(units, 1)};
    auto need = [&](int parts) { return parts > 1 ? gsr::kMeetBytes + (int64_t)parts * M * g.blocks_n * CB * 4 : 0; };
    if (bytes >= 0 && need(p.parts) > bytes) p = Parts{1, (int)std::max<int64_t>(units, 1)};
    g.parts = p.parts;
    g.chunk = p.chunk;
    g.per = (int)cdiv(g.blocks_n, gsr::kMeetCounters);
    g.bytes = need(p.parts);
    return g;
}

typedef void (*gemm_kernel)(gsr::W4Gemm);
template <int MT>
gemm_kernel gemm_form(int glog2)
{
    return glog2 == 5 ? gsr::w4_gemm_kernel<MT, 1> : glog2 == 6 ? gsr::w4_gemm_kernel<MT, 2> : gsr::w4_gemm_kernel<MT, 4>;
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
    const dim3 grid((unsigned)cdiv(N, 256), (unsigned)std::min(matrices * p.groups, kGridY));
    return status_of(launch_kernel(gsr::w4_quantize_kernel, grid, dim3(256), (hipStream_t)stream, p));
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
    const dim3 grid((unsigned)cdiv(N, 256), (unsigned)std::min(matrices * cdiv(K, 8), kGridY));
    return status_of(launch_kernel(gsr::w4_dequantize_kernel, grid, dim3(256), (hipStream_t)stream, p));
}

int64_t gsr_w4_workspace_bytes(int64_t M, int64_t N, int64_t K)
{
    if (M < 0 || N < 0 || K < 0 || M >= kLimit || N >= gsr::host::kStreamWidth || K >= gsr::host::kStreamWidth) return -1;
    return M == 0 || N == 0 ? 0 : gemm_plan(M, N, K, -1).bytes;
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
    const GemmPlan g = gemm_plan(M, N, K, (int64_t)w.bytes);
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
    p.blocks_n = g.blocks_n;
    p.parts = g.parts;
    p.chunk = g.chunk;
    p.per = g.per;
    p.count = (uint32_t*)workspace;
    p.part = (float*)((uint8_t*)workspace + gsr::kMeetBytes);
    const int64_t grid = g.row_blocks * g.blocks_n * g.parts;
    if (!grid_fits(grid, gsr::kStreamThreads)) return GSR_ERROR_TOO_LARGE;
    const gemm_kernel f = g.mt == 1 ? gemm_form<1>(p.w.glog2) : g.mt == 2 ? gemm_form<2>(p.w.glog2) : gemm_form<4>(p.w.glog2);
    return status_of(launch_kernel(f, dim3((unsigned)grid), dim3(gsr::kStreamThreads), (hipStream_t)stream, p));
}

}  // extern "C"
