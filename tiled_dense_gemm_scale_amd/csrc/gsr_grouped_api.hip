// gsr_grouped_api.hip -- host side of the grouped products of include/gsr.h:
// argument checks, the tile and the launch on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gsr.h"
#include "gsr_host.hpp"
#include "gsr_interleave16c.hpp"
#include "gsr_interleave16d.hpp"
#include "gsr_kspec.hpp"

namespace gsr {

// K == 0: every row of a group is act(alpha * 0 + bias[n]) (+0 without one).
static __global__ void __launch_bounds__(256) fill_grouped_kernel(Problem p)
{
    for (int e = blockIdx.x; e < p.groups; e += gridDim.x) {
        const int lo = min(max(p.offsets[e], 0), p.M), hi = min(p.offsets[e + 1], p.M);
        for (int64_t i = (int64_t)lo * p.N + threadIdx.x; i < (int64_t)hi * p.N; i += 256) {
            const int n = (int)(i % p.N);
            const float b = p.bias ? (float)__builtin_bit_cast(_Float16, p.bias[(int64_t)e * p.N + n]) : 0.0f;
            p.C[i] = (p.bias != nullptr || p.act != kActRelu)
                         ? __builtin_bit_cast(uint16_t, (_Float16)activate(0.0f * p.alpha + b, p.act))
                         : (uint16_t)0;
        }
    }
}

}  // namespace gsr

namespace {

using gsr::Problem;
using namespace gsr::host;

constexpr int64_t kLimit = (int64_t)1 << 31;
constexpr int64_t kMaxGroups = 1024;

typedef hipError_t (*launch_fn)(const Problem&, int grid, hipStream_t);

template <class T>
hipError_t launch_ilv16d(const Problem& p, int grid, hipStream_t s)
{
    return launch_kernel(gsr::gemm_scale_relu_ilv16d_kernel<T, true>, dim3(grid), dim3(T::NT), s, p);
}

template <class T>
hipError_t launch_ilv16c(const Problem& p, int grid, hipStream_t s)
{
    return launch_kernel(gsr::gemm_scale_relu_ilv16c_kernel<T, true>, dim3(grid), dim3(T::NT), s, p);
}

template <int BM, int BN, int S, int D>
hipError_t launch_kspec(const Problem& p, int grid, hipStream_t s)
{
    return launch_kernel((gsr::gemm_scale_relu_kspec_kernel<BM, BN, S, D, false, true>), dim3(grid), dim3(512), s, p);
}

template <int BM, int BN, int KG>
hipError_t launch_staged(const Problem& p, int grid, hipStream_t s)
{
    return launch_kernel((gsr::gemm_scale_relu_kernel<BM, BN, 64, 2, 2, false, true, gsr::kAdaptNone, KG>), dim3(grid),
                         dim3(256 * KG), s, p);
}

// The element-wise kernels, in the order of kElemTiles.
const launch_fn kElem[] = {launch_staged<64, 64, 4>, launch_staged<64, 64, 1>, launch_staged<128, 128, 1>};

// The grouped forms of the selector's tiles, under the ids of their dense
// forms.
struct Entry {
    int id;
    int bm, bn, threads;
    launch_fn vec;
};
const Entry kTable[] = {
    {21, 64, 64, 512, launch_kspec<64, 64, 4, 2>},
    {22, 32, 64, 512, launch_kspec<32, 64, 4, 2>},
    {28, 256, 256, 256, launch_ilv16d<gsr::Ilv16DCfg>},
    {31, 128, 256, 512, launch_ilv16c<gsr::Ilv16CCfg>},
    {32, 128, 128, 512, launch_ilv16c<gsr::Ilv16QCCfg>},
};

const Entry* entry_of(int id)
{
    for (const Entry& e : kTable)
        if (e.id == id) return &e;
    return nullptr;
}

// Tiles of bm rows to expect of P rows in `used` groups.  The group sizes are on
// the device, so they are taken as spread about their mean like an exponential
// distribution's, for which a group has 1 / (1 - exp(-bm / mean)) of them on
// average.
double tile_rows(int64_t P, int64_t used, int bm)
{
    return (double)used / (1.0 - std::exp(-(double)bm * (double)used / (double)P));
}

// The tile rows of a launch, at most: one part-filled tile for each group that
// has rows.
int64_t most_tile_rows(int64_t P, int64_t used, int bm) { return (P + used * (bm - 1)) / bm; }

// The tile.  Decode steps are bound by B's bytes (16 tokens, 2 of 8 experts,
// 4096 -> 11008: 116 to 126 us, 5.5 TB/s and more of what the hit experts hold),
// prefills by the matrix cores (8192 tokens: 1.22 ms, 1.21 PFLOP/s), and in
// between it is whole rounds of tiles that count (1025 tokens, 11008 -> 4096:
// 231 us, 0.80 PFLOP/s: 184 tiles of 256 x 256 on 256 CUs, 69 % of their rows
// filled).  The estimate is the larger of two times plus a twentieth of the smaller: the
// tiles' (the dense selector's time of one, in rounds of 256 workgroups, a
// part-filled last round costing 0.6 + 0.4 fill) and that of reading B once
// per tile row at 5.5 TB/s.  Its constants come from a grid search over the
// times of all five tiles on 40 cases on one MI355X (1 to 8192 tokens, two of
// 8 experts of 4096 x 11008 and 11008 x 4096, eight of 64 experts of 2048 x
// 1024 and 1024 x 2048): on average 1.6 % above the fastest tile, 29 % on the
// worst (64 rows per expert, where 1.2 rounds of 256 x 256 tiles are expected
// and one happens); the dense selector's own rule was 4 % above on average.
// The 128 x 128 tile runs 5 % faster here than the dense fit has it.
const Entry& select(int64_t P, int64_t groups, int64_t N, int64_t K)
{
    const int64_t used = std::min(groups, P);
    const Entry* best = nullptr;
    double best_t = 1e300;
    for (const Entry& e : kTable) {
        // (the tile with the fewest threads per output stays in any case)
        if (e.id != 28 && !grid_fits(most_tile_rows(P, used, e.bm) * cdiv(N, e.bn), e.threads)) continue;
        const double rows = tile_rows(P, used, e.bm);
        const double rounds = std::ceil(rows * (double)cdiv(N, e.bn)) / 256.0;
        const double full = std::floor(rounds), fill = rounds - full;
        const double work = std::max(1.0, full + (fill > 0.0 ? 0.6 + 0.4 * fill : 0.0)) * tile_time(e.id, K) *
                            (e.id == 32 ? 0.95 : 1.0);
        const double read = rows * (double)K * (double)N * 2.0 / 5.5e6;
        const double t = std::max(work, read) + 0.05 * std::min(work, read);
        if (t < best_t) best_t = t, best = &e;
    }
    return *best;
}

}  // namespace

extern "C" {

int gemm_grouped_scale_bias_act(int64_t P, int64_t N, int64_t K, int64_t groups, const void* A, int64_t a_rows,
                                const int32_t* rows, const void* B, const void* bias, void* C,
                                const int32_t* offsets, float alpha, int32_t activation, void* stream,
                                int32_t config_id)
{
    if (P < 0 || N < 0 || K < 0 || groups < 0 || a_rows < 0) return GSR_ERROR_INVALID_VALUE;
    if (rows == nullptr) a_rows = P;
    // 32-bit byte offsets within a tile of C, within one group's B and, with
    // rows, within A
    if (P >= kLimit || N >= kLimit || K >= kLimit || a_rows >= kLimit || groups > kMaxGroups) return GSR_ERROR_TOO_LARGE;
    if (N * 512 >= kLimit || K * 512 >= kLimit || N * K * 2 >= kLimit) return GSR_ERROR_TOO_LARGE;
    if (rows != nullptr && a_rows * K * 2 >= kLimit) return GSR_ERROR_TOO_LARGE;
    if (!std::isfinite(alpha)) return GSR_ERROR_INVALID_VALUE;
    if (activation != GSR_ACT_RELU && activation != GSR_ACT_GELU && activation != GSR_ACT_NONE)
        return GSR_ERROR_INVALID_VALUE;
    if (config_id < -1 || (config_id >= 0 && entry_of(config_id) == nullptr)) return GSR_ERROR_INVALID_CONFIG;
    if (P == 0 || N == 0 || groups == 0) return GSR_SUCCESS;
    if (C == nullptr || offsets == nullptr || misaligned(C, 2) || misaligned(offsets, 4) || misaligned(rows, 4) ||
        misaligned(A, 2) || misaligned(B, 2) || misaligned(bias, 2))
        return GSR_ERROR_INVALID_VALUE;
    if (K > 0 && (B == nullptr || (A == nullptr && a_rows > 0))) return GSR_ERROR_INVALID_VALUE;
    const uint64_t cb = (uint64_t)P * (uint64_t)N * 2u;
    if (overlaps(C, cb, A, (uint64_t)a_rows * (uint64_t)K * 2u) ||
        overlaps(C, cb, B, (uint64_t)groups * (uint64_t)K * (uint64_t)N * 2u) ||
        overlaps(C, cb, offsets, (uint64_t)(groups + 1) * 4u) ||
        (rows != nullptr && overlaps(C, cb, rows, (uint64_t)P * 4u)) ||
        (bias != nullptr && overlaps(C, cb, bias, (uint64_t)groups * (uint64_t)N * 2u)))
        return GSR_ERROR_INVALID_VALUE;
    Problem p{};
    p.A = (const uint16_t*)A;
    p.B = (const uint16_t*)B;
    p.C = (uint16_t*)C;
    p.bias = (const uint16_t*)bias;
    p.M = (int)P;
    p.N = (int)N;
    p.K = (int)K;
    p.alpha = alpha;
    p.act = (int)activation;
    p.offsets = offsets;
    p.rows = rows;
    p.groups = (int)groups;
    p.a_rows = (int)a_rows;
    p.ksplit = 1;
    p.kchunk = (int)K;
    p.xcd_remap = 1;
    p.unit_a = load_unit(A, K);
    p.unit_b = load_unit(B, N);
    p.unit_c = load_unit(C, N);
    const bool vec = p.unit_a == 16 && p.unit_b == 16 && (((uintptr_t)bias & 7u) == 0);
    const int64_t used = std::min(groups, P);
    int bm, bn, threads;
    launch_fn fn;
    p.group_m = 4;
    if (vec) {
        const Entry& e = config_id >= 0 ? *entry_of(config_id) : select(P, groups, N, K);
        bm = e.bm, bn = e.bn, threads = e.threads, fn = e.vec;
    } else {
        const int i = elem_choice(config_id, K, tile_rows(P, used, 64) * (double)cdiv(N, 64), tile_rows(P, used, 128) * (double)cdiv(N, 128));
        bm = kElemTiles[i].bm, bn = kElemTiles[i].bn, threads = kElemTiles[i].threads, fn = kElem[i];
    }
    const int64_t tiles_n = cdiv(N, bn), tiles_m = most_tile_rows(P, used, bm);
    if (K > 0 && !grid_fits(tiles_m * tiles_n, threads)) return GSR_ERROR_TOO_LARGE;
    const int st = check_device();
    if (st != GSR_SUCCESS) return st;
    hipStream_t s = (hipStream_t)stream;
    if (K == 0) return status_of(launch_kernel(gsr::fill_grouped_kernel, dim3((unsigned)groups), dim3(256), s, p));
    p.tiles_n = (int)tiles_n;
    p.tiles_m = (int)tiles_m;
    return status_of(fn(p, (int)(tiles_m * tiles_n), s));
}

}  // extern "C"
