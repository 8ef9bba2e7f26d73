// gsr_adapters_api.hip -- host side of the product with low-rank adapters:
// argument checks, the workspace's layout, the two launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "gsr.h"
#include "gsr_adapters.hpp"
#include "gsr_host.hpp"
#include "gsr_interleave16c.hpp"
#include "gsr_interleave16d.hpp"
#include "gsr_kspec.hpp"

namespace {

using gsr::Problem;
using gsr::ShrinkArgs;
using namespace gsr::host;

constexpr int64_t kLimit = (int64_t)1 << 31;
constexpr int64_t kMaxRank = gsr::kShrinkMaxRank;
constexpr int64_t kCounterBytes = kSplitCounters * 4;

typedef hipError_t (*launch_fn)(const Problem&, int grid, hipStream_t);

template <class T>
hipError_t launch_ilv16d(const Problem& p, int grid, hipStream_t s)
{
    return launch_kernel(p.lb_vec ? gsr::gemm_scale_relu_ilv16d_kernel<T, false, gsr::kAdaptVec>
                                  : gsr::gemm_scale_relu_ilv16d_kernel<T, false, gsr::kAdaptElem>,
                         dim3(grid), dim3(T::NT), s, p);
}

template <class T>
hipError_t launch_ilv16c(const Problem& p, int grid, hipStream_t s)
{
    return launch_kernel(p.lb_vec ? gsr::gemm_scale_relu_ilv16c_kernel<T, false, gsr::kAdaptVec>
                                  : gsr::gemm_scale_relu_ilv16c_kernel<T, false, gsr::kAdaptElem>,
                         dim3(grid), dim3(T::NT), s, p);
}

template <int BM, int BN, int S, int D, bool SPLIT>
hipError_t launch_kspec(const Problem& p, int grid, hipStream_t s)
{
    return launch_kernel((gsr::gemm_scale_relu_kspec_kernel<BM, BN, S, D, SPLIT, false, gsr::kAdaptVec>), dim3(grid), dim3(512), s, p);
}

template <int BM, int BN, int S, int D>
hipError_t launch_shared(const Problem& p, const ShrinkArgs& a, int makers, int grid, hipStream_t s)
{
    return launch_kernel((gsr::gemm_adapters_kspec_kernel<BM, BN, S, D>), dim3(grid), dim3(512), s, p, a, makers);
}

template <int BM, int BN, int KG>
hipError_t launch_staged(const Problem& p, int grid, hipStream_t s)
{
    return launch_kernel((gsr::gemm_scale_relu_kernel<BM, BN, 64, 2, 2, false, false, gsr::kAdaptVec, KG>), dim3(grid),
                         dim3(256 * KG), s, p);
}

// The element-wise kernels, in the order of kElemTiles.
const launch_fn kElem[] = {launch_staged<64, 64, 4>, launch_staged<64, 64, 1>, launch_staged<128, 128, 1>};

// The tiles with an adapter form, under the ids of their dense forms.
struct Entry {
    int id;
    int bm, bn, threads;
    launch_fn vec, split;
    hipError_t (*shared)(const Problem&, const ShrinkArgs&, int makers, int grid, hipStream_t);  // both steps, or null
};
const Entry kTable[] = {
    {21, 64, 64, 512, launch_kspec<64, 64, 4, 2, false>, launch_kspec<64, 64, 4, 2, true>, launch_shared<64, 64, 4, 2>},
    {22, 32, 64, 512, launch_kspec<32, 64, 4, 2, false>, launch_kspec<32, 64, 4, 2, true>, launch_shared<32, 64, 4, 2>},
    {28, 256, 256, 256, launch_ilv16d<gsr::Ilv16DCfg>, nullptr, nullptr},
    {31, 128, 256, 512, launch_ilv16c<gsr::Ilv16CCfg>, nullptr, nullptr},
    {32, 128, 128, 512, launch_ilv16c<gsr::Ilv16QCCfg>, nullptr, nullptr},
};

const Entry* entry_of(int id)
{
    for (const Entry& e : kTable)
        if (e.id == id) return &e;
    return nullptr;
}

// A dense configuration's stand-in here: the four-wave K-split tiles run as
// their copy-wave twins, 25 and 29 as 28 and 31.
const Entry& stand_in(int id)
{
    switch (id) {
    case 16: id = 21; break;
    case 17: case 18: id = 22; break;
    case 25: id = 28; break;
    case 29: id = 31; break;
    default: break;
    }
    return *entry_of(id);
}

int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// The shrink launch.  In a decode step (kShrinkMixedRows) a workgroup has one
// block of 16 rows, one chunk of ranks, one of the block's adapters (the rows
// are mixed) and, while that makes fewer than kShrinkGrid workgroups, one of
// the parts of about kShrinkPart values of K; a block's workgroups count
// arrivals in the counters at the workspace's start and the last adds up.
// More rows have one workgroup per block and share of its adapters, for all
// of K and all ranks, as many shares as the chip has room for.  In between,
// where few blocks (times chunks: kShrinkFew) walk far (K times the passes
// over the ranks: kShrinkDeep), the parts are the faster way: product and
// sums, us, without and with: 256x4096x11008 rank 64 85 and 67, 230x10112x7808
// rank 107 138 and 105, 512x4096x11008 rank 16 102 and 99; but
// 256x4096x8192 rank 16 39 and 42, 256x4096x4096 23 and 28, and 1024 rows of
// mixed adapters, K 11008, rank 64, 183 and 238.
constexpr int64_t kShrinkMixedRows = 64, kShrinkPart = 1024, kShrinkMaxParts = 16, kShrinkGrid = 512, kShrinkFew = 128,
                  kShrinkDeep = 9216;

struct ShrinkPlan {
    int blocks, parts, kchunk;  // parts 0: all of K in one workgroup
    int slots;
};

ShrinkPlan shrink_plan(int64_t M, int64_t K, int64_t adapters, int64_t rank)
{
    ShrinkPlan s{(int)cdiv(M, gsr::kShrinkRows), 0, (int)K, 1};
    const int64_t most = std::min<int64_t>({M, adapters, gsr::kShrinkRows});
    int64_t wgs = (int64_t)s.blocks * cdiv(rank, gsr::kAdapterChunk);
    if (M > kShrinkMixedRows &&
        (wgs > kShrinkFew || s.blocks >= kSplitCounters || K * cdiv(rank, 4 * gsr::kAdapterChunk) < kShrinkDeep)) {
        s.slots = (int)std::max<int64_t>(1, std::min<int64_t>(most, 256 / s.blocks));
        return s;
    }
    if (M <= kShrinkMixedRows) s.slots = (int)most, wgs *= most;
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>({kShrinkMaxParts, cdiv(K, kShrinkPart), kShrinkGrid / wgs}));
    s.kchunk = (int)(cdiv(cdiv(K, parts), 32) * 32);
    s.parts = (int)cdiv(K, s.kchunk);
    if (M > kShrinkMixedRows) s.slots = (int)std::max<int64_t>(1, std::min<int64_t>(most, kShrinkGrid / (wgs * s.parts)));
    return s;
}

// Few rows on a copy-wave K-split tile: both steps in one launch, if the
// workgroups that make the inner sums are few enough to run beside the tiles'
// (the launch holds one workgroup per CU).
constexpr int kSharedMakers = 128, kSharedLooks = 64;
// its counters, behind those of a K split of at most 64 tiles: arrivals per
// block, flags per block, done
constexpr int kSharedCounters = 64, kSharedFlags = 68, kSharedDone = 72;

// The workspace: counters, the records of t, the rows' scales, the partial
// sums of step 1, those of the product's K split.
struct Layout {
    int chunks;
    int64_t t, t_scale, partial, split;
};

Layout layout_of(int64_t M, int64_t K, int64_t rank)
{
    Layout w;
    w.chunks = (int)cdiv(rank, gsr::kAdapterChunk);
    w.t = kCounterBytes;
    w.t_scale = w.t + round256(M * w.chunks * 64);
    w.partial = w.t_scale + round256(M * 4);
    const ShrinkPlan s = shrink_plan(M, K, 1, rank);  // one adapter: the most parts
    w.split = w.partial + round256((int64_t)s.parts * s.blocks * gsr::kShrinkRows * w.chunks * gsr::kAdapterChunk * 4);
    return w;
}

}  // namespace

extern "C" {

int64_t gsr_adapter_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t rank)
{
    if (M < 0 || N < 0 || K < 0 || rank < 0 || M >= kLimit || N >= kLimit || K >= kLimit || rank > kMaxRank) return -1;
    if (M == 0 || N == 0 || K == 0) return 0;
    if (rank == 0) return gsr_workspace_bytes(M, N, K);
    if (!grid_fits(cdiv(M, gsr::kShrinkRows), 512)) return -1;
    const Entry& e = stand_in(dense_launch(M, N, K).id);
    const int64_t split = e.split ? dense_split(M, N, K, cdiv(M, e.bm) * cdiv(N, e.bn), e.bm, e.bn, 0).partial_bytes : 0;
    return layout_of(M, K, rank).split + split;
}

int gemm_adapters_scale_bias_act(int64_t M, int64_t N, int64_t K, const void* A, const void* B, const void* bias,
                                 void* C, int64_t adapters, int64_t rank, const void* la, const void* lb,
                                 const int32_t* ids, const float* scales, float alpha, int32_t activation,
                                 void* workspace, int64_t workspace_bytes, void* stream, int32_t config_id,
                                 int32_t splits, int32_t looks)
{
    if (config_id < -1 || (config_id >= 0 && entry_of(config_id) == nullptr)) return GSR_ERROR_INVALID_CONFIG;
    if (M < 0 || N < 0 || K < 0 || adapters < 0 || rank < 0 || splits < 0 || splits > kSplitMaxParts || workspace_bytes < 0)
        return GSR_ERROR_INVALID_VALUE;
    if (adapters == 0 || rank == 0 || M == 0 || N == 0 || K == 0)  // the product alone
        return gemm_scale_bias_act_ws(M, N, K, A, B, bias, C, alpha, activation, workspace, workspace_bytes, stream, config_id, splits);
    if (M >= kLimit || N >= kLimit || K >= kLimit || adapters >= kLimit || rank > kMaxRank) return GSR_ERROR_TOO_LARGE;
    // 32-bit byte offsets within a matrix and within one adapter
    if (M * K * 2 >= kLimit || K * N * 2 >= kLimit || M * N * 2 >= kLimit || N * rank * 2 >= kLimit || K * rank * 2 >= kLimit)
        return GSR_ERROR_TOO_LARGE;
    if (!std::isfinite(alpha)) return GSR_ERROR_INVALID_VALUE;
    if (activation != GSR_ACT_RELU && activation != GSR_ACT_GELU && activation != GSR_ACT_NONE)
        return GSR_ERROR_INVALID_VALUE;
    if (A == nullptr || B == nullptr || C == nullptr || la == nullptr || lb == nullptr || ids == nullptr ||
        workspace == nullptr)
        return GSR_ERROR_INVALID_VALUE;
    if (misaligned(A, 2) || misaligned(B, 2) || misaligned(C, 2) || misaligned(bias, 2) || misaligned(la, 2) ||
        misaligned(lb, 2) || misaligned(ids, 4) || misaligned(scales, 4) || misaligned(workspace, 16))
        return GSR_ERROR_INVALID_VALUE;
    const struct {
        const void* p;
        uint64_t bytes;
    } in[] = {{A, (uint64_t)(M * K * 2)},
              {B, (uint64_t)(K * N * 2)},
              {bias, bias ? (uint64_t)(N * 2) : 0},
              {la, (uint64_t)adapters * (uint64_t)(rank * K * 2)},
              {lb, (uint64_t)adapters * (uint64_t)(rank * N * 2)},
              {ids, (uint64_t)(M * 4)},
              {scales, scales ? (uint64_t)(adapters * 4) : 0}};
    const uint64_t cb = (uint64_t)(M * N * 2), wb = (uint64_t)workspace_bytes;
    for (const auto& i : in)
        if (overlaps(C, cb, i.p, i.bytes) || overlaps(workspace, wb, i.p, i.bytes)) return GSR_ERROR_INVALID_VALUE;
    if (overlaps(C, cb, workspace, wb)) return GSR_ERROR_INVALID_VALUE;

    Launch l = dense_launch(M, N, K);
    const Entry& e = config_id >= 0 ? *entry_of(config_id) : stand_in(l.id);
    if (e.id != l.id) l = Launch{e.id, 4, e.id == 28 ? 2 : 1};
    Problem p{};
    p.A = (const uint16_t*)A;
    p.B = (const uint16_t*)B;
    p.C = (uint16_t*)C;
    p.bias = (const uint16_t*)bias;
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.alpha = alpha;
    p.act = (int)activation;
    p.group_m = l.group_m;
    p.xcd_remap = l.xcd_remap;
    p.ksplit = 1;
    p.kchunk = (int)K;
    p.unit_a = load_unit(A, K);
    p.unit_b = load_unit(B, N);
    p.unit_c = load_unit(C, N);
    const bool vec = p.unit_a == 16 && p.unit_b == 16 && (((uintptr_t)bias & 7u) == 0);
    const int elem = elem_choice(config_id, K, (double)cdiv(M, 64) * (double)cdiv(N, 64), (double)cdiv(M, 128) * (double)cdiv(N, 128));
    const int64_t tiles_m = cdiv(M, vec ? e.bm : kElemTiles[elem].bm), tiles_n = cdiv(N, vec ? e.bn : kElemTiles[elem].bn);
    if (!grid_fits(tiles_m * tiles_n, vec ? e.threads : kElemTiles[elem].threads) || !grid_fits(cdiv(M, gsr::kShrinkRows), 512))
        return GSR_ERROR_TOO_LARGE;
    p.tiles_m = (int)tiles_m;
    p.tiles_n = (int)tiles_n;
    const int tiles = p.tiles_m * p.tiles_n;

    const Layout w = layout_of(M, K, rank);
    if (workspace_bytes < w.split) return GSR_ERROR_INVALID_VALUE;
    Split split{1, K, 0};
    if (splits > 1 && e.split == nullptr) return GSR_ERROR_INVALID_CONFIG;
    if (vec && e.split != nullptr) {
        split = dense_split(M, N, K, tiles, e.bm, e.bn, splits);
        if (split.parts > 1 && (tiles > kSplitCounters || workspace_bytes < w.split + split.partial_bytes)) {
            if (splits > 1) return GSR_ERROR_INVALID_VALUE;
            split = Split{1, K, 0};
        }
    }
    const ShrinkPlan sp = shrink_plan(M, K, adapters, rank);
    const int makers = sp.blocks * std::max(sp.parts, 1) * w.chunks * sp.slots;
    const bool shrink_vec = p.unit_a == 16 && load_unit(la, K) == 16;
    const bool shared = M <= kShrinkMixedRows && sp.parts > 0 && vec && e.shared != nullptr && shrink_vec && makers <= kSharedMakers &&
                        (split.parts == 1 || tiles <= kSharedCounters);
    // a split leaves the makers their CUs
    while (shared && splits == 0 && split.parts > 1 && tiles * split.parts + makers > 256)
        split = dense_split(M, N, K, tiles, e.bm, e.bn, split.parts - 1);
    const int st = check_device();
    if (st != GSR_SUCCESS) return st;

    uint8_t* const ws = (uint8_t*)workspace;
    ShrinkArgs a{};
    a.A = p.A;
    a.la = (const uint16_t*)la;
    a.ids = ids;
    a.scales = scales;
    a.t = (uint16_t*)(ws + w.t);
    a.t_scale = (float*)(ws + w.t_scale);
    a.M = p.M;
    a.K = p.K;
    a.adapters = (int)adapters;
    a.rank = (int)rank;
    a.chunks = w.chunks;
    a.partial = (float*)(ws + w.partial);
    a.count = (uint32_t*)ws + (shared ? kSharedCounters : 0);
    a.blocks = sp.blocks;
    a.parts = sp.parts;
    a.kchunk = sp.kchunk;
    a.slots = sp.slots;
    a.flags = (uint32_t*)ws + kSharedFlags;
    a.done = (uint32_t*)ws + kSharedDone;
    a.looks = looks < 0 ? kSharedLooks : looks;
    p.ids = ids;
    p.t = a.t;
    p.t_scale = a.t_scale;
    p.lb = (const uint16_t*)lb;
    p.adapters = (int)adapters;
    p.rank = (int)rank;
    p.chunks = w.chunks;
    p.lb_vec = load_unit(lb, rank) == 16;
    if (split.parts > 1) {
        p.ksplit = split.parts;
        p.kchunk = (int)split.kchunk;
        p.ws_count = (uint32_t*)ws;
        p.ws_part = (float*)(ws + w.split);
    }
    hipStream_t s = (hipStream_t)stream;
    if (shared)
        return status_of(e.shared(p, a, makers, makers + tiles * split.parts, s));
    hipError_t err;
    if (sp.parts > 0)
        err = launch_kernel(shrink_vec ? gsr::adapter_shrink_parts_kernel<true> : gsr::adapter_shrink_parts_kernel<false>,
                            dim3((unsigned)makers), dim3(512), s, a);
    else if (w.chunks == 1)
        err = launch_kernel(shrink_vec ? gsr::adapter_shrink_rows_kernel<true, gsr::ShrinkRows1>
                                       : gsr::adapter_shrink_rows_kernel<false, gsr::ShrinkRows1>,
                            dim3((unsigned)sp.blocks, 1, (unsigned)sp.slots), dim3(512), s, a);
    else
        err = launch_kernel(shrink_vec ? gsr::adapter_shrink_rows_kernel<true, gsr::ShrinkRows4>
                                       : gsr::adapter_shrink_rows_kernel<false, gsr::ShrinkRows4>,
                            dim3((unsigned)sp.blocks, 1, (unsigned)sp.slots), dim3(512), s, a);
    if (err != hipSuccess) return status_of(err);
    if (split.parts > 1) err = e.split(p, tiles * split.parts, s);
    else err = (vec ? e.vec : kElem[elem])(p, tiles, s);
    return status_of(err);
}

}  // extern "C"
