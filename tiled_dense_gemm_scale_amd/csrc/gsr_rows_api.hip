// gsr_rows_api.hip -- host side of the row entry points of include/gsr.h:
// argument checks and launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gsr.h"
#include "gsr_host.hpp"
#include "gsr_rows.hpp"

namespace {

using namespace gsr::host;

using gsr::GroupPlan;
using gsr::group_plan;

constexpr int64_t kLimit = (int64_t)1 << 31;

// slots = tokens * k, or -1 (invalid) / -2 (too large)
int64_t slots_of(int64_t tokens, int64_t k)
{
    if (tokens < 0 || k < 0) return -1;
    if (tokens >= kLimit || k >= kLimit || (tokens > 0 && k > 0 && tokens > (kLimit - 1) / k)) return -2;
    return tokens * k;
}

// threads per row (a power of two up to 256), as its log2: as many as the
// row has units, so that short rows share a workgroup
int lanes_log2_of(int64_t units)
{
    int l = 0;
    while (l < 8 && ((int64_t)1 << l) < units) ++l;
    return l;
}

#define GSR_BY_UNIT(KERNEL, UNIT)                                                           \
    ((UNIT) == 16 ? gsr::KERNEL<16> : (UNIT) == 8 ? gsr::KERNEL<8> : (UNIT) == 4 ? gsr::KERNEL<4> : gsr::KERNEL<2>)

// combine_rows_backward_kernel's form for rows of `units` units.
typedef void (*rows_kernel)(gsr::RowArgs);
template <int J, int S>
rows_kernel backward16(bool stream)
{
    return stream ? gsr::combine_rows_backward_kernel<16, J, S, true> : gsr::combine_rows_backward_kernel<16, J, S, false>;
}
rows_kernel backward_kernel(int unit, int units, int k, bool stream)
{
    switch (unit) {
    case 8: return gsr::combine_rows_backward_kernel<8, 4, 4, false>;
    case 4: return gsr::combine_rows_backward_kernel<4, 4, 4, false>;
    case 2: return gsr::combine_rows_backward_kernel<2, 4, 4, false>;
    default: break;
    }
    if (units >= 512) return k <= 2 ? backward16<2, 8>(stream) : backward16<4, 8>(stream);
    if (units > 128) return backward16<4, 4>(stream);
    return units > 64 ? backward16<4, 2>(stream) : backward16<4, 1>(stream);
}

dim3 row_grid(int64_t blocks)
{
    return dim3((unsigned)std::min(blocks, gsr::kRowBlocks), (unsigned)cdiv(blocks, gsr::kRowBlocks));
}

}  // namespace

extern "C" {

int64_t gsr_group_workspace_bytes(int64_t tokens, int64_t k, int64_t groups)
{
    const int64_t n = slots_of(tokens, k);
    if (n < 0 || groups < 1 || groups > gsr::kGroupMax) return -1;
    const GroupPlan plan = group_plan(n, groups);
    return plan.blocks > 1 ? (int64_t)plan.blocks * (groups + 1) * 4 : 0;
}

int gsr_group_rows(int64_t tokens, int64_t k, int64_t groups, const void* ids, int32_t id_bytes, int32_t* offsets,
                   int32_t* rows, int32_t* positions, void* workspace, int64_t workspace_bytes, void* stream)
{
    const int64_t n = slots_of(tokens, k);
    if (n == -1 || groups < 1 || (id_bytes != 4 && id_bytes != 8) || workspace_bytes < 0) return GSR_ERROR_INVALID_VALUE;
    if (n == -2 || groups > gsr::kGroupMax) return GSR_ERROR_TOO_LARGE;
    if (offsets == nullptr || misaligned(offsets, 4)) return GSR_ERROR_INVALID_VALUE;
    const uint64_t idb = (uint64_t)n * (uint64_t)id_bytes, nb = (uint64_t)n * 4u, ob = (uint64_t)(groups + 1) * 4u;
    const int64_t need = gsr_group_workspace_bytes(tokens, k, groups);
    const uint64_t wb = (uint64_t)workspace_bytes;
    if (n > 0) {
        if (ids == nullptr || rows == nullptr || positions == nullptr || misaligned(ids, (uintptr_t)id_bytes) ||
            misaligned(rows, 4) || misaligned(positions, 4))
            return GSR_ERROR_INVALID_VALUE;
        if (overlaps(rows, nb, ids, idb) || overlaps(positions, nb, ids, idb) || overlaps(rows, nb, positions, nb) ||
            overlaps(offsets, ob, ids, idb) || overlaps(offsets, ob, rows, nb) || overlaps(offsets, ob, positions, nb))
            return GSR_ERROR_INVALID_VALUE;
    }
    if (need > 0) {
        if (workspace == nullptr || misaligned(workspace, 16) || workspace_bytes < need) return GSR_ERROR_INVALID_VALUE;
        if (overlaps(workspace, wb, ids, idb) || overlaps(workspace, wb, rows, nb) ||
            overlaps(workspace, wb, positions, nb) || overlaps(workspace, wb, offsets, ob))
            return GSR_ERROR_INVALID_VALUE;
    }
    const int st = check_device();
    if (st != GSR_SUCCESS) return st;
    const GroupPlan plan = group_plan(n, groups);
    gsr::GroupArgs g;
    g.ids = ids;
    g.offsets = offsets;
    g.rows = rows;
    g.positions = positions;
    g.hist = plan.blocks > 1 ? (uint32_t*)workspace : nullptr;
    g.n = (int32_t)n;
    g.k = (int32_t)std::max<int64_t>(k, 1);
    g.groups = (int32_t)groups;
    g.chunk = plan.chunk;
    g.blocks = plan.blocks;
    g.bits = 0;
    while ((groups >> g.bits) != 0) ++g.bits;
    hipStream_t s = (hipStream_t)stream;
    const bool wide = id_bytes == 8;
    if (plan.blocks > 1) {
        const hipError_t err = launch_kernel(wide ? gsr::group_count_kernel<int64_t> : gsr::group_count_kernel<int32_t>,
                                             dim3((unsigned)plan.blocks), dim3(1024), s, g);
        if (err != hipSuccess) return status_of(err);
    }
    const int waves = (int)std::min<int64_t>(gsr::kGroupWaves, std::max<int64_t>(1, cdiv(plan.chunk, 64)));
    return status_of(launch_kernel(wide ? gsr::group_place_kernel<int64_t> : gsr::group_place_kernel<int32_t>,
                                   dim3((unsigned)plan.blocks), dim3((unsigned)(64 * waves)), s, g));
}

int gsr_gather_rows(int64_t rows_out, int64_t rows_in, int64_t width, const void* x, const int32_t* rows, void* out,
                    void* stream)
{
    if (rows_out < 0 || rows_in < 0 || width < 0) return GSR_ERROR_INVALID_VALUE;
    if (rows_out >= kLimit || rows_in >= kLimit || width >= kLimit / 2) return GSR_ERROR_TOO_LARGE;
    if (rows_out == 0 || width == 0) return GSR_SUCCESS;
    const uint64_t xb = (uint64_t)rows_in * (uint64_t)width * 2u, outb = (uint64_t)rows_out * (uint64_t)width * 2u;
    if (rows == nullptr || out == nullptr || (rows_in > 0 && x == nullptr) || misaligned(x, 2) || misaligned(out, 2) ||
        misaligned(rows, 4))
        return GSR_ERROR_INVALID_VALUE;
    if (overlaps(out, outb, x, xb) || overlaps(out, outb, rows, (uint64_t)rows_out * 4u)) return GSR_ERROR_INVALID_VALUE;
    const int st = check_device();
    if (st != GSR_SUCCESS) return st;
    const int unit = std::min(load_unit(x, width), load_unit(out, width));
    gsr::RowArgs r{};
    r.x = (const uint16_t*)x;
    r.index = rows;
    r.out = (uint16_t*)out;
    r.T = (int32_t)rows_in;
    r.P = (int32_t)rows_out;
    r.units = (int32_t)(width * 2 / unit);
    r.lanes_log2 = lanes_log2_of(r.units);
    return status_of(launch_kernel(GSR_BY_UNIT(gather_rows_kernel, unit),
                                   row_grid(cdiv(rows_out, 256 >> r.lanes_log2)), dim3(256), (hipStream_t)stream, r));
}

int gsr_combine_rows(int64_t tokens, int64_t k, int64_t rows_in, int64_t width, const void* y, const int32_t* positions,
                     const float* weights, void* out, void* stream)
{
    const int64_t n = slots_of(tokens, k);
    if (n == -1 || rows_in < 0 || width < 0) return GSR_ERROR_INVALID_VALUE;
    if (n == -2 || rows_in >= kLimit || width >= kLimit / 2) return GSR_ERROR_TOO_LARGE;
    if (tokens == 0 || width == 0) return GSR_SUCCESS;
    const uint64_t yb = (uint64_t)rows_in * (uint64_t)width * 2u, outb = (uint64_t)tokens * (uint64_t)width * 2u;
    if (out == nullptr || misaligned(out, 2) || misaligned(y, 2) || (rows_in > 0 && y == nullptr) ||
        (n > 0 && positions == nullptr) || misaligned(positions, 4) || misaligned(weights, 4))
        return GSR_ERROR_INVALID_VALUE;
    if (overlaps(out, outb, y, yb) || overlaps(out, outb, positions, (uint64_t)n * 4u) ||
        (weights != nullptr && overlaps(out, outb, weights, (uint64_t)n * 4u)))
        return GSR_ERROR_INVALID_VALUE;
    const int st = check_device();
    if (st != GSR_SUCCESS) return st;
    const int unit = std::min(load_unit(y, width), load_unit(out, width));
    gsr::RowArgs r{};
    r.x = (const uint16_t*)y;
    r.index = positions;
    r.weights = weights;
    r.out = (uint16_t*)out;
    r.T = (int32_t)tokens;
    r.P = (int32_t)rows_in;
    r.k = (int32_t)k;
    r.units = (int32_t)(width * 2 / unit);
    r.lanes_log2 = lanes_log2_of(r.units);
    return status_of(launch_kernel(GSR_BY_UNIT(combine_rows_kernel, unit),
                                   row_grid(cdiv(tokens, 256 >> r.lanes_log2)), dim3(256), (hipStream_t)stream, r));
}

int gsr_combine_rows_backward(int64_t tokens, int64_t k, int64_t rows_in, int64_t width, const void* dout, const void* y,
                              const int32_t* positions, const float* weights, const int32_t* rows, void* dy,
                              float* dweights, void* stream)
{
    const int64_t n = slots_of(tokens, k);
    if (n == -1 || rows_in < 0 || width < 0) return GSR_ERROR_INVALID_VALUE;
    if (n == -2 || rows_in >= kLimit || width >= kLimit / 2) return GSR_ERROR_TOO_LARGE;
    if ((dweights != nullptr) != (weights != nullptr)) return GSR_ERROR_INVALID_VALUE;
    const uint64_t rb = (uint64_t)rows_in * (uint64_t)width * 2u, db = (uint64_t)tokens * (uint64_t)width * 2u;
    const uint64_t nb = (uint64_t)n * 4u, ib = (uint64_t)rows_in * 4u;
    if (misaligned(dout, 2) || misaligned(y, 2) || misaligned(dy, 2) || misaligned(positions, 4) ||
        misaligned(weights, 4) || misaligned(rows, 4) || misaligned(dweights, 4))
        return GSR_ERROR_INVALID_VALUE;
    if ((n > 0 && positions == nullptr) || (rows_in > 0 && rows == nullptr) || (db > 0 && dout == nullptr) ||
        (rb > 0 && (dy == nullptr || (weights != nullptr && y == nullptr))))
        return GSR_ERROR_INVALID_VALUE;
    if (overlaps(dy, rb, dout, db) || (y != nullptr && overlaps(dy, rb, y, rb)) || overlaps(dy, rb, positions, nb) ||
        overlaps(dy, rb, rows, ib) || (weights != nullptr && overlaps(dy, rb, weights, nb)))
        return GSR_ERROR_INVALID_VALUE;
    if (dweights != nullptr &&
        (overlaps(dweights, nb, dout, db) || overlaps(dweights, nb, y, rb) || overlaps(dweights, nb, positions, nb) ||
         overlaps(dweights, nb, weights, nb) || overlaps(dweights, nb, rows, ib) || overlaps(dweights, nb, dy, rb)))
        return GSR_ERROR_INVALID_VALUE;
    if ((rows_in == 0 || width == 0) && (n == 0 || dweights == nullptr)) return GSR_SUCCESS;
    const int st = check_device();
    if (st != GSR_SUCCESS) return st;
    const int unit = width == 0 ? 16 : std::min({load_unit(dout, width), weights ? load_unit(y, width) : 16, load_unit(dy, width)});
    gsr::RowArgs r{};
    r.x = (const uint16_t*)dout;
    r.y = (const uint16_t*)y;
    r.index = rows;
    r.positions = positions;
    r.weights = weights;
    r.out = (uint16_t*)dy;
    r.dweights = dweights;
    r.T = (int32_t)tokens;
    r.P = (int32_t)rows_in;
    r.k = (int32_t)k;
    r.units = (int32_t)(width * 2 / unit);
    const int64_t waves = std::max<int64_t>({tokens, cdiv(rows_in, 64), 1});
    return status_of(launch_kernel(backward_kernel(unit, r.units, r.k, weights != nullptr && rb >= (uint64_t)gsr::kStreamBytes),
                                   row_grid(cdiv(waves, 4)), dim3(256), (hipStream_t)stream, r));
}

}  // extern "C"
