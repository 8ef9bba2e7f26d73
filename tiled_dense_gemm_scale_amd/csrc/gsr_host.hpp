// gsr_host.hpp -- host-side pieces that the library's translation units
// share: the launch, the device check and the argument helpers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "gsr.h"

namespace gsr {
namespace host {

template <typename T>
struct as_is {
    using type = T;
};

// Whether `blocks` workgroups of `threads` threads fit a dimension of a grid,
// which holds fewer than 2^32 threads.  The runtime refuses 2^32 itself, but of
// more it runs a part and reports nothing.
inline bool grid_fits(int64_t blocks, int64_t threads) { return blocks * threads < (int64_t)1 << 32; }

// Enqueues `kernel` and returns the status of this launch alone.  The status
// comes from hipLaunchKernel's return value, not from hipGetLastError: an
// error that an earlier, unrelated HIP call left pending on the calling
// thread is neither reported as this launch's nor cleared.
template <typename... P>
hipError_t launch_kernel(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t s, typename as_is<P>::type... args)
{
    if (!grid_fits(grid.x, block.x)) return hipErrorInvalidConfiguration;
    void* argv[] = {(void*)&args...};
    return hipLaunchKernel((const void*)kernel, grid, block, argv, 0, s);
}

inline int status_of(hipError_t e)
{
    return e == hipSuccess ? GSR_SUCCESS : e == hipErrorInvalidConfiguration ? GSR_ERROR_TOO_LARGE : GSR_ERROR_LAUNCH;
}

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The widest unit (16, 8, 4 or 2 bytes) for an operand whose rows are `len`
// fp16 values long: the largest power of two up to 16 bytes dividing both the
// address and the row length in bytes, so that every row start (and the end
// of the matrix) falls on a multiple of it.
inline int load_unit(const void* p, int64_t len)
{
    int u = 16;
    while (u > 2 && ((((uintptr_t)p) % (uintptr_t)u) != 0 || ((uint64_t)len * 2u) % (uint64_t)u != 0)) u >>= 1;
    return u;
}

inline bool overlaps(const void* a, uint64_t abytes, const void* b, uint64_t bbytes)
{
    const uint64_t x = (uint64_t)(uintptr_t)a, y = (uint64_t)(uintptr_t)b;
    return abytes > 0 && bbytes > 0 && x < y + bbytes && y < x + abytes;
}

inline bool misaligned(const void* p, uintptr_t unit) { return ((uintptr_t)p & (unit - 1)) != 0; }

// GSR_SUCCESS when the current device is a gfx950 (gsr_api.hip).
__attribute__((visibility("hidden"))) int check_device();

// The selector's time of one tile of configuration `id` over K, in us
// (gsr_api.hip; 0 for an id that is no candidate of it).
__attribute__((visibility("hidden"))) double tile_time(int id, int64_t K);

// The selector's time of the whole dense product on the 128-bit path, in us
// (gsr_api.hip).
__attribute__((visibility("hidden"))) double dense_time(int64_t M, int64_t N, int64_t K);

// The dense product's launch for a shape (the tuning table, else the
// selector), and the library's K split of it on bm x bn tiles: `parts` parts
// of kchunk values of K (parts 1: none) whose fp32 partial tiles take
// `partial_bytes`.  want 0: the library's choice; else at most that many.
struct Launch {
    int id, group_m, xcd_remap;
};
struct Split {
    int parts;
    int64_t kchunk, partial_bytes;
};
__attribute__((visibility("hidden"))) Launch dense_launch(int64_t M, int64_t N, int64_t K);
__attribute__((visibility("hidden"))) Split dense_split(int64_t M, int64_t N, int64_t K, int64_t tiles, int bm, int bn, int want);
constexpr int kSplitMaxParts = 16;
constexpr int64_t kSplitCounters = 128;  // arrival counters at a workspace's start that every call leaves at zero

// The element-wise kernels of the grouped products and of those with adapters:
// 0: 64x64 with four groups of waves on K, 1: 64x64, 2: 128x128.  For a forced
// configuration id one whose sums are those of its dense form, bit for bit (1
// for the copy-wave K-split ones, 21 and 22; 0 adds up four runs of K); else by
// the number of tiles the launch has of 64x64 and of 128x128, which fill the
// chip from one per CU on (the 64x64 ones from two if K is deep).  In us, the
// three in turn, K 517: 136 tiles of 64x64 12, 15 and 22, 264 tiles 24, 17 and
// 22, 272 of 128x128 55, 33 and 25; K 10044: 136 tiles 85, 210 and 264, 264
// tiles 198, 247 and 298, 528 tiles 296, 260 and 321, 272 of 128x128 423, 431
// and 272.  Unaligned 16-byte loads go out at about one lane per clock, which
// bounds all three.
struct ElemTile {
    int bm, bn, threads;
};
constexpr ElemTile kElemTiles[3] = {{64, 64, 1024}, {64, 64, 256}, {128, 128, 256}};
constexpr int64_t kElemFull = 256, kElemDeep = 2048;
inline int elem_choice(int config_id, int64_t K, double tiles64, double tiles128)
{
    if (config_id >= 0) return config_id == 21 || config_id == 22 ? 1 : 2;
    if (tiles128 >= (double)kElemFull) return 2;
    return tiles64 > (double)(K > kElemDeep ? 2 * kElemFull : kElemFull) ? 1 : 0;
}

}  // namespace host
}  // namespace gsr
