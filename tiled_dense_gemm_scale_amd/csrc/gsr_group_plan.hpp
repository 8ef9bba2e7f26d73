// gsr_group_plan.hpp -- how the stable sort of slots by group (gsr_rows.hpp)
// cuts its slots: blocks, and the runs of a block's waves.  Plain C++, for the
// host and the kernels alike.  Counts go up to 2^31 - 1, so no place is formed
// that could lie past the last slot: a length is taken from what is left.
#pragma once

#include <cstdint>

namespace gsr {

constexpr int kGroupMax = 1024;       // groups
constexpr int kGroupWaves = 16;       // waves of a full workgroup
constexpr int kGroupSingle = 8192;    // slots one workgroup handles alone
constexpr int kGroupChunk = 2048;     // smallest block of the two-launch form
constexpr int kGroupCounts = 20000;   // counts per block from which blocks grow
constexpr int kGroupBlocks = 256;     // most blocks of it

struct GroupPlan {
    int chunk, blocks;
};

// Up to kGroupSingle slots: one block.  Above, blocks of kGroupChunk slots or,
// where the counts that each block has to read (blocks x groups) pass
// kGroupCounts, of up to four times as many; kGroupBlocks blocks at most.
constexpr GroupPlan group_plan(int64_t n, int64_t groups)
{
    if (n <= kGroupSingle) return GroupPlan{(int)n, 1};
    int64_t chunk = kGroupChunk;
    while (chunk < 4 * kGroupChunk && (n + chunk - 1) / chunk * (groups + 1) > kGroupCounts) chunk *= 2;
    const int64_t least = (((n + kGroupBlocks - 1) / kGroupBlocks) + 1023) / 1024 * 1024;
    if (chunk < least) chunk = least;
    return GroupPlan{(int)chunk, (int)((n + chunk - 1) / chunk)};
}

// `len` slots from slot `beg` on.
struct GroupSpan {
    int beg, len;
};

// Block `block` of n slots in blocks of `chunk`.
constexpr GroupSpan group_block(int n, int chunk, int block)
{
    const int beg = block * chunk;
    return GroupSpan{beg, n - beg < chunk ? n - beg : chunk};
}

// The run of wave `wave` of `waves` in a block, in whole steps of 64 slots (the
// last ones shorter or empty).
constexpr GroupSpan group_run(GroupSpan block, int wave, int waves)
{
    const int run = ((block.len + waves - 1) / waves + 63) & ~63;
    const int skip = wave * run < block.len ? wave * run : block.len;
    return GroupSpan{block.beg + skip, block.len - skip < run ? block.len - skip : run};
}

}  // namespace gsr
