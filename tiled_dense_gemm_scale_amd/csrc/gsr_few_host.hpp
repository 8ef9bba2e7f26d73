// gsr_few_host.hpp -- host helpers of the few-token entry points: operands as
// ranges of bytes, and 4-bit weights.
#pragma once

#include <algorithm>
#include <cstdint>
#include <initializer_list>

#include "gsr_host.hpp"
#include "gsr_stream.hpp"

namespace gsr {
namespace host {

struct Span {
    const void* p;
    uint64_t bytes;
    uintptr_t unit;  // alignment
};

// Whether a range that has bytes is null or misaligned.
inline bool unusable(std::initializer_list<Span> spans)
{
    for (const Span& s : spans)
        if (s.bytes > 0 && (s.p == nullptr || misaligned(s.p, s.unit))) return true;
    return false;
}

inline bool clash(const Span& out, std::initializer_list<Span> others)
{
    for (const Span& s : others)
        if (overlaps(out.p, out.bytes, s.p, s.bytes)) return true;
    return false;
}

// log2 of a group size (a power of two from 32 on), or -1.
inline int group_log2(int64_t group)
{
    if (group < 32 || group > ((int64_t)1 << 30) || (group & (group - 1)) != 0) return -1;
    int l = 5;
    while (((int64_t)1 << l) < group) ++l;
    return l;
}

inline uint64_t w4_code_bytes(uint64_t matrices, int64_t K, int64_t N) { return matrices * (uint64_t)cdiv(K, 8) * (uint64_t)N * 4u; }
inline uint64_t w4_scale_count(uint64_t matrices, int64_t K, int64_t N, int64_t group)
{
    return matrices * (uint64_t)cdiv(K, group) * (uint64_t)N;
}

// Widths from here on are refused: a step's rows are addressed by 32-bit offsets.
constexpr int64_t kStreamWidth = (int64_t)1 << 22;

}  // namespace host
}  // namespace gsr
