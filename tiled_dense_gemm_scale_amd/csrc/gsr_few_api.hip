// gsr_few_api.hip -- host side of the few-token layer of routed experts:
// argument checks and its two launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gsr.h"
#include "gsr_few.hpp"
#include "gsr_few_host.hpp"

namespace {

using namespace gsr::host;

bool bad_sizes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t F, int64_t O)
{
    return T < 0 || k < 0 || E < 0 || H < 0 || F < 0 || O < 0;
}

bool large_sizes(int64_t T, int64_t k, int64_t E, int64_t H, int64_t F, int64_t O)
{
    return T > gsr::kFewTokens || k > gsr::kFewSlots || T * k > gsr::kFewSlots || E > gsr::kFewExperts ||
           H >= kStreamWidth || F >= kStreamWidth || O >= kStreamWidth || T * k * (cdiv(F, 8) * 8) >= ((int64_t)1 << 29);
}

struct Plan {
    int blocks_up, grid_up, waves_log2, blocks, groups;
    int64_t hidden_wide, part_wide, hidden_bytes, bytes;
};

// Workgroups of a launch: one to a CU, which is what their registers allow.
constexpr int64_t kFewGrid = 256;

Plan plan_of(bool w4, int64_t T, int64_t k, int64_t E, int64_t F, int64_t O)
{
    const int64_t CB = w4 ? gsr::W4Stream<1, true, false>::CB : gsr::HalfStream<true, false>::CB;
    Plan g;
    // tiles at most: one per expert that is hit, and one for each 16 slots more
    const int64_t slots = T * k, most = std::max<int64_t>(1, std::min(slots, std::min(E, slots) + slots / gsr::kFewRows));
    g.blocks_up = (int)cdiv(F, CB);
    // as many workgroups as items, up to a power of two of them
    for (g.grid_up = 1, g.waves_log2 = 3; g.grid_up < kFewGrid && g.grid_up < g.blocks_up * most; g.grid_up *= 2) ++g.waves_log2;
    g.blocks = (int)cdiv(O, CB);
    // a job is a tile and 128 rows of F at least, eight to a workgroup; at most
    // 128 blocks have more than one workgroup, and so a counter each
    g.groups = (int)std::max<int64_t>(1, std::min({(int64_t)16, kFewGrid / std::max(g.blocks, 1), cdiv(most * cdiv(F, 128), gsr::kStreamWaves)}));
    g.hidden_wide = cdiv(F, 8) * 8;
    g.part_wide = g.blocks * CB;
    g.hidden_bytes = slots * g.hidden_wide * 4;  // two halves
    g.bytes = gsr::kMeetBytes + g.hidden_bytes + (g.groups > 1 ? g.groups * T * g.part_wide * 4 : 0);
    return g;
}

// The ranges of `E` matrices of K x N; false where a pointer or the group is bad.
struct Ranges {
    Span data, scales, zeros, bias;
};
bool ranges_of(const gsr_weights* w, int64_t E, int64_t K, int64_t N, Ranges& r)
{
    const uint64_t all = (uint64_t)E * (uint64_t)K * (uint64_t)N;
    r.bias = Span{w->bias, w->bias ? (uint64_t)E * (uint64_t)N * 2u : 0u, 2};
    if (w->group == 0) {
        if (w->scales != nullptr || w->zeros != nullptr) return false;
        r.data = Span{w->data, all * 2u, 2};
        r.scales = r.zeros = Span{nullptr, 0, 1};
    } else {
        if (group_log2(w->group) < 0) return false;
        const uint64_t sc = w4_scale_count((uint64_t)E, K, N, w->group);
        r.data = Span{w->data, w4_code_bytes((uint64_t)E, K, N), 4};
        r.scales = Span{w->scales, 2u * sc, 2};
        r.zeros = Span{w->zeros, w->zeros ? sc : 0u, 1};
    }
    return !unusable({r.data, r.scales, r.zeros, r.bias});
}

gsr::FewWeights weights_of(const gsr_weights* w)
{
    return gsr::FewWeights{w->data, (const uint16_t*)w->scales, w->zeros, (const uint16_t*)w->bias,
                           w->group ? group_log2(w->group) : 0};
}

typedef void (*few_kernel)(gsr::FewArgs);
struct Kernels {
    few_kernel up, gated, down;
};
template <int FORM, bool DW>
Kernels kernels_of()
{
    constexpr bool DD = DW || FORM != gsr::kFewHalf;  // its rows of A are h's, which lie on dwords
    return Kernels{gsr::few_up_kernel<FORM, DW, false>, gsr::few_up_kernel<FORM, DW, true>, gsr::few_down_kernel<FORM, DD>};
}
// For matrices of `w` (and `w2`, or null) of N columns, and rows of A of K values.
Kernels kernels_at(const gsr_weights* w, const gsr_weights* w2, const void* a, int64_t K, int64_t N)
{
    bool dwords = K % 2 == 0 && !misaligned(a, 4);
    if (w->group == 0) dwords = dwords && N % 2 == 0 && !misaligned(w->data, 4) && (w2 == nullptr || !misaligned(w2->data, 4));
    switch (w->group) {
    case 0: return dwords ? kernels_of<gsr::kFewHalf, true>() : kernels_of<gsr::kFewHalf, false>();
    case 32: return dwords ? kernels_of<gsr::kFewW4x1, true>() : kernels_of<gsr::kFewW4x1, false>();
    case 64: return dwords ? kernels_of<gsr::kFewW4x2, true>() : kernels_of<gsr::kFewW4x2, false>();
    default: return dwords ? kernels_of<gsr::kFewW4x4, true>() : kernels_of<gsr::kFewW4x4, false>();
    }
}

}  // namespace

extern "C" {

int64_t gsr_expert_few_workspace_bytes(int64_t tokens, int64_t k, int64_t experts, int64_t F, int64_t O)
{
    if (bad_sizes(tokens, k, experts, 0, F, O) || large_sizes(tokens, k, experts, 0, F, O)) return -1;
    return std::max(plan_of(false, tokens, k, experts, F, O).bytes, plan_of(true, tokens, k, experts, F, O).bytes);
}

int gsr_expert_mlp_few(int64_t tokens, int64_t k, int64_t experts, int64_t H, int64_t F, int64_t O, const void* x,
                       const void* ids, int32_t id_bytes, const float* weights, const gsr_weights* up,
                       const gsr_weights* gate, const gsr_weights* down, int32_t activation, void* out, void* workspace,
                       int64_t workspace_bytes, void* stream)
{
    if (bad_sizes(tokens, k, experts, H, F, O) || (id_bytes != 4 && id_bytes != 8) || workspace_bytes < 0 ||
        up == nullptr || down == nullptr || activation < GSR_ACT_RELU || activation > GSR_ACT_SILU)
        return GSR_ERROR_INVALID_VALUE;
    if (large_sizes(tokens, k, experts, H, F, O)) return GSR_ERROR_TOO_LARGE;
    const bool w4 = up->group != 0;
    if ((down->group != 0) != w4 || (gate != nullptr && gate->group != up->group)) return GSR_ERROR_INVALID_VALUE;
    if (tokens == 0 || O == 0) return GSR_SUCCESS;
    Ranges ru, rg{}, rd;
    if (!ranges_of(up, experts, H, F, ru) || (gate != nullptr && !ranges_of(gate, experts, H, F, rg)) ||
        !ranges_of(down, experts, F, O, rd))
        return GSR_ERROR_INVALID_VALUE;
    const uint64_t slots = (uint64_t)tokens * (uint64_t)k;
    const Span sx{x, (uint64_t)tokens * (uint64_t)H * 2u, 2}, si{ids, slots * (uint64_t)id_bytes, (uintptr_t)id_bytes},
        sw{weights, weights ? slots * 4u : 0u, 4}, so{out, (uint64_t)tokens * (uint64_t)O * 2u, 2},
        ws{workspace, (uint64_t)workspace_bytes, 16};
    const Plan g = plan_of(w4, tokens, k, experts, F, O);
    if (unusable({sx, si, sw, so, ws}) || workspace_bytes < g.bytes) return GSR_ERROR_INVALID_VALUE;
    for (const Span& o : {so, ws})
        if (clash(o, {sx, si, sw, ru.data, ru.scales, ru.zeros, ru.bias, rg.data, rg.scales, rg.zeros, rg.bias, rd.data,
                      rd.scales, rd.zeros, rd.bias}))
            return GSR_ERROR_INVALID_VALUE;
    if (clash(so, {ws})) return GSR_ERROR_INVALID_VALUE;
    const int st = check_device();
    if (st != GSR_SUCCESS) return st;

    gsr::FewArgs p{};
    p.x = (const uint16_t*)x;
    p.ids = ids;
    p.weights = weights;
    p.up = weights_of(up);
    if (gate != nullptr) p.gate = weights_of(gate);
    p.down = weights_of(down);
    p.out = (uint16_t*)out;
    p.count = (uint32_t*)workspace;
    p.hidden = (uint16_t*)((uint8_t*)workspace + gsr::kMeetBytes);
    p.part = (float*)((uint8_t*)workspace + gsr::kMeetBytes + g.hidden_bytes);
    p.T = (int)tokens;
    p.k = (int)k;
    p.slots = (int)slots;
    p.experts = (int)experts;
    p.H = (int)H;
    p.F = (int)F;
    p.O = (int)O;
    p.hidden_wide = (int)g.hidden_wide;
    p.part_wide = (int)g.part_wide;
    p.act = activation;
    p.wide_ids = id_bytes == 8;
    p.blocks_up = g.blocks_up;
    p.waves_log2 = g.waves_log2;
    p.blocks = g.blocks;
    p.groups = g.groups;
    hipStream_t s = (hipStream_t)stream;
    if (F > 0 && slots > 0) {
        const Kernels f = kernels_at(up, gate, x, H, F);
        const hipError_t err = launch_kernel(gate != nullptr ? f.gated : f.up, dim3((unsigned)g.grid_up), dim3(gsr::kStreamThreads), s, p);
        if (err != hipSuccess) return status_of(err);
    }
    return status_of(launch_kernel(kernels_at(down, nullptr, p.hidden, p.hidden_wide, O).down, dim3((unsigned)(g.blocks * g.groups)), dim3(gsr::kStreamThreads), s, p));
}

}  // extern "C"
