// gsr_few.hpp -- a whole layer of routed experts for a few tokens, in two
// launches:
//
//     h[s, f] = act(x[t] up[e] + bias_up[e])                (slot s = t k + j, e = ids[s])
//     h[s, f] = act(x[t] gate[e] + bias_gate[e]) (x[t] up[e] + bias_up[e])    with a gate
//     out[t, o] = sum_j weights[s] (h[s] down[e] + bias_down[e])
//
// With a few tokens the layer is bound by the bytes of the weights that the
// choices hit, so there is no sort and no gather in front: every wave finds the
// experts that are hit, and its expert's slots, from the ids itself, without a
// barrier, and streams its columns of that expert's matrix past the slots' rows
// (gsr_stream.hpp).  How many experts are hit is known on the device only, so
// the grid is fixed and the waves share out what there is.
//  * up: an item is an expert and a block of columns; 1, 2, 4 or 8 waves of a
//    workgroup split its H, whichever leaves the fewest idle.
//  * down: a workgroup has a block of columns; its waves take jobs, an expert
//    and a part of F, weigh their rows and add them per token in LDS, in order
//    of the experts.  The workgroups of a block meet in the workspace and the
//    last one adds their sums in order, so equal inputs give equal bits.
// h is rounded to fp16 between the launches, as the fp16 matrix cores take it.
#pragma once

#include "gsr_stream.hpp"
#include "gsr_w4.hpp"

namespace gsr {

constexpr int kFewTokens = 64, kFewSlots = 1024, kFewExperts = 1024;

// One of the layer's matrices: `experts` of them, in fp16 (data; scales null) or
// in 4 bits, and a bias each or null.
struct FewWeights {
    const void* data;
    const uint16_t* scales;
    const uint8_t* zeros;
    const uint16_t* bias;
    int glog2;
};

struct FewArgs {
    const uint16_t* x;     // T x H
    const void* ids;       // T x k
    const float* weights;  // T x k, or null (ones)
    FewWeights up, gate, down;
    uint16_t* out;         // T x O
    uint16_t* hidden;      // slots x hidden_wide
    float* part;           // groups x T x part_wide
    uint32_t* count;
    int T, k, slots, experts, H, F, O;
    int hidden_wide, part_wide;
    int act;
    bool wide_ids;
    int blocks_up;         // column blocks of the first launch
    int waves_log2;        // its waves (a power of two)
    int blocks, groups;    // of the second: column blocks, workgroups to each
    int per;               // column blocks per counter
};

// The stream of a form of weights: fp16, 4 bits with groups of 32, 64, and 128 or
// more rows.  DW: every row of fp16 weights and of A starts on a dword.
enum : int { kFewHalf = 0, kFewW4x1 = 1, kFewW4x2 = 2, kFewW4x4 = 3 };
template <int FORM, int MT, bool DW>
struct FewStream : W4Stream<MT, FORM == kFewW4x1 ? 1 : FORM == kFewW4x2 ? 2 : 4, DW> {
    __device__ static __forceinline__ W4Matrix matrix(const FewWeights& w, int e, int K, int N)
    {
        const size_t words = (size_t)((K + 7) / 8) * N, groups = (size_t)((((int64_t)K - 1) >> w.glog2) + 1) * N;
        return W4Matrix{(const uint32_t*)w.data + e * words, w.scales + e * groups, w.zeros ? w.zeros + e * groups : nullptr,
                        w.glog2};
    }
};
template <int MT, bool DW>
struct FewStream<kFewHalf, MT, DW> : HalfStream<MT, DW> {
    __device__ static __forceinline__ HalfMatrix matrix(const FewWeights& w, int e, int K, int N)
    {
        return HalfMatrix{(const uint16_t*)w.data + (size_t)e * K * N};
    }
};

// What a wave finds out from the ids, without the others.
constexpr int kFewRows = 16;  // rows of a tile
struct FewWave {
    uint32_t hit[kFewExperts / 32];
    int16_t slot[2 * kFewRows];  // the rows in hand: slots of the wave's expert, ascending
};

__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Fills key (a slot's expert, -1: none; every wave writes the same values) and
// the wave's set of experts; returns how many are hit.
__device__ __forceinline__ int few_keys(FewWave& s, int16_t* key, const FewArgs& p)
{
    const int lane = threadIdx.x & 63, words = (p.experts + 31) / 32;
    if (lane < kFewExperts / 32) s.hit[lane] = 0u;
    wave_fence();
    for (int i = lane; i < p.slots; i += kWave) {
        const int64_t id = p.wide_ids ? ((const int64_t*)p.ids)[i] : (int64_t)((const int32_t*)p.ids)[i];
        const bool in = id >= 0 && id < p.experts;
        key[i] = in ? (int16_t)id : (int16_t)-1;
        if (in) atomicOr(&s.hit[(int)id >> 5], 1u << ((int)id & 31));
    }
    wave_fence();
    const uint32_t w = s.hit[lane & (kFewExperts / 32 - 1)];
    int n = 0;
    for (int i = 0; i < words; ++i) n += __popc(__builtin_amdgcn_readlane(w, i));
    return n;
}

// The d-th expert that is hit, ascending (d below their number).
__device__ __forceinline__ int few_expert(const FewWave& s, int d)
{
    const uint32_t w = s.hit[threadIdx.x & (kFewExperts / 32 - 1)];
    int i = 0;
    uint32_t bits;
    for (;; ++i) {
        bits = __builtin_amdgcn_readlane(w, i);
        const int n = __popc(bits);
        if (d < n) break;
        d -= n;
    }
    for (; d > 0; --d) bits &= bits - 1u;
    return 32 * i + __ffs((int)bits) - 1;
}

// The slots m0 .. m0 + 2 kFewRows - 1 of expert e into s.slot; how many it has in all.
__device__ __forceinline__ int few_rows(FewWave& s, const int16_t* key, int slots, int e, int m0)
{
    const int lane = threadIdx.x & 63;
    int n = 0;
    wave_fence();
    for (int i0 = 0; i0 < slots; i0 += kWave) {
        const bool mine = i0 + lane < slots && key[i0 + lane] == e;
        const uint64_t m = __ballot(mine);
        const int at = n + __popcll(m & ((1ull << lane) - 1ull)) - m0;
        if (mine && at >= 0 && at < 2 * kFewRows) s.slot[at] = (int16_t)(i0 + lane);
        n += __popcll(m);
    }
    wave_fence();
    return __builtin_amdgcn_readfirstlane(n);
}

// acc of MT tiles from `left` rows: streams one tile where that is all.
template <int FORM, int MT, bool DW>
__device__ __forceinline__ void few_stream(const FewWeights& w, int e, int K, int N, int n0, const StreamRows<MT, DW>& rows, int left,
                                           int u0, int u1, typename FewStream<FORM, MT, DW>::Sums& acc)
{
    acc.clear();
    if (MT > 1 && left <= kFewRows) {
        using S = FewStream<FORM, 1, DW>;
        typename S::Sums sums;
        sums.clear();
        S::run(S::matrix(w, e, K, N), K, N, n0, StreamRows<1, DW>(rows), u0, u1, sums);
#pragma unroll
        for (int j = 0; j < S::CPL; ++j) acc.v[j][0] = sums.v[j][0];
    } else {
        using S = FewStream<FORM, MT, DW>;
        S::run(S::matrix(w, e, K, N), K, N, n0, rows, u0, u1, acc);
    }
}

// log2 of how many of a workgroup's waves split an item's K of `units` (2^least
// at least): the count for which the rounds of `waves` (a power of two) waves,
// each `fixed` units longer than its share of K, are shortest.
__device__ __forceinline__ int few_split(int items, int waves_log2, int units, int fixed, int least)
{
    int best = least, shortest = INT32_MAX;
    for (int s = least; s <= 3; ++s) {
        const int rounds = (int)((((int64_t)items << s) + (1 << waves_log2) - 1) >> waves_log2);
        const int share = units >> (s - least);  // of 2^22 / 32 units at most; rounded down, as it is an estimate
        const int64_t cost = (int64_t)rounds * (share + fixed);
        if (cost < shortest) {
            shortest = (int)cost;
            best = s;
        }
    }
    return best;
}

// h of the experts' slots.  With a gate the first half of an item's waves
// streams the gate and the second half up.
template <int FORM, int MT, bool DW, bool GATED>
__global__ void __launch_bounds__(kStreamThreads, 2) few_up_kernel(FewArgs p)
{
    using S = FewStream<FORM, MT, DW>;
    constexpr int CPL = S::CPL, CB = S::CB, UNIT = S::UNIT, SETS = GATED ? 2 : 1;
    __shared__ __attribute__((aligned(16))) float lds[kStreamWaves * 16 * CB];
    __shared__ FewWave waves[kStreamWaves];
    __shared__ int16_t key[kFewSlots];
    __shared__ int experts[kStreamWaves], counts[kStreamWaves];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 15;
    FewWave& mine = waves[wave];
    const int hits = few_keys(mine, key, p), items = hits * p.blocks_up, units = (p.H + UNIT - 1) / UNIT;
    const int kl = few_split(items, p.waves_log2, units, 256 / UNIT, SETS - 1), kg = 1 << kl, cg = kStreamWaves >> kl;
    const int turn = wave & (kg - 1), half = kg / SETS;  // the waves of one matrix
    const FewWeights& w = GATED && turn < half ? p.gate : p.up;
    const int u0 = units * (turn & (half - 1)) / half, u1 = units * ((turn & (half - 1)) + 1) / half;

    for (int first = blockIdx.x * cg; first < items; first += gridDim.x * cg) {
        const int item = first + (wave >> kl), d = item / p.blocks_up, n0 = (item - d * p.blocks_up) * CB;
        const bool have = item < items;
        const int e = have ? few_expert(mine, d) : -1;
        int count = 0, m0 = 0;
        do {
            if (have) count = few_rows(mine, key, p.slots, e, m0);
            typename S::Sums acc;
            if (m0 < count) {
                typename S::Rows rows(p.x, (uint64_t)p.T * (uint32_t)p.H * 2u);
#pragma unroll
                for (int t = 0; t < MT; ++t) rows.row(t, (uint32_t)mine.slot[min(16 * t + l, count - 1 - m0)] / (uint32_t)p.k * (uint32_t)p.H);
                few_stream<FORM, MT, DW>(w, e, p.H, p.F, n0, rows, count - m0, u0, u1, acc);
            }
            if ((threadIdx.x & 63) == 0) {
                experts[wave] = e;
                counts[wave] = count;
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                __syncthreads();
                if (m0 + 16 * t < count) stream_put<CPL, MT>(lds + wave * 16 * CB, acc, t);
                __syncthreads();
#pragma unroll 1
                for (int c = 0; c < cg; ++c) {
                    const int at_n0 = (first + c) % p.blocks_up * CB, ex = experts[c << kl], here = min(16, counts[c << kl] - m0 - 16 * t);
                    const float* slices = lds + (c << kl) * 16 * CB;
#pragma unroll 1
                    for (int u = threadIdx.x; u < here * CB; u += kStreamThreads) {
                        const int m = u / CB, at = u % CB, col = stream_position<CPL>(at_n0, at, p.F);
                        if (col < 0) continue;
                        const size_t b = (size_t)ex * p.F + col;
                        float v = stream_sum<CPL>(slices + (kg - half) * 16 * CB, half, m, at) + (p.up.bias ? half_at(p.up.bias + b) : 0.0f);
                        if constexpr (GATED) {
                            const float g = stream_sum<CPL>(slices, half, m, at) + (p.gate.bias ? half_at(p.gate.bias + b) : 0.0f);
                            v *= stream_activate(g, p.act);
                        } else {
                            v = stream_activate(v, p.act);
                        }
                        p.hidden[(size_t)waves[c << kl].slot[16 * t + m] * p.hidden_wide + col] = to_half(v);
                    }
                }
            }
            m0 += 16 * MT;
        } while (__syncthreads_or(m0 < count));
    }
}

// out of a block of columns.  T is at most 16 NT.  A tile's rows are weighed and
// added to their tokens' sums in LDS: per token a mask of the waves that have
// rows of it (two masks in turn, one cleared while the other is read), and its
// first row in each; the rows of a token lie behind each other.
template <int FORM, int MT, int NT, bool DW>
__global__ void __launch_bounds__(kStreamThreads, 2) few_down_kernel(FewArgs p)
{
    using S = FewStream<FORM, MT, DW>;
    constexpr int CPL = S::CPL, CB = S::CB, UNIT = S::UNIT, TOKENS = 16 * NT;
    __shared__ __attribute__((aligned(16))) float lds[kStreamWaves * 16 * CB];
    __shared__ float sums[TOKENS * CB];
    __shared__ FewWave waves[kStreamWaves];
    __shared__ int16_t key[kFewSlots];
    __shared__ uint32_t mask[2][TOKENS];
    __shared__ int8_t row_of[kStreamWaves][TOKENS], token_of[kStreamWaves][kFewRows + 1];
    __shared__ float weight_of[kStreamWaves][kFewRows];
    __shared__ int bias_of[kStreamWaves];  // the expert whose bias a wave's rows get, or -1
    __shared__ int flag;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 15;
    const int nb = blockIdx.x / p.groups, group = blockIdx.x - nb * p.groups, n0 = nb * CB;
    FewWave& mine = waves[wave];
    const int hits = few_keys(mine, key, p), units = (p.F + UNIT - 1) / UNIT;
    // every wave of the block has a job where that leaves each 256 rows of F
    const int parts = max(1, min(p.groups * kStreamWaves / max(hits, 1), units * UNIT / 256)), jobs = hits * parts;
    const int j0 = jobs * group / p.groups, j1 = jobs * (group + 1) / p.groups;
    for (int i = tid; i < p.T * CB; i += kStreamThreads) sums[i] = 0.0f;
    if (tid < TOKENS) mask[0][tid] = mask[1][tid] = 0u;

    int turn = 0;
    for (int first = j0; first < j1; first += kStreamWaves) {
        const int job = first + wave, d = job / parts, part = job - d * parts;
        const bool have = job < j1;
        const int e = have ? few_expert(mine, d) : -1;
        const int u0 = (int)((int64_t)units * part / parts), u1 = (int)((int64_t)units * (part + 1) / parts);
        int count = 0, m0 = 0;
        do {
            if (have) count = few_rows(mine, key, p.slots, e, m0);
            typename S::Sums acc;
            if (m0 < count) {
                typename S::Rows rows(p.hidden, (uint64_t)p.slots * (uint32_t)p.hidden_wide * 2u);
#pragma unroll
                for (int t = 0; t < MT; ++t) rows.row(t, (uint32_t)mine.slot[min(16 * t + l, count - 1 - m0)] * (uint32_t)p.hidden_wide);
                few_stream<FORM, MT, DW>(p.down, e, p.F, p.O, n0, rows, count - m0, u0, u1, acc);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                __syncthreads();
                const int here = min(16, count - m0 - 16 * t);
                if (here > 0) {
                    if (lane < here) {
                        const int slot = mine.slot[16 * t + lane], token = slot / p.k;
                        token_of[wave][lane] = (int8_t)token;
                        weight_of[wave][lane] = p.weights ? p.weights[slot] : 1.0f;
                        if (lane == 0 || mine.slot[16 * t + lane - 1] / p.k != token) row_of[wave][token] = (int8_t)lane;
                        atomicOr(&mask[turn][token], 1u << wave);
                    }
                    if (lane == 0) {
                        token_of[wave][here] = -1;
                        bias_of[wave] = p.down.bias && part == 0 ? e : -1;
                    }
                    stream_put<CPL, MT>(lds + wave * 16 * CB, acc, t);
                }
                __syncthreads();
#pragma unroll 1
                for (int u = tid; u < p.T * CB; u += kStreamThreads) {
                    const int token = u / CB, at = u % CB;
                    uint32_t from = mask[turn][token];
                    if (from == 0u) continue;
                    const int col = stream_position<CPL>(n0, at, p.O);
                    float s = sums[u];
                    do {
                        const int w = __ffs((int)from) - 1;
                        from &= from - 1u;
                        const float b = bias_of[w] >= 0 && col >= 0 ? half_at(p.down.bias + (size_t)bias_of[w] * p.O + col) : 0.0f;
                        int r = row_of[w][token];
                        do s = fmaf(weight_of[w][r], lds[(w * 16 + r) * CB + at] + b, s);
                        while (token_of[w][++r] == token);
                    } while (from != 0u);
                    sums[u] = s;
                }
                turn ^= 1;
                if (tid < TOKENS) mask[turn][tid] = 0u;  // read before the barriers above
            }
            m0 += 16 * MT;
        } while (__syncthreads_or(m0 < count));
    }
    __syncthreads();

    auto finish = [&](int u, int n_block, float s) {
        const int col = stream_position<CPL>(n_block, u % CB, p.O);
        if (col >= 0) p.out[(size_t)(u / CB) * p.O + col] = to_half(s);
    };
    for (int u = tid; u < p.T * CB; u += kStreamThreads) {
        if (p.groups == 1) finish(u, n0, sums[u]);
        else meet_store(p.part + ((size_t)group * p.T + u / CB) * p.part_wide + n0 + u % CB, sums[u]);
    }
    if (p.groups == 1) return;
    const int b0 = nb / p.per * p.per, b1 = min(b0 + p.per, p.blocks);
    if (!meet_last(p.count + nb / p.per, (uint32_t)((b1 - b0) * p.groups), &flag)) return;
    for (int b = b0; b < b1; ++b)
#pragma unroll 1
        for (int u = tid; u < p.T * CB; u += kStreamThreads)
            finish(u, b * CB, meet_sum(p.part + (size_t)(u / CB) * p.part_wide + b * CB + u % CB, p.groups, (size_t)p.T * p.part_wide));
}

}  // namespace gsr
