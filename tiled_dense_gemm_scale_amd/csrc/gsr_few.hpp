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
    int blocks, groups;    // of the second: column blocks, workgroups to each
    int per;               // column blocks per counter
};

// The stream of a form of weights: fp16 with rows on dwords, fp16 at any
// address, 4 bits with groups of 32, 64, and 128 or more rows.
enum : int { kFewHalf = 0, kFewHalfAny = 1, kFewW4x1 = 2, kFewW4x2 = 3, kFewW4x4 = 4 };
template <int FORM, int MT>
struct FewStream : W4Stream<MT, FORM == kFewW4x1 ? 1 : FORM == kFewW4x2 ? 2 : 4> {
    __device__ static __forceinline__ W4Matrix matrix(const FewWeights& w, int e, int K, int N)
    {
        const size_t words = (size_t)((K + 7) / 8) * N, groups = (size_t)((((int64_t)K - 1) >> w.glog2) + 1) * N;
        return W4Matrix{(const uint32_t*)w.data + e * words, w.scales + e * groups, w.zeros ? w.zeros + e * groups : nullptr,
                        w.glog2};
    }
};
template <int MT>
struct FewStream<kFewHalf, MT> : HalfStream<MT, true> {
    __device__ static __forceinline__ HalfMatrix matrix(const FewWeights& w, int e, int K, int N)
    {
        return HalfMatrix{(const uint16_t*)w.data + (size_t)e * K * N};
    }
};
template <int MT>
struct FewStream<kFewHalfAny, MT> : HalfStream<MT, false> {
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
    const int lane = threadIdx.x & 63;
    if (lane < kFewExperts / 32) s.hit[lane] = 0u;
    wave_fence();
    for (int i = lane; i < p.slots; i += kWave) {
        const int64_t id = p.wide_ids ? ((const int64_t*)p.ids)[i] : (int64_t)((const int32_t*)p.ids)[i];
        const bool in = id >= 0 && id < p.experts;
        key[i] = in ? (int16_t)id : (int16_t)-1;
        if (in) atomicOr(&s.hit[(int)id >> 5], 1u << ((int)id & 31));
    }
    wave_fence();
    int n = lane < kFewExperts / 32 ? __popc(s.hit[lane]) : 0;
#pragma unroll
    for (int x = 1; x < kFewExperts / 32; x <<= 1) n += __shfl_xor(n, x);
    return __builtin_amdgcn_readfirstlane(n);
}

// The d-th expert that is hit, ascending (d below their number).
__device__ __forceinline__ int few_expert(const FewWave& s, int d)
{
    const int lane = threadIdx.x & 63;
    const uint32_t w = lane < kFewExperts / 32 ? s.hit[lane] : 0u;
    const int mine = __popc(w);
    int upto = mine;
#pragma unroll
    for (int x = 1; x < kFewExperts / 32; x <<= 1) {
        const int o = __shfl_up(upto, x);
        if (lane >= x) upto += o;
    }
    const int word = __ffsll((unsigned long long)__ballot(d < upto)) - 1;  // the lowest lane of these holds it
    uint32_t bits = __builtin_amdgcn_readlane(w, word);
    int left = d - (__builtin_amdgcn_readlane(upto, word) - __popc(bits));
    for (; left > 0; --left) bits &= bits - 1u;
    return __builtin_amdgcn_readfirstlane(32 * word + __ffs((int)bits) - 1);
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
template <int FORM, int MT>
__device__ __forceinline__ void few_stream(const FewWeights& w, int e, int K, int N, int n0, const StreamRows<MT>& rows, int left,
                                           int u0, int u1, typename FewStream<FORM, MT>::Sums& acc)
{
    acc.clear();
    if (MT > 1 && left <= kFewRows) {
        using S = FewStream<FORM, 1>;
        StreamRows<1> one;
        one.p[0] = rows.p[0];
        typename S::Sums sums;
        sums.clear();
        S::run(S::matrix(w, e, K, N), K, N, n0, one, u0, u1, sums);
#pragma unroll
        for (int j = 0; j < S::CPL; ++j) acc.v[j][0] = sums.v[j][0];
    } else {
        using S = FewStream<FORM, MT>;
        S::run(S::matrix(w, e, K, N), K, N, n0, rows, u0, u1, acc);
    }
}

// How many of a workgroup's waves split an item's K of `units` (`least` at
// least): the count for which the grid's rounds, each `fixed` units longer than
// its share of K, are shortest.
__device__ __forceinline__ int few_split(int items, int workgroups, int units, int fixed, int least)
{
    int best = least;
    int64_t shortest = INT64_MAX;
    for (int kg = least; kg <= kStreamWaves; kg *= 2) {
        const int64_t rounds = ((int64_t)items * kg + workgroups * kStreamWaves - 1) / (workgroups * kStreamWaves);
        const int64_t cost = rounds * ((units * least + kg - 1) / kg + fixed);
        if (cost < shortest) {
            shortest = cost;
            best = kg;
        }
    }
    return best;
}

// h of the experts' slots.  With a gate the first half of an item's waves
// streams the gate and the second half up.
template <int FORM, int MT, bool GATED>
__global__ void __launch_bounds__(kStreamThreads, 2) few_up_kernel(FewArgs p)
{
    using S = FewStream<FORM, MT>;
    constexpr int CPL = S::CPL, CB = S::CB, UNIT = S::UNIT, QUADS = CB / 4, EACH = 16 * QUADS, SETS = GATED ? 2 : 1;
    __shared__ __attribute__((aligned(16))) float lds[kStreamWaves * 16 * CB];
    __shared__ FewWave waves[kStreamWaves];
    __shared__ int16_t key[kFewSlots];
    __shared__ int experts[kStreamWaves], counts[kStreamWaves];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 15;
    FewWave& mine = waves[wave];
    const int hits = few_keys(mine, key, p), items = hits * p.blocks_up, units = (p.H + UNIT - 1) / UNIT;
    const int kg = few_split(items, gridDim.x, units, 256 / UNIT, SETS), cg = kStreamWaves / kg;
    const int turn = wave % kg, half = kg / SETS;  // the waves of one matrix
    const FewWeights& w = GATED && turn < half ? p.gate : p.up;
    const int u0 = (int)((int64_t)units * (turn % half) / half), u1 = (int)((int64_t)units * (turn % half + 1) / half);

    for (int first = blockIdx.x * cg; first < items; first += gridDim.x * cg) {
        const int item = first + wave / kg, n0 = item % p.blocks_up * CB;
        const bool have = item < items;
        const int e = have ? few_expert(mine, item / p.blocks_up) : -1;
        int count = 0, m0 = 0;
        do {
            if (have) count = few_rows(mine, key, p.slots, e, m0);
            typename S::Sums acc;
            if (m0 < count) {
                StreamRows<MT> rows;
#pragma unroll
                for (int t = 0; t < MT; ++t)
                    rows.p[t] = p.x + (size_t)(mine.slot[min(16 * t + l, count - 1 - m0)] / p.k) * p.H;
                few_stream<FORM, MT>(w, e, p.H, p.F, n0, rows, count - m0, u0, u1, acc);
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
                for (int u = threadIdx.x; u < cg * EACH; u += kStreamThreads) {
                    const int c = u / EACH, m = u % EACH / QUADS, q = u % QUADS;
                    const int col = stream_position<CPL>((first + c) % p.blocks_up * CB, q, p.F);
                    if (m0 + 16 * t + m >= counts[c * kg] || col < 0) continue;
                    const f32x4 s = stream_sum<CPL>(lds + (c * kg + kg - half) * 16 * CB, half, m, q);
                    f32x4 gate = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (GATED) gate = stream_sum<CPL>(lds + c * kg * 16 * CB, half, m, q);
                    uint16_t* to = p.hidden + (size_t)waves[c * kg].slot[16 * t + m] * p.hidden_wide + col;
                    const size_t b = (size_t)experts[c * kg] * p.F + col;
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        if (col + x >= p.F) break;
                        const float v = s[x] + (p.up.bias ? half_at(p.up.bias + b + x) : 0.0f);
                        if constexpr (GATED) {
                            const float g = gate[x] + (p.gate.bias ? half_at(p.gate.bias + b + x) : 0.0f);
                            to[x] = to_half(stream_activate(g, p.act) * v);
                        } else {
                            to[x] = to_half(stream_activate(v, p.act));
                        }
                    }
                }
            }
            m0 += 16 * MT;
        } while (__syncthreads_or(m0 < count));
    }
}

// out of a block of columns.  T is at most 16 NT.
template <int FORM, int MT, int NT>
__global__ void __launch_bounds__(kStreamThreads, 2) few_down_kernel(FewArgs p)
{
    using S = FewStream<FORM, MT>;
    constexpr int CPL = S::CPL, CB = S::CB, UNIT = S::UNIT, QUADS = CB / 4, UNITS = (16 * NT * QUADS + kStreamThreads - 1) / kStreamThreads;
    __shared__ __attribute__((aligned(16))) float lds[kStreamWaves * 16 * CB];
    __shared__ FewWave waves[kStreamWaves];
    __shared__ int16_t key[kFewSlots];
    __shared__ int8_t row_of[kStreamWaves][kFewTokens];  // a token's first row of a wave's tile, or -1
    __shared__ int8_t token_of[kStreamWaves][kFewRows + 1];
    __shared__ float weight_of[kStreamWaves][kFewRows];
    __shared__ int bias_of[kStreamWaves];                // the expert whose bias a wave's rows get, or -1
    __shared__ int flag;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), l = tid & 15;
    const int group = blockIdx.x % p.groups, nb = blockIdx.x / p.groups, n0 = nb * CB;
    FewWave& mine = waves[wave];
    const int hits = few_keys(mine, key, p), units = (p.F + UNIT - 1) / UNIT;
    // every wave of the block has a job where that leaves each 256 rows of F
    const int parts = max(1, min(p.groups * kStreamWaves / max(hits, 1), units * UNIT / 256)), jobs = hits * parts;
    const int j0 = (int)((int64_t)jobs * group / p.groups), j1 = (int)((int64_t)jobs * (group + 1) / p.groups);

    f32x4 sum[UNITS];
#pragma unroll
    for (int i = 0; i < UNITS; ++i) sum[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int first = j0; first < j1; first += kStreamWaves) {
        const int job = first + wave, part = job % parts;
        const bool have = job < j1;
        const int e = have ? few_expert(mine, job / parts) : -1;
        const int u0 = (int)((int64_t)units * part / parts), u1 = (int)((int64_t)units * (part + 1) / parts);
        int count = 0, m0 = 0;
        do {
            if (have) count = few_rows(mine, key, p.slots, e, m0);
            typename S::Sums acc;
            if (m0 < count) {
                StreamRows<MT> rows;
#pragma unroll
                for (int t = 0; t < MT; ++t) rows.p[t] = p.hidden + (size_t)mine.slot[min(16 * t + l, count - 1 - m0)] * p.hidden_wide;
                few_stream<FORM, MT>(p.down, e, p.F, p.O, n0, rows, count - m0, u0, u1, acc);
            }
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                __syncthreads();
                const int here = min(16, count - m0 - 16 * t);
                row_of[wave][lane] = -1;
                wave_fence();
                if (here > 0) {
                    if (lane < here) {
                        const int slot = mine.slot[16 * t + lane], token = slot / p.k;
                        token_of[wave][lane] = (int8_t)token;
                        weight_of[wave][lane] = p.weights ? p.weights[slot] : 1.0f;
                        if (lane == 0 || mine.slot[16 * t + lane - 1] / p.k != token) row_of[wave][token] = (int8_t)lane;
                    }
                    if (lane == 0) {
                        token_of[wave][here] = -1;
                        bias_of[wave] = p.down.bias && part == 0 ? e : -1;
                    }
                    stream_put<CPL, MT>(lds + wave * 16 * CB, acc, t);
                }
                __syncthreads();
#pragma unroll
                for (int i = 0; i < UNITS; ++i) {
                    const int u = tid + i * kStreamThreads, token = u / QUADS, q = u % QUADS;
                    if (token >= p.T) continue;
                    for (int w = 0; w < kStreamWaves; ++w) {
                        int r = row_of[w][token];
                        if (r < 0) continue;
                        const int col = stream_position<CPL>(n0, q, p.O);
                        f32x4 b = {0.f, 0.f, 0.f, 0.f};
                        if (bias_of[w] >= 0 && col >= 0)
#pragma unroll
                            for (int x = 0; x < 4; ++x) b[x] = col + x < p.O ? half_at(p.down.bias + (size_t)bias_of[w] * p.O + col + x) : 0.0f;
                        do {
                            const f32x4 y = *(const f32x4*)(lds + (w * 16 + r) * CB + 4 * q);
#pragma unroll
                            for (int x = 0; x < 4; ++x) sum[i][x] = fmaf(weight_of[w][r], y[x] + b[x], sum[i][x]);
                        } while (token_of[w][++r] == token);
                    }
                }
            }
            m0 += 16 * MT;
        } while (__syncthreads_or(m0 < count));
    }

    auto finish = [&](int u, int at, const f32x4& s) {
        const int col = stream_position<CPL>(at, u % QUADS, p.O);
        if (col < 0) return;
#pragma unroll
        for (int x = 0; x < 4; ++x)
            if (col + x < p.O) p.out[(size_t)(u / QUADS) * p.O + col + x] = to_half(s[x]);
    };
#pragma unroll
    for (int i = 0; i < UNITS; ++i) {
        const int u = tid + i * kStreamThreads;
        if (u >= p.T * QUADS) continue;
        if (p.groups == 1) finish(u, n0, sum[i]);
        else meet_store(p.part + ((size_t)group * p.T + u / QUADS) * p.part_wide + n0 + 4 * (u % QUADS), sum[i]);
    }
    if (p.groups == 1) return;
    const int b0 = nb / p.per * p.per, b1 = min(b0 + p.per, p.blocks);
    if (!meet_last(p.count + nb / p.per, (uint32_t)((b1 - b0) * p.groups), &flag)) return;
    for (int b = b0; b < b1; ++b)
        for (int u = tid; u < p.T * QUADS; u += kStreamThreads) {
            f32x4 s = {0.f, 0.f, 0.f, 0.f};
            for (int g = 0; g < p.groups; ++g) {
                const f32x4 v = meet_load(p.part + ((size_t)g * p.T + u / QUADS) * p.part_wide + b * CB + 4 * (u % QUADS));
#pragma unroll
                for (int x = 0; x < 4; ++x) s[x] += v[x];
            }
            finish(u, b * CB, s);
        }
}

}  // namespace gsr
