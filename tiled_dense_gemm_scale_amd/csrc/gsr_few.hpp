// gsr_few.hpp -- a whole layer of routed experts for a few tokens, in two
// launches:
//
//     h[s, f] = act(x[t] up[e] + bias_up[e])                (slot s = t k + j, e = ids[s])
//     h[s, f] = act(x[t] gate[e] + bias_gate[e]) (x[t] up[e] + bias_up[e])    with a gate
//     out[t, o] = sum_j weights[s] (h[s] down[e] + bias_down[e])
//
// With a few tokens the layer is bound by the bytes of the weights that the
// choices hit, so there is no sort and no gather in front: every workgroup
// finds the experts that are hit, and its expert's slots, from the ids itself,
// and streams its columns of that expert's matrix past the slots' rows
// (gsr_stream.hpp).  The grid holds as many experts as the choices can hit, and
// the surplus ends at once.  The second launch also adds a token's choices: the
// slots' sums meet in the workspace and the last workgroup of a column block
// weighs and adds them in order of j, so equal inputs give equal bits.  h is
// rounded to fp16 between the launches, as the fp16 matrix cores take it.
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
    float* part;           // parts x slots x part_wide
    uint32_t* count;
    int T, k, slots, experts, H, F, O;
    int most;              // experts that a grid holds, at most min(experts, slots), at least 1
    int hidden_wide, part_wide;
    int act;
    bool wide_ids;
    int blocks, parts, chunk;  // of the second launch: column blocks; parts of F, of `chunk` units each
    int per;                   // column blocks per counter
};

template <int FMT, int MT, int FL>
struct FewStream;
template <int MT, int FL>
struct FewStream<0, MT, FL> : HalfStream<MT> {
    __device__ static __forceinline__ HalfMatrix matrix(const FewWeights& w, int e, int K, int N)
    {
        return HalfMatrix{(const uint16_t*)w.data + (size_t)e * K * N};
    }
};
template <int MT, int FL>
struct FewStream<1, MT, FL> : W4Stream<MT, FL> {
    __device__ static __forceinline__ W4Matrix matrix(const FewWeights& w, int e, int K, int N)
    {
        const size_t words = (size_t)((K + 7) / 8) * N, groups = (size_t)((((int64_t)K - 1) >> w.glog2) + 1) * N;
        return W4Matrix{(const uint32_t*)w.data + e * words, w.scales + e * groups, w.zeros ? w.zeros + e * groups : nullptr,
                        w.glog2};
    }
};

// What a workgroup finds out from the ids.
struct FewPlan {
    int16_t key[kFewSlots];   // a slot's expert, -1: none
    int16_t list[kFewSlots];  // the slots of this workgroup's expert, ascending
    uint32_t hit[kFewExperts / 32];
    int total, expert, count;  // experts hit; this workgroup's (-1: none left), its slots
    int flag;
};

// The d-th of the experts that are hit, ascending, and its slots.
__device__ __forceinline__ void few_plan(FewPlan& s, const FewArgs& p, int d)
{
    const int tid = threadIdx.x, lane = tid & 63;
    if (tid < kFewExperts / 32) s.hit[tid] = 0u;
    __syncthreads();
    for (int i = tid; i < p.slots; i += kStreamThreads) {
        const int64_t id = p.wide_ids ? ((const int64_t*)p.ids)[i] : (int64_t)((const int32_t*)p.ids)[i];
        const bool in = id >= 0 && id < p.experts;
        s.key[i] = in ? (int16_t)id : (int16_t)-1;
        if (in) atomicOr(&s.hit[(int)id >> 5], 1u << ((int)id & 31));
    }
    __syncthreads();
    if (tid < kWave) {
        const uint32_t w = lane < kFewExperts / 32 ? s.hit[lane] : 0u;
        const int mine = __popc(w);
        int upto = mine;
#pragma unroll
        for (int x = 1; x < kFewExperts / 32; x <<= 1) {
            const int o = __shfl_up(upto, x);
            if (lane >= x) upto += o;
        }
        const int total = __shfl(upto, kFewExperts / 32 - 1);
        const uint64_t at = __ballot(d < upto);  // the lowest lane of these holds the word
        int expert = -1;
        if (d < total) {
            const int word = __ffsll((unsigned long long)at) - 1;
            uint32_t bits = (uint32_t)__shfl((int)w, word);
            for (int left = d - (__shfl(upto, word) - __shfl(mine, word)); left > 0; --left) bits &= bits - 1u;
            expert = 32 * word + __ffs((int)bits) - 1;
        }
        int n = 0;
        for (int i0 = 0; i0 < p.slots; i0 += kWave) {
            const bool mine_too = expert >= 0 && i0 + lane < p.slots && s.key[i0 + lane] == expert;
            const uint64_t m = __ballot(mine_too);
            if (mine_too) s.list[n + __popcll(m & ((1ull << lane) - 1ull))] = (int16_t)(i0 + lane);
            n += __popcll(m);
        }
        if (lane == 0) {
            s.total = total;
            s.expert = expert;
            s.count = n;
        }
    }
    __syncthreads();
}

// h of one expert's slots and CB hidden columns.  With a gate the first half
// of the waves streams the gate and the second half up.
template <int FMT, int MT, int FL, bool GATED>
__global__ void __launch_bounds__(kStreamThreads) few_up_kernel(FewArgs p)
{
    using S = FewStream<FMT, MT, FL>;
    constexpr int CPL = S::CPL, CB = S::CB, SETS = GATED ? 2 : 1, W = kStreamWaves / SETS;
    __shared__ __attribute__((aligned(16))) float lds[kStreamWaves * 16 * CB];
    __shared__ FewPlan plan;
    few_plan(plan, p, blockIdx.x % p.most);
    if (plan.expert < 0) return;
    const int e = plan.expert, count = plan.count, n0 = blockIdx.x / p.most * CB;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 15;
    const FewWeights& w = GATED && wave < W ? p.gate : p.up;
    const int units = (p.H + S::UNIT - 1) / S::UNIT, turn = wave % W;
    const int u0 = (int)((int64_t)units * turn / W), u1 = (int)((int64_t)units * (turn + 1) / W);

    for (int m0 = 0; m0 < count; m0 += 16 * MT) {
        const int tiles = min(MT, (count - m0 + 15) / 16);
        StreamRows<MT> rows;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int m = m0 + 16 * t + l;
            rows.p[t] = m < count ? p.x + (size_t)(plan.list[m] / p.k) * p.H : nullptr;
        }
        typename S::Sums acc;
        acc.clear();
        S::run(S::matrix(w, e, p.H, p.F), p.H, p.F, n0, rows, tiles, u0, u1, acc);
        stream_reduce<CPL, MT, SETS>(lds, acc, tiles, [&](int m, int q, f32x4 s, f32x4 s2) {
            const int col = stream_position<CPL>(n0, q, p.F);
            if (m0 + m >= count || col < 0) return;
            uint16_t* to = p.hidden + (size_t)plan.list[m0 + m] * p.hidden_wide + col;
            const size_t at = (size_t)e * p.F + col;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (col + i >= p.F) break;
                const float bu = p.up.bias ? half_at(p.up.bias + at + i) : 0.0f;
                float v;
                if constexpr (GATED) {
                    const float bg = p.gate.bias ? half_at(p.gate.bias + at + i) : 0.0f;
                    v = stream_activate(s[i] + bg, p.act) * (s2[i] + bu);
                } else {
                    v = stream_activate(s[i] + bu, p.act);
                }
                to[i] = to_half(v);
            }
        });
    }
}

// One expert's slots, CB output columns and a part of F; then, in the workgroup
// that comes last of a counter's blocks, the tokens' sums.
template <int FMT, int MT, int FL>
__global__ void __launch_bounds__(kStreamThreads) few_down_kernel(FewArgs p)
{
    using S = FewStream<FMT, MT, FL>;
    constexpr int CPL = S::CPL, CB = S::CB, QUADS = CB / 4;
    __shared__ __attribute__((aligned(16))) float lds[kStreamWaves * 16 * CB];
    __shared__ FewPlan plan;
    const int d = blockIdx.x % p.most, rest = blockIdx.x / p.most, part = rest % p.parts, nb = rest / p.parts;
    few_plan(plan, p, d);
    if (plan.expert < 0 && d > 0) return;  // without any expert the first of each part still counts
    const int e = plan.expert, count = plan.count, n0 = nb * CB;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = threadIdx.x & 15;
    const int units = (p.F + S::UNIT - 1) / S::UNIT;
    const int first = part * p.chunk, here = max(0, min(p.chunk, units - first));
    const int u0 = first + here * wave / kStreamWaves, u1 = first + here * (wave + 1) / kStreamWaves;

    for (int m0 = 0; m0 < count; m0 += 16 * MT) {
        const int tiles = min(MT, (count - m0 + 15) / 16);
        StreamRows<MT> rows;
#pragma unroll
        for (int t = 0; t < MT; ++t) {
            const int m = m0 + 16 * t + l;
            rows.p[t] = m < count ? p.hidden + (size_t)plan.list[m] * p.hidden_wide : nullptr;
        }
        typename S::Sums acc;
        acc.clear();
        S::run(S::matrix(p.down, e, p.F, p.O), p.F, p.O, n0, rows, tiles, u0, u1, acc);
        stream_reduce<CPL, MT, 1>(lds, acc, tiles, [&](int m, int q, f32x4 s, f32x4) {
            if (m0 + m < count)
                meet_store(p.part + ((size_t)part * p.slots + plan.list[m0 + m]) * p.part_wide + n0 + 4 * q, s);
        });
    }
    const int b0 = nb / p.per * p.per, b1 = min(b0 + p.per, p.blocks);
    if (!meet_last(p.count + nb / p.per, (uint32_t)((b1 - b0) * p.parts * max(plan.total, 1)), &plan.flag)) return;
    for (int b = b0; b < b1; ++b)
        for (int u = threadIdx.x; u < p.T * QUADS; u += kStreamThreads) {
            const int t = u / QUADS, q = u % QUADS, col = stream_position<CPL>(b * CB, q, p.O);
            if (col < 0) continue;
            f32x4 sum = {0.f, 0.f, 0.f, 0.f};
            for (int j = 0; j < p.k; ++j) {
                const int slot = t * p.k + j, key = plan.key[slot];
                if (key < 0) continue;
                f32x4 y = {0.f, 0.f, 0.f, 0.f};
                for (int g = 0; g < p.parts; ++g) {
                    const f32x4 v = meet_load(p.part + ((size_t)g * p.slots + slot) * p.part_wide + b * CB + 4 * q);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] += v[i];
                }
                const float w = p.weights ? p.weights[slot] : 1.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (p.down.bias && col + i < p.O) y[i] += half_at(p.down.bias + (size_t)key * p.O + col + i);
                    sum[i] = fmaf(w, y[i], sum[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col + i < p.O) p.out[(size_t)t * p.O + col + i] = to_half(sum[i]);
        }
}

}  // namespace gsr
