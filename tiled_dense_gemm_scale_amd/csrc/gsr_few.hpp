// gsr_few.hpp -- a whole layer of routed experts for a few tokens, in two
// launches:
//
//     h[s, f] = act(x[t] up[e] + bias_up[e])                (slot s = t k + j, e = ids[s])
//     h[s, f] = act(x[t] gate[e] + bias_gate[e]) (x[t] up[e] + bias_up[e])    with a gate
//     out[t, o] = sum_j weights[s] (h[s] down[e] + bias_down[e])
//
// With a few tokens the layer is bound by the bytes of the weights that the
// choices hit, so there is no sort and no gather in front: every workgroup counts
// the experts' slots from the ids itself, and every wave finds the slots of its
// own expert and streams its columns of that expert's matrix past their rows
// (gsr_stream.hpp), 16 of them: a tile.  An expert of more rows has more
// tiles, on neighbouring waves, which read its weights from the caches.  How many
// tiles there are is known on the device only, so the grid is fixed and the waves
// share out what there is.
//  * up: an item is a tile and a block of columns; 1, 2, 4 or 8 waves of a
//    workgroup split its H, whichever leaves the fewest idle.
//  * down: a workgroup has a block of columns; its waves take jobs, a tile and a
//    part of F, weigh their rows and add them per token in LDS, in order of the
//    experts.  The workgroups of a block meet in the workspace and the last one
//    adds their sums in order, so equal inputs give equal bits.
// Between the launches h is two fp16 values, rounded and 2^11 times what that lost
// (stream_split), as the matrix cores take it: one rounding to fp16 would be as large as that of out, and
// the error of out against 64 bits 0.00029 in place of 0.00021, its own rounding's
// (64 tokens x 2 of 8 in 4 bits 129 us so and 154 with both halves, when A was read
// row by row; the others within 2 us).
// Measured: 4096 -> 11008 -> 4096, 2 of 8 experts, one token: 361 MB in fp16 in 77
// us (36 and 40 of them the launches' own), in 4 bits 93 MB in 34 to 38 us (15 and
// 18, of which the ids, the tiles, the first loads and the meeting take about 5
// each); 16 tokens x 8 of 64 gated experts 2048 -> 1024 -> 2048, 710 MB in 104 to
// 113 us and 194 MB in 51.  With many tokens in 4 bits the waves wait 39 and 48 %
// of their time and unpack codes for most of the rest: 64 tokens x 2 of 8 141 to
// 144 us (54 and 77 under the profiler) for 373 MB.  With several rows to an expert
// the layer of four launches is as fast or faster: 4096 -> 11008 in fp16, 2 of 8
// experts, 16 tokens 266 us here and 272 there, 32 272 and 266, 64 311 and 266 (8
// of 64 experts 2048 -> 1024, 64 tokens 122 and 127).
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
    uint16_t* hidden;      // slots x 2 x hidden_wide
    float* part;           // groups x T x part_wide
    uint32_t* count;
    int T, k, slots, experts, H, F, O;
    int hidden_wide, part_wide;
    int act;
    bool wide_ids;
    int blocks_up;         // column blocks of the first launch
    int waves_log2;        // its waves (a power of two)
    int blocks, groups;    // of the second: column blocks, workgroups to each
};

// The stream of a form of weights: fp16, 4 bits with groups of 32, 64, and 128 or
// more rows.  DW: every row of fp16 weights and of A starts on a dword.
enum : int { kFewHalf = 0, kFewW4x1 = 1, kFewW4x2 = 2, kFewW4x4 = 3 };
template <int FORM, bool DW, bool SPLIT>
struct FewStream : W4Stream<FORM == kFewW4x1 ? 1 : FORM == kFewW4x2 ? 2 : 4, DW, SPLIT> {
    __device__ static __forceinline__ W4Matrix matrix(const FewWeights& w, int e, int K, int N)
    {
        const size_t words = (size_t)((K + 7) / 8) * N, groups = (size_t)((((int64_t)K - 1) >> w.glog2) + 1) * N;
        return W4Matrix{(const uint32_t*)w.data + e * words, w.scales + e * groups, w.zeros ? w.zeros + e * groups : nullptr,
                        w.glog2};
    }
};
template <bool DW, bool SPLIT>
struct FewStream<kFewHalf, DW, SPLIT> : HalfStream<DW, SPLIT> {
    __device__ static __forceinline__ HalfMatrix matrix(const FewWeights& w, int e, int K, int N)
    {
        return HalfMatrix{(const uint16_t*)w.data + (size_t)e * K * N};
    }
};

// What a workgroup finds out from the ids: a slot's expert (-1: none), and the
// tiles of the experts up to each.
constexpr int kFewRows = 16;  // rows of a tile
struct FewPlan {
    int16_t key[kFewSlots];
    int32_t upto[kFewExperts];  // slots of the expert first
    int16_t slot[kStreamWaves][kFewRows];  // the slots of a wave's tile, ascending
};

// Fills key and upto; returns the tiles.
__device__ __forceinline__ int few_plan(FewPlan& s, const FewArgs& p)
{
    const int tid = threadIdx.x, lane = tid & 63;
    for (int i = tid; i < p.experts; i += kStreamThreads) s.upto[i] = 0;
    __syncthreads();
    for (int i = tid; i < p.slots; i += kStreamThreads) {
        const int64_t id = p.wide_ids ? ((const int64_t*)p.ids)[i] : (int64_t)((const int32_t*)p.ids)[i];
        const bool in = id >= 0 && id < p.experts;
        s.key[i] = in ? (int16_t)id : (int16_t)-1;
        if (in) atomicAdd(&s.upto[(int)id], 1);
    }
    __syncthreads();
    int total = 0;
    if (tid < kWave)
        for (int e0 = 0; e0 < p.experts; e0 += kWave) {
            int n = e0 + lane < p.experts ? (s.upto[e0 + lane] + kFewRows - 1) / kFewRows : 0;
#pragma unroll
            for (int x = 1; x < kWave; x <<= 1) {
                const int o = __shfl_up(n, x);
                if (lane >= x) n += o;
            }
            if (e0 + lane < p.experts) s.upto[e0 + lane] = total + n;
            total += __builtin_amdgcn_readlane(n, kWave - 1);
        }
    __syncthreads();
    return p.experts > 0 ? __builtin_amdgcn_readfirstlane(s.upto[p.experts - 1]) : 0;
}

// Each tile stands `times` times in the waves' items, those of an expert of more
// than one next to each other: item i is the `turn`-th of its tile.
struct FewItem {
    int e, tile, turn;
};
__device__ __forceinline__ FewItem few_item(const FewPlan& s, int experts, int i, int times)
{
    const int lane = threadIdx.x & 63, d = (int)((uint32_t)i / (uint32_t)times);
    int e0 = 0;
    uint64_t m;
    while ((m = __ballot(e0 + lane < experts && s.upto[e0 + lane] > d)) == 0) e0 += kWave;
    const int e = e0 + __ffsll((unsigned long long)m) - 1;
    const int before = e > 0 ? __builtin_amdgcn_readfirstlane(s.upto[e - 1]) : 0;
    const int n = __builtin_amdgcn_readfirstlane(s.upto[e]) - before, at = i - before * times;
    if (n == 1) return FewItem{e, 0, at};
    const int turn = (int)((uint32_t)at / (uint32_t)n);
    return FewItem{e, at - turn * n, turn};
}

// The slots of expert e's tile into this wave's list; how many there are.
__device__ __forceinline__ int few_rows(int16_t* list, const int16_t* key, int slots, int e, int tile)
{
    const int lane = threadIdx.x & 63, m0 = tile * kFewRows;
    int n = 0;
    wave_fence();
    for (int i0 = 0; i0 < slots && n < m0 + kFewRows; i0 += kWave) {
        const bool mine = i0 + lane < slots && key[i0 + lane] == e;
        const uint64_t m = __ballot(mine);
        const int at = n + __popcll(m & ((1ull << lane) - 1ull)) - m0;
        if (mine && at >= 0 && at < kFewRows) list[at] = (int16_t)(i0 + lane);
        n += __popcll(m);
    }
    wave_fence();
    return __builtin_amdgcn_readfirstlane(min(n - m0, kFewRows));
}

// log2 of how many of a workgroup's waves split an item's K of `units` (2^least
// at least): the count for which the rounds of `waves` (a power of two) waves,
// each `fixed` units longer than its share of K, are shortest.  (16 tokens x 8 of
// 64 gated experts in fp16 with 1, 2, 4 and 8 waves: 143, 143, 113 and 117 us.)
__device__ __forceinline__ int few_split(int items, int waves_log2, int units, int fixed, int least)
{
    int best = least;
    float shortest = 1e30f;
#pragma unroll 1
    for (int s = least; s <= 3; ++s) {
        const int rounds = ((items << s) + (1 << waves_log2) - 1) >> waves_log2;  // items are below 2^27
        const float cost = (float)rounds * (float)((units >> (s - least)) + fixed);
        if (cost < shortest) {
            shortest = cost;
            best = s;
        }
    }
    return best;
}

// h of the experts' slots.  With a gate the first half of an item's waves
// streams the gate and the second half up.
template <int FORM, bool DW, bool GATED>
__global__ void __launch_bounds__(kStreamThreads, 2) few_up_kernel(FewArgs p)
{
    using S = FewStream<FORM, DW, false>;
    constexpr int CPL = S::CPL, CB = S::CB, UNIT = S::UNIT, QUADS = CB / 4, SETS = GATED ? 2 : 1;
    __shared__ __attribute__((aligned(16))) float lds[kStreamWaves * 16 * CB];
    __shared__ FewPlan plan;
    __shared__ int expert_of[kStreamWaves], block_of[kStreamWaves], count_of[kStreamWaves];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int items = few_plan(plan, p) * p.blocks_up, units = (p.H + UNIT - 1) / UNIT;
    const int kl = few_split(items, p.waves_log2, units, 256 / UNIT, SETS - 1), kg = 1 << kl, cg = kStreamWaves >> kl;
    const int turn = wave & (kg - 1), half = kg / SETS;  // the waves of one matrix
    const FewWeights& w = GATED && turn < half ? p.gate : p.up;
    const int hl = kl - (SETS - 1), u0 = (units * (turn & (half - 1))) >> hl, u1 = (units * ((turn & (half - 1)) + 1)) >> hl;

    for (int first = blockIdx.x * cg; first < items; first += gridDim.x * cg) {
        const int item = first + (wave >> kl);
        FewItem at{-1, 0, 0};
        int count = 0;
        typename S::Sums acc;
        if (item < items) {
            at = few_item(plan, p.experts, item, p.blocks_up);
            count = few_rows(plan.slot[wave], plan.key, p.slots, at.e, at.tile);
            typename S::Rows rows(p.x, (uint64_t)p.T * (uint32_t)p.H * 2u, count);
            rows.row((uint32_t)plan.slot[wave][min(stream_row(), count - 1)] / (uint32_t)p.k * (uint32_t)p.H);
            acc.clear();
            S::run(S::matrix(w, at.e, p.H, p.F), p.H, p.F, at.turn * CB, rows, u0, u1, lds + wave * 16 * CB, acc);
        }
        if ((threadIdx.x & 63) == 0) {
            expert_of[wave] = at.e;
            block_of[wave] = at.turn * CB;
            count_of[wave] = count;
        }
        if (count > 0) stream_put<CPL>(lds + wave * 16 * CB, acc);
        __syncthreads();
#pragma unroll 1
        for (int u = threadIdx.x; u < cg * 16 * QUADS; u += kStreamThreads) {
            const int c = u / (16 * QUADS) << kl, m = u / QUADS % 16, q = u % QUADS;
            if (m >= count_of[c]) continue;
            const int ex = expert_of[c], col = stream_position<CPL>(block_of[c], q, p.F);
            const float* slices = lds + c * 16 * CB;
            if (col < 0) continue;
            const f32x4 none = {0.f, 0.f, 0.f, 0.f};
            f32x4 v = add4(stream_sum<CPL>(slices + (kg - half) * 16 * CB, half, m, q),
                           p.up.bias ? half4_at(p.up.bias + (size_t)ex * p.F, col, p.F) : none);
            if constexpr (GATED) {
                const f32x4 g = add4(stream_sum<CPL>(slices, half, m, q),
                                     p.gate.bias ? half4_at(p.gate.bias + (size_t)ex * p.F, col, p.F) : none);
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] *= stream_activate(g[i], p.act);
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = stream_activate(v[i], p.act);
            }
            uint16_t* row = p.hidden + (size_t)plan.slot[c][m] * 2 * p.hidden_wide;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col + i < p.F) {
                    const StreamHalves h = stream_split(v[i]);
                    row[S::order(col + i)] = h.hi;
                    row[p.hidden_wide + S::order(col + i)] = h.lo;
                }
            if (col + 4 >= p.F)  // zeros up to the width
                for (int i = p.F; i < p.hidden_wide; ++i) row[S::order(i)] = row[p.hidden_wide + S::order(i)] = (uint16_t)0;
        }
        __syncthreads();
    }
}

// out of a block of columns.  A job's rows are weighed and
// added to their tokens' sums in LDS: per token a mask of the waves that have
// rows of it (two masks in turn, one cleared while the other is read), and its
// first row in each; the rows of a token lie behind each other.
template <int FORM, bool DW>
__global__ void __launch_bounds__(kStreamThreads, 2) few_down_kernel(FewArgs p)
{
    using S = FewStream<FORM, DW, true>;
    constexpr int CPL = S::CPL, CB = S::CB, UNIT = S::UNIT, QUADS = CB / 4;
    __shared__ __attribute__((aligned(16))) float lds[kStreamWaves * 16 * CB];
    __shared__ f32x4 sums[kFewTokens * QUADS];
    __shared__ FewPlan plan;
    __shared__ uint32_t mask[2][kFewTokens];
    __shared__ int8_t row_of[kStreamWaves][kFewTokens], token_of[kStreamWaves][kFewRows + 1];
    __shared__ float weight_of[kStreamWaves][kFewRows];
    __shared__ int bias_of[kStreamWaves];  // the expert whose bias a wave's rows get, or -1
    __shared__ int flag;
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int nb = blockIdx.x / p.groups, group = blockIdx.x - nb * p.groups, n0 = nb * CB;
    for (int i = tid; i < p.T * QUADS; i += kStreamThreads) sums[i] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (tid < kFewTokens) mask[0][tid] = mask[1][tid] = 0u;
    const int tiles = few_plan(plan, p), units = (p.F + UNIT - 1) / UNIT;
    // every wave of the block has a job where that leaves each 128 rows of F (7
    // tokens x 3 of 10 experts 1001 -> 517 -> 1001 27.6 us, with 256 rows 29.3)
    const int parts = max(1, min(p.groups * kStreamWaves / max(tiles, 1), units * UNIT / 128)), jobs = tiles * parts;
    const int j0 = jobs * group / p.groups, j1 = jobs * (group + 1) / p.groups;

    int turn = 0;
    for (int first = j0; first < j1; first += kStreamWaves) {
        const int job = first + wave;
        typename S::Sums acc;
        if (job < j1) {
            const FewItem it = few_item(plan, p.experts, job, parts);
            const int e = it.e, part = it.turn, count = few_rows(plan.slot[wave], plan.key, p.slots, e, it.tile);
            if (lane < count) {
                const int slot = plan.slot[wave][lane], token = slot / p.k;
                token_of[wave][lane] = (int8_t)token;
                weight_of[wave][lane] = p.weights ? p.weights[slot] : 1.0f;
                if (lane == 0 || plan.slot[wave][lane - 1] / p.k != token) row_of[wave][token] = (int8_t)lane;
                atomicOr(&mask[turn][token], 1u << wave);
            }
            if (lane == 0) {
                token_of[wave][count] = -1;
                bias_of[wave] = p.down.bias && part == 0 ? e : -1;
            }
            typename S::Rows rows(p.hidden, (uint64_t)p.slots * (uint32_t)p.hidden_wide * 4u, count);
            rows.wide = p.hidden_wide;
            rows.row((uint32_t)plan.slot[wave][min(stream_row(), count - 1)] * 2u * (uint32_t)p.hidden_wide);
            acc.clear();
            S::run(S::matrix(p.down, e, p.F, p.O), p.F, p.O, n0, rows, (int)((uint32_t)(units * part) / (uint32_t)parts),
                   (int)((uint32_t)(units * (part + 1)) / (uint32_t)parts), lds + wave * 16 * CB, acc);  // 2^17 units, 2^7 parts at most
            stream_put<CPL>(lds + wave * 16 * CB, acc);
        }
        __syncthreads();
#pragma unroll 1
        for (int u = tid; u < p.T * QUADS; u += kStreamThreads) {
            const int token = u / QUADS, q = u % QUADS;
            uint32_t from = mask[turn][token];
            if (from == 0u) continue;
            const int col = stream_position<CPL>(n0, q, p.O);
            f32x4 s = sums[u];
            do {
                const int w = __ffs((int)from) - 1;
                from &= from - 1u;
                f32x4 b = {0.f, 0.f, 0.f, 0.f};
                if (bias_of[w] >= 0 && col >= 0) b = half4_at(p.down.bias + (size_t)bias_of[w] * p.O, col, p.O);
                int r = row_of[w][token];
                do {
                    const f32x4 y = *(const f32x4*)(lds + (w * 16 + r) * CB + 4 * q);
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[i] = fmaf(weight_of[w][r], y[i] + b[i], s[i]);
                } while (token_of[w][++r] == token);
            } while (from != 0u);
            sums[u] = s;
        }
        turn ^= 1;
        if (tid < kFewTokens) mask[turn][tid] = 0u;  // read before the barrier above
        __syncthreads();
    }

    auto finish = [&](int u, f32x4 s) {
        const int col = stream_position<CPL>(n0, u % QUADS, p.O);
        if (col >= 0) put_half4(p.out + (size_t)(u / QUADS) * p.O, col, p.O, s);
    };
    for (int u = tid; u < p.T * QUADS; u += kStreamThreads) {
        if (p.groups == 1) finish(u, sums[u]);
        else meet_store(p.part + ((size_t)group * p.T + u / QUADS) * p.part_wide + n0 + 4 * (u % QUADS), sums[u]);
    }
    if (p.groups == 1) return;
    if (!meet_last(p.count + nb, (uint32_t)p.groups, &flag)) return;
    for (int u = tid; u < p.T * QUADS; u += kStreamThreads)
        finish(u, meet_sum(p.part + (size_t)(u / QUADS) * p.part_wide + n0 + 4 * (u % QUADS), p.groups, (size_t)p.T * p.part_wide));
}

}  // namespace gsr
