// gsr_rows.hpp -- rows sorted by group and back: the plan of a grouped
// product (group_*), the copy of rows into that order (gather), and the
// weighted sum of a token's rows with its gradient (combine).
//
// All of them move bytes: a row is read and written in the widest unit
// (16, 8, 4 or 2 bytes) that its addresses and its length allow, row bases are
// 64-bit, and no atomics on memory are used, so every call gives the same
// bits.  A row index outside its table means "no row": it reads as nothing
// (zeros in gather, no term in combine), and what it names is never touched,
// so NaN or infinity there does not spread.
#pragma once

#include "gsr_group_plan.hpp"
#include "gsr_kernels.hpp"

namespace gsr {

// ---- the plan: a stable counting sort of n slots by group --------------------
//
// Slots are cut into blocks of `chunk` consecutive slots, a block's into one
// run per wave, and a run is walked 64 slots at a time.  Inside such a step
// the lanes with the same key find each other with one ballot per key bit;
// a lane's rank is the number of such lanes below it, and the lowest of them
// adds their count to the wave's counter of that key, whose value before is
// where the step's slots of that key start within the wave.  Once all waves
// have counted, the counters are turned into start positions, and every slot
// has its place in stable order.  Runs of up to kGroupKept steps keep their
// slots' keys and places in registers meanwhile, longer ones walk twice.  Key
// `groups` collects the dropped slots (ids outside [0, groups)), which so sort
// behind all others.
//
// Up to kGroupSingle slots one workgroup does all of it.  Above, one launch
// counts per block and a second places: each of its blocks adds up the other
// blocks' counts by itself, which costs blocks x (groups + 1) reads per block
// (at most 256 blocks) but no third launch and no block waits for another.
// The work is bound by latency: the passes of a step depend on each other.
// 64 slots of 8 groups take 2.8 us, 8192 of 64 11.8 (walked twice: 15.8), and
// both launches for 131072 of 64 groups 11.9 (blocks of 4096 slots: 13.7; of
// 2048 and walked twice: 15.7), of 256 groups 16.7 (4096: 17.7, 1024: 20.1).
constexpr int kGroupKept = 8;  // steps whose keys and places a wave keeps

struct GroupArgs {
    const void* ids;      // n ids of 4 or 8 bytes
    int32_t* offsets;     // groups + 1
    int32_t* rows;        // n
    int32_t* positions;   // n
    uint32_t* hist;       // blocks x (groups + 1), or null (one block)
    int32_t n, k, groups;
    int32_t chunk, blocks;
    int32_t bits;         // key bits: groups < 2^bits
};

template <typename ID>
__device__ __forceinline__ int group_key(const GroupArgs& g, int i)
{
    const ID v = ((const ID*)g.ids)[i];
    return (v >= 0 && v < (ID)g.groups) ? (int)v : g.groups;
}

// The lanes of this wave that hold the same key (among those with key >= 0).
__device__ __forceinline__ uint64_t same_key(int key, int bits)
{
    uint64_t m = __ballot(key >= 0);
    for (int b = 0; b < bits; ++b) {
        const uint64_t one = __ballot((key >> b) & 1);
        m &= ((key >> b) & 1) ? one : ~one;
    }
    return m;
}

template <typename ID>
__global__ void __launch_bounds__(1024) group_count_kernel(GroupArgs g)
{
    __shared__ uint32_t cnt[kGroupMax + 1];
    const int nb = g.groups + 1;
    for (int i = threadIdx.x; i < nb; i += blockDim.x) cnt[i] = 0;
    __syncthreads();
    const GroupSpan all = group_block(g.n, g.chunk, blockIdx.x);
    const int lane = threadIdx.x & 63;
    for (int at = (int)(threadIdx.x & ~63u); at < all.len; at += blockDim.x) {
        const int key = at + lane < all.len ? group_key<ID>(g, all.beg + at + lane) : -1;
        const uint64_t m = same_key(key, g.bits);
        if (key >= 0 && lane == __ffsll((unsigned long long)m) - 1) atomicAdd(&cnt[key], (uint32_t)__popcll(m));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < nb; i += blockDim.x) g.hist[(size_t)blockIdx.x * nb + i] = cnt[i];
}

template <typename ID>
__global__ void __launch_bounds__(1024) group_place_kernel(GroupArgs g)
{
    __shared__ uint32_t cnt[kGroupWaves * (kGroupMax + 1)];  // [wave][key]: counts, then start positions
    __shared__ uint32_t total[kGroupMax + 1], prior[kGroupMax + 1];
    const int nb = g.groups + 1, nt = blockDim.x, waves = nt >> 6;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    for (int i = tid; i < waves * nb; i += nt) cnt[i] = 0;
    for (int i = tid; i < nb; i += nt) total[i] = prior[i] = 0;
    __syncthreads();

    const GroupSpan run = group_run(group_block(g.n, g.chunk, blockIdx.x), wave, waves);
    uint32_t* const mine = cnt + wave * nb;
    // the place of this lane's slot of a step among the wave's slots of its key
    auto place_of = [&](int key) {
        const uint64_t m = same_key(key, g.bits);
        const int leader = __ffsll((unsigned long long)m) - 1;
        uint32_t first = 0;
        if (key >= 0 && lane == leader) first = atomicAdd(&mine[key], (uint32_t)__popcll(m));
        return (uint32_t)__shfl((int)first, key >= 0 ? leader : lane) + (uint32_t)__popcll(m & ((1ull << lane) - 1ull));
    };
    const bool kept = run.len <= 64 * kGroupKept;
    int key[kGroupKept];
    uint32_t place[kGroupKept];
    if (kept) {
#pragma unroll
        for (int s = 0; s < kGroupKept; ++s) {
            const int at = 64 * s + lane;
            key[s] = at < run.len ? group_key<ID>(g, run.beg + at) : -1;
        }
#pragma unroll
        for (int s = 0; s < kGroupKept; ++s) place[s] = 64 * s < run.len ? place_of(key[s]) : 0u;
    } else {
        for (int at = 0; at < run.len; at += 64) place_of(at + lane < run.len ? group_key<ID>(g, run.beg + at + lane) : -1);
    }
    if (g.blocks > 1) {
        // every block's count of key e, and those of the blocks before this one
        const int seg = nt / nb > 0 ? nt / nb : 1;
        for (int e = tid % nb, s = tid / nb; s < seg && e < nb; e += nt) {
            uint32_t all = 0, before = 0;
            for (int b = s; b < g.blocks; b += seg) {
                const uint32_t c = g.hist[(size_t)b * nb + e];
                all += c;
                before += b < (int)blockIdx.x ? c : 0u;
            }
            atomicAdd(&total[e], all);
            atomicAdd(&prior[e], before);
        }
    }
    __syncthreads();
    // counts of the waves before, per key
    for (int e = tid; e < nb; e += nt) {
        uint32_t sum = 0;
        for (int w = 0; w < waves; ++w) {
            const uint32_t c = cnt[w * nb + e];
            cnt[w * nb + e] = sum;
            sum += c;
        }
        if (g.blocks == 1) total[e] = sum;
    }
    __syncthreads();
    // keys' start positions: an exclusive scan over the totals, by one wave
    if (wave == 0) {
        uint32_t carry = 0;
        for (int e0 = 0; e0 < nb; e0 += 64) {
            const int e = e0 + lane;
            const uint32_t v = e < nb ? total[e] : 0u;
            uint32_t inc = v;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const uint32_t o = (uint32_t)__shfl_up((int)inc, d);
                if (lane >= d) inc += o;
            }
            const uint32_t start = carry + inc - v;
            if (e < nb) {
                if (blockIdx.x == 0) g.offsets[e] = (int32_t)start;
                prior[e] += start;
            }
            carry += (uint32_t)__shfl((int)inc, 63);
        }
    }
    __syncthreads();
    auto put = [&](int i, int key, uint32_t at) {
        if (key < 0) return;
        const bool in = key < g.groups;
        at += prior[key];
        g.rows[at] = in ? (int32_t)(i / g.k) : -1;
        g.positions[i] = in ? (int32_t)at : -1;
    };
    if (kept) {
#pragma unroll
        for (int s = 0; s < kGroupKept; ++s)
            if (key[s] >= 0) put(run.beg + 64 * s + lane, key[s], mine[key[s]] + place[s]);
    } else {
        for (int at = 0; at < run.len; at += 64) {
            const bool in = at + lane < run.len;
            const int i = run.beg + at + (in ? lane : 0), k = in ? group_key<ID>(g, i) : -1;
            put(i, k, place_of(k));
        }
    }
}

// ---- units of a row -------------------------------------------------------------
// U bytes as U / 2 fp16 values (U = 16, 8, 4 or 2).
template <int U>
struct RowUnit;
template <>
struct RowUnit<16> {
    typedef u32x4 type;
};
template <>
struct RowUnit<8> {
    typedef u32x2 type;
};
template <>
struct RowUnit<4> {
    typedef uint32_t type;
};
template <>
struct RowUnit<2> {
    typedef uint16_t type;
};

template <int U>
struct HalfVec {
    typedef _Float16 type __attribute__((ext_vector_type(U / 2)));
    __device__ static __forceinline__ float at(const typename RowUnit<U>::type& v, int i)
    {
        return (float)__builtin_bit_cast(type, v)[i];
    }
    __device__ static __forceinline__ typename RowUnit<U>::type pack(const float (&f)[U / 2])
    {
        type h;
#pragma unroll
        for (int i = 0; i < U / 2; ++i) h[i] = (_Float16)f[i];
        return __builtin_bit_cast(typename RowUnit<U>::type, h);
    }
};
template <>
struct HalfVec<2> {
    __device__ static __forceinline__ float at(const uint16_t& v, int) { return (float)__builtin_bit_cast(_Float16, v); }
    __device__ static __forceinline__ uint16_t pack(const float (&f)[1])
    {
        return __builtin_bit_cast(uint16_t, (_Float16)f[0]);
    }
};

template <bool STREAM, typename V>
__device__ __forceinline__ V row_load(const V* p)
{
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    else return *p;
}

struct RowArgs {
    const uint16_t* x;         // gather: the table; combine: y; backward: dout
    const uint16_t* y;         // backward: y
    const int32_t* index;      // gather, backward's zero rows: rows; combine: positions
    const int32_t* positions;  // backward: positions
    const float* weights;      // T x k, or null (ones)
    uint16_t* out;             // gather: P x H; combine: T x H; backward: dy
    float* dweights;           // backward: T x k, or null
    int32_t T, P, k;
    int32_t units;             // units per row
    int32_t lanes_log2;        // threads per row
};

// A grid dimension holds fewer than 2^32 threads (of more, a part runs and nothing
// is reported), so from kRowBlocks workgroups on a launch has
// several rows of so many, numbered one behind the other.  (Reading the grid's
// size instead of the constant costs a small call 0.6 us.)
constexpr int64_t kRowBlocks = 1 << 20;
__device__ __forceinline__ int64_t row_block() { return (int64_t)blockIdx.y * kRowBlocks + blockIdx.x; }

// out[p] = x[rows[p]], zeros where rows[p] names no row of x.  2^lanes_log2
// threads walk a row; their loads of four units are in flight together.  It
// runs at the rate of a copy: 4098 rows of 4096 (50 MB) in 10.8 us, 8192x2x4096
// (201 MB) in 39 us (5.2 TB/s); rows of odd length go 2 bytes at a time, 2331
// of 1001 in 3.4 us, 8192x2x4095 in 41.
template <int U>
__global__ void __launch_bounds__(256) gather_rows_kernel(RowArgs r)
{
    typedef typename RowUnit<U>::type V;
    const int tpr = 1 << r.lanes_log2;
    const int64_t p = row_block() * (256 >> r.lanes_log2) + (threadIdx.x >> r.lanes_log2);
    if (p >= r.P) return;
    const int32_t t = r.index[p];
    const bool ok = (uint32_t)t < (uint32_t)r.T;
    const V* src = (const V*)r.x + (int64_t)(ok ? t : 0) * r.units;
    V* dst = (V*)r.out + p * r.units;
    for (int u = threadIdx.x & (tpr - 1); u < r.units; u += 4 * tpr) {
        V v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = (ok && u + i * tpr < r.units) ? src[u + i * tpr] : V{};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (u + i * tpr < r.units) dst[u + i * tpr] = v[i];
    }
}

// out[t] = sum_j w[t, j] y[positions[t, j]], fp32 in order of j from +0,
// rounded once to fp16.  Four choices' units are requested before the first
// is used.  Bound by the bytes of y: 8192x2x4096 (195 MB) in 30 us.  A decode
// step is bound by latency: 16x8x4096 is 16 workgroups whose threads walk two
// units and, in each, two batches of four choices one behind the other, 5.3 us
// beside an empty launch's 2.3.  Rows of odd length go 2 bytes at a time, which
// issues eight times the loads: 8192x2x4095 90 us.
template <int U>
__global__ void __launch_bounds__(256) combine_rows_kernel(RowArgs r)
{
    typedef typename RowUnit<U>::type V;
    const int tpr = 1 << r.lanes_log2;
    const int64_t t = row_block() * (256 >> r.lanes_log2) + (threadIdx.x >> r.lanes_log2);
    if (t >= r.T) return;
    const int32_t* pos = r.index + t * r.k;
    const float* w = r.weights ? r.weights + t * r.k : nullptr;
    for (int u = threadIdx.x & (tpr - 1); u < r.units; u += tpr) {
        float acc[U / 2] = {};
        for (int j0 = 0; j0 < r.k; j0 += 4) {
            V v[4];
            float f[4];
            bool ok[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int32_t q = j0 + i < r.k ? pos[j0 + i] : -1;
                ok[i] = (uint32_t)q < (uint32_t)r.P;
                f[i] = (w && ok[i]) ? w[j0 + i] : 1.0f;
                v[i] = ok[i] ? ((const V*)r.x)[(int64_t)q * r.units + u] : V{};
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (ok[i]) {
#pragma unroll
                    for (int e = 0; e < U / 2; ++e) acc[e] += f[i] * HalfVec<U>::at(v[i], e);
                }
        }
        ((V*)r.out)[t * r.units + u] = HalfVec<U>::pack(acc);
    }
}

// The gradient of combine: dy[positions[t, j]] = w[t, j] dout[t] and
// dw[t, j] = <dout[t], y[positions[t, j]]> (fp32, 0 for a dropped choice).
// One wave per token and J choices at a time, so dout[t] is read once for all
// of them, each y row is read once and each dy row written once, and the dot
// needs no LDS, only a sum over the lanes.  A wave requests S units per row
// before it uses one: S follows the row's length (up to 64, 128, more and
// from 512 units on: 1, 2, 4, 8; steps past a row's end cost their
// instructions), J is 2 where two choices of 8 steps are all there is.  y of
// kStreamBytes and more is read without a claim on the caches.  One choice at
// a time and 4 steps, then this: 8192x2x4096 78 and 57 us (335 MB: 5.9 TB/s),
// 16384x4x1024 57 and 51, 8192x4x512 16.3 and 14.2, 16384x8x256 59 and 31;
// 8192x2x512 10.7 and 10.9.  Units of 8, 4 and 2 bytes have one form (J = S =
// 4), bound by the loads' issue: 8192x2x4095 198 us.  Rows of dy that no choice names (rows[p] < 0)
// are set to zero by the same waves.
constexpr int64_t kStreamBytes = 64 << 20;

template <int U, int J, int S, bool STREAM>
__global__ void __launch_bounds__(256) combine_rows_backward_kernel(RowArgs r)
{
    typedef typename RowUnit<U>::type V;
    const int lane = threadIdx.x & 63;
    const int64_t wid = row_block() * 4 + (threadIdx.x >> 6), nw = (int64_t)gridDim.x * gridDim.y * 4;
    for (int64_t t = wid; t < r.T; t += nw) {
        const V* d = (const V*)r.x + t * r.units;
        for (int j0 = 0; j0 < r.k; j0 += J) {
            float dot[J], w[J];
            bool ok[J];
            const V* y[J];
            V* dy[J];
#pragma unroll
            for (int j = 0; j < J; ++j) {
                const int64_t at = t * r.k + j0 + j;
                const int32_t q = j0 + j < r.k ? r.positions[at] : -1;
                ok[j] = (uint32_t)q < (uint32_t)r.P;
                w[j] = (ok[j] && r.weights) ? r.weights[at] : 1.0f;
                y[j] = (const V*)r.y + (int64_t)(ok[j] ? q : 0) * r.units;
                dy[j] = (V*)r.out + (int64_t)(ok[j] ? q : 0) * r.units;
                dot[j] = 0.0f;
            }
            for (int u0 = lane; u0 < r.units; u0 += 64 * S) {
                V dv[S], yv[J][S];
#pragma unroll
                for (int i = 0; i < S; ++i) {
                    const bool in = u0 + 64 * i < r.units;
                    dv[i] = in ? d[u0 + 64 * i] : V{};
#pragma unroll
                    for (int j = 0; j < J; ++j) yv[j][i] = (in && ok[j] && r.dweights) ? row_load<STREAM>(y[j] + u0 + 64 * i) : V{};
                }
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (!ok[j]) continue;
#pragma unroll
                    for (int i = 0; i < S; ++i) {
                        float g[U / 2];
#pragma unroll
                        for (int e = 0; e < U / 2; ++e) {
                            const float de = HalfVec<U>::at(dv[i], e);
                            dot[j] += de * HalfVec<U>::at(yv[j][i], e);
                            g[e] = w[j] * de;
                        }
                        if (u0 + 64 * i < r.units) dy[j][u0 + 64 * i] = HalfVec<U>::pack(g);
                    }
                }
            }
            if (r.dweights) {
#pragma unroll
                for (int j = 0; j < J; ++j) {
#pragma unroll
                    for (int x = 32; x > 0; x >>= 1) dot[j] += __shfl_xor(dot[j], x);
                    if (lane == 0 && j0 + j < r.k) r.dweights[t * r.k + j0 + j] = dot[j];
                }
            }
        }
    }
    for (int64_t p0 = wid * 64; p0 < r.P; p0 += nw * 64) {
        const int64_t p = p0 + lane;
        uint64_t none = __ballot(p < r.P && (uint32_t)r.index[p < r.P ? p : p0] >= (uint32_t)r.T);
        while (none) {
            V* dy = (V*)r.out + (p0 + __ffsll((unsigned long long)none) - 1) * r.units;
            for (int u = lane; u < r.units; u += 64) dy[u] = V{};
            none &= none - 1;
        }
    }
}

}  // namespace gsr
