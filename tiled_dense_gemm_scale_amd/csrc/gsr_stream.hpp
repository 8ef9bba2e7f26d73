// gsr_stream.hpp -- products of a few rows with weights read once: a wave's
// share of C (16 rows x CB columns) over a run of K, operands from memory
// straight into registers.
//
// Such products are bound by the weights' bytes, so nothing stands between their
// loads and the matrix cores: no LDS, no barrier (rows of A pass through the wave's
// own LDS where a tile has more than one, stream_turn).  A wave's 64 lanes hold an
// MFMA 16x16x32 operand as 16 columns x 4 runs of 8 values of k.  With weights
// in rows of N (k-major) lane (l, g) = (lane % 16, lane / 16) reads the CPL
// columns c .. c + CPL - 1 of the rows 8g .. 8g + 7 of a step of 32 rows, which
// is one operand for each of its columns once the 8 x CPL block is transposed
// in registers (byte permutes, half an instruction per value); the 16 lanes of
// a group so read 16 CPL consecutive columns of a row.  4-bit codes hold 8
// values of k in a word and need no transpose (gsr_w4.hpp).
//
// Waves of a workgroup take runs of K of their own and add their sums through
// LDS in wave order.  One workgroup of eight waves has a CU to itself: its ring of
// two units needs 150 to 244 registers a lane (and the few-token kernels keep 24 to 68
// scalar values in lanes of them, which the scalar registers have no room for).
//
// Columns past N: a lane whose columns would pass N is moved back to end at N,
// so its sums are those of columns that its neighbour has too, the same bits,
// and no load needs a mask; matrices of fewer than CPL columns are read value
// by value.  Rows past K read as zeros on both sides, so whatever lies behind
// the matrix adds nothing.  Rows of C are independent of one another in the
// matrix cores (infinities and NaN stay in their row and column).
#pragma once

#include "gsr_kernels.hpp"

namespace gsr {

// Vectors at addresses of any even (words: any 4-byte, bytes: any) alignment;
// the hardware takes global loads at every address.
typedef u32x4 u32x4_at2 __attribute__((aligned(2)));
typedef u32x4 u32x4_at4 __attribute__((aligned(4)));
typedef u32x2 u32x2_at2 __attribute__((aligned(2)));
typedef uint32_t u32_at1 __attribute__((aligned(1)));

__device__ __forceinline__ uint32_t join16(uint16_t lo, uint16_t hi) { return (uint32_t)lo | ((uint32_t)hi << 16); }

// eight fp16 values at p of which `n` exist (zeros for the others)
__device__ __forceinline__ u32x4 load8_first(const uint16_t* p, int n)
{
    u32x4 v = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint16_t lo = 2 * i < n ? p[2 * i] : (uint16_t)0, hi = 2 * i + 1 < n ? p[2 * i + 1] : (uint16_t)0;
        v[i] = join16(lo, hi);
    }
    return v;
}

__device__ __forceinline__ f32x4 add4(f32x4 a, f32x4 b) { return f32x4{a[0] + b[0], a[1] + b[1], a[2] + b[2], a[3] + b[3]}; }

__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c)
{
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(half8, a), __builtin_bit_cast(half8, b), c, 0, 0, 0);
}

constexpr int kStep = 32;  // k per MFMA

// Eight fp16 values at byte `off` of a buffer whose base lies on a dword: one
// 16-byte load at the dword below, one of the dword behind, shifted together
// (a 16-byte load at an odd element goes out at about a lane per clock, one on a
// dword whole).
__device__ __forceinline__ u32x4 load8_shifted(__amdgpu_buffer_rsrc_t rs, uint32_t off)
{
    const uint32_t o = off & ~3u, sh = (off & 2u) << 3;
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0);
    const uint32_t w = __builtin_amdgcn_raw_buffer_load_b32(rs, o + 16u, 0, 0);
    return u32x4{__builtin_amdgcn_alignbit(v[1], v[0], sh), __builtin_amdgcn_alignbit(v[2], v[1], sh),
                 __builtin_amdgcn_alignbit(v[3], v[2], sh), __builtin_amdgcn_alignbit(w, v[3], sh)};
}

// A descriptor of `bytes` bytes from `at`, from the dword that holds its first
// to the one that holds its last; what `at` lies behind that base.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t dword_rsrc(const void* at, uint64_t bytes, uint32_t& behind)
{
    behind = (uint32_t)(uintptr_t)at & 2u;
    return make_rsrc((const uint8_t*)at - behind, (uint32_t)min((bytes + behind + 3u) & ~(uint64_t)3, (uint64_t)0x7ffffffcu));
}

// A lane's place in the loads of A: lane t reads the eight values 8 c .. 8 c + 7
// of the t / 4-th of 16 rows, c = t % 4 ^ t / 16, so that four lanes next to each
// other read 64 bytes next to each other.  (As the matrix cores take A, row t % 16
// and run t / 16, each lane's 16 bytes are an access of their own, four in five of
// all: 64 tokens x 2 of 8 experts in 4 bits 154 us so, 138 with this step.)
// stream_turn brings them into that order through the wave's LDS; with that c no
// two lanes meet in a bank.  A tile of one row needs neither (one token x 2 of 8
// experts in 4 bits 39.0 us turned, 37.7 not).
__device__ __forceinline__ int stream_row() { return (int)(threadIdx.x & 63) >> 2; }
__device__ __forceinline__ int stream_run() { return (int)(threadIdx.x & 3) ^ (int)((threadIdx.x >> 4) & 3); }

__device__ __forceinline__ void wave_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

template <int STEPS>
__device__ __forceinline__ void stream_turn(u32x4 (&a)[STEPS], float* slice)
{
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
    u32x4* s = (u32x4*)slice;
#pragma unroll
    for (int i = 0; i < STEPS; ++i) s[64 * i + lane] = a[i];
    wave_fence();
#pragma unroll
    for (int i = 0; i < STEPS; ++i) a[i] = s[64 * i + 4 * l + (g ^ (l >> 2))];
    wave_fence();
}

// The row of A that a lane reads, of a table of less than 2^31 bytes.  Rows past the
// last are that one again, whose sums nobody takes, and loads behind the table are
// zeros: no load is masked, and lanes with one address are one access.  DW: every
// row starts on a dword.  A table can also hold values as two halves, the value
// rounded and 2^11 times what that lost (stream_split); each of a row's halves is
// `wide` values long, zeros at the end, the second behind the first, and in the
// order of k that the stream multiplies in.
template <bool DW>
struct StreamRows {
    __amdgpu_buffer_rsrc_t rs;
    uint32_t off;
    int wide = 0;
    int run;   // the lane's place in a step's 32 values, in eights
    bool turn;

    // `count` rows of a tile are looked at (the same in the whole wave)
    __device__ __forceinline__ StreamRows(const uint16_t* table, uint64_t bytes, int count) : turn(count > 1)
    {
        rs = dword_rsrc(table, bytes, off);
        run = turn ? stream_run() : (int)(threadIdx.x & 63) >> 4;
    }
    __device__ __forceinline__ void row(uint32_t at) { off += 2u * at; }  // `at` values into the table
    __device__ __forceinline__ u32x4 load(int k) const
    {
        const uint32_t o = off + 2u * (uint32_t)k;
        if constexpr (DW) return __builtin_amdgcn_raw_buffer_load_b128(rs, o, 0, 0);
        else return load8_shifted(rs, o);
    }
};

// v as two fp16 values, hi + lo / 2048: within 2^-22 of v, or 2^-35 where that is
// more (|v| below 2^-13).  fp16's least step is 2^-24, so the rest is kept 2^11
// larger, the most that the rest of the largest value, 16, leaves room for; its own
// rounding is then 2^-36.  hi of a v that is not zero is not zero either (lo gives
// back the difference, rounded once more on the way), so that v keeps its sign beside
// an infinite weight; past fp16 hi is an infinity, alone.
constexpr float kRest = 2048.0f;
struct StreamHalves {
    uint16_t hi, lo;
};
__device__ __forceinline__ StreamHalves stream_split(float v)
{
    _Float16 hi = (_Float16)v;
    if (hi == (_Float16)0.0f && v != 0.0f) hi = __builtin_bit_cast(_Float16, (uint16_t)(v < 0.0f ? 0x8001u : 1u));
    const float rest = (v - (float)hi) * kRest;
    return StreamHalves{__builtin_bit_cast(uint16_t, hi),
                        __builtin_bit_cast(uint16_t, (_Float16)(fabsf((float)hi) <= 65504.0f ? rest : 0.0f))};
}

// The first n of eight values, zeros for the others.
__device__ __forceinline__ u32x4 first8(u32x4 v, int n)
{
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = n >= 2 * i + 2 ? v[i] : n == 2 * i + 1 ? v[i] & 0xffffu : 0u;
    return v;
}

// A descriptor of the rows k0 and on of a matrix of `rows` rows of `pitch` bytes
// (whole dwords): loads behind the last row are zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_rsrc(const void* base, int rows, int k0, uint32_t pitch)
{
    const uint64_t left = (uint64_t)max(rows - k0, 0) * pitch;  // none: nothing is read
    return make_rsrc((const uint8_t*)base + (size_t)k0 * pitch, (uint32_t)min(left, (uint64_t)0x7fffffffu));
}

// The column where lane l's CPL columns of the block from n0 start.
template <int CPL>
__device__ __forceinline__ int stream_column(int n0, int l, int N)
{
    const int c = n0 + CPL * l;
    return N >= CPL ? min(c, N - CPL) : c;
}

// v[j]: column c + j of lane l (its 16 lanes' columns), rows 4 g + r.
template <int CT>
struct StreamSums {
    f32x4 v[CT];
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int j = 0; j < CT; ++j) v[j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
};

// multiply(b, i) for n > 0 units in turn, the next one's loads in flight: load(b,
// i) is called for the unit past the last too, and has to be one that reads
// nothing new there, so that no wait depends on which way a branch went.  A third
// unit gained nothing when it was tried (fp16 one token x 2 of 8 experts 77 us either
// way; 16 x 11008 x 4096 in 4 bits 11.3 us with two, 12.5 with three): with two,
// eight waves have the 46 KB per CU in flight that the card's rate times its latency
// comes to.
template <class Batch, class Load, class Multiply>
__device__ __forceinline__ void stream_ring(int n, Load&& load, Multiply&& multiply)
{
    Batch b[2];
    load(b[0], 0);
    for (int i = 0;; i += 2) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            load(b[j ^ 1], i + j + 1);
            multiply(b[j], i + j);
            if (i + j + 1 >= n) return;
        }
    }
}

// ---- fp16 weights ------------------------------------------------------------
struct HalfMatrix {
    const uint16_t* b;  // K x N
};

// DW: every row starts on a dword (N even, b on one), and every row of A.
// SPLIT: A in halves.
template <bool DW, bool SPLIT>
struct HalfStream {
    static __device__ __forceinline__ int order(int k) { return k; }  // where k lies in a row of halves
    static constexpr int CPL = 8, CB = 16 * CPL, UNIT = kStep;  // UNIT: k of the smallest run
    typedef StreamSums<CPL> Sums;
    typedef StreamRows<DW> Rows;

    struct Step {
        u32x4 b[8];
        u32x4 a[SPLIT ? 2 : 1];
    };
    struct Place {
        const uint16_t* b;
        float* slice;
        int K, N, c, g;
        uint32_t off[8];  // bytes from a step's first row
    };

    // Unit u of a run of units before `end` (from there on nothing is read anew).
    __device__ static __forceinline__ void load(Step& s, const Place& p, const Rows& rows, int u, int end)
    {
        const int k0 = min(u, end - 1) * kStep;
        if constexpr (DW) {
            const __amdgpu_buffer_rsrc_t rs = rows_rsrc(p.b, u < end ? p.K : 0, k0, 2u * (uint32_t)p.N);
#pragma unroll
            for (int i = 0; i < 8; ++i) s.b[i] = __builtin_amdgcn_raw_buffer_load_b128(rs, p.off[i], 0, 0);
        } else {
            uint32_t behind;
            const __amdgpu_buffer_rsrc_t rs =
                dword_rsrc(p.b + (size_t)k0 * p.N, u < end ? (uint64_t)(p.K - k0) * (uint32_t)p.N * 2u : 0u, behind);
#pragma unroll
            for (int i = 0; i < 8; ++i) s.b[i] = load8_shifted(rs, p.off[i] + behind);
        }
        s.a[0] = rows.load(k0 + 8 * rows.run);
        if constexpr (SPLIT) s.a[1] = rows.load(rows.wide + k0 + 8 * rows.run);
        __builtin_amdgcn_sched_barrier(0);
    }

    // Zeros for what lies past K on both sides (behind a row of A lies the next
    // one, and the last row of B may share its last dword with other values).
    __device__ static __forceinline__ void cut(Step& s, const Place& p, const Rows& rows, int k0)
    {
        const int n = p.K - k0 - 8 * p.g;
#pragma unroll
        for (int h = 0; h < (SPLIT ? 2 : 1); ++h) s.a[h] = first8(s.a[h], SPLIT ? rows.wide - k0 - 8 * p.g : n);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i >= n) s.b[i] = u32x4{0u, 0u, 0u, 0u};
    }

    __device__ static __forceinline__ void multiply(Step& s, const Place& p, const Rows& rows, int u, Sums& acc, Sums& low)
    {
        if (rows.turn) stream_turn(s.a, p.slice);
        if ((u + 1) * kStep > p.K) cut(s, p, rows, u * kStep);
#pragma unroll
        for (int d = 0; d < 4; ++d) {  // columns 2d and 2d + 1
            u32x4 even, odd;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                even[e] = pack_lo(s.b[2 * e][d], s.b[2 * e + 1][d]);
                odd[e] = pack_hi(s.b[2 * e][d], s.b[2 * e + 1][d]);
            }
            acc.v[2 * d] = mfma16(s.a[0], even, acc.v[2 * d]);
            acc.v[2 * d + 1] = mfma16(s.a[0], odd, acc.v[2 * d + 1]);
            if constexpr (SPLIT) {
                low.v[2 * d] = mfma16(s.a[1], even, low.v[2 * d]);
                low.v[2 * d + 1] = mfma16(s.a[1], odd, low.v[2 * d + 1]);
            }
            __builtin_amdgcn_sched_barrier(0);  // a pair's values live no longer than it
        }
    }

    // acc += A[:, k] B[k, :] over the units u0 <= u < u1 of 32 k; slice: this wave's
    // LDS, 16 x CB floats
    __device__ static __forceinline__ void run(const HalfMatrix& m, int K, int N, int n0, const Rows& rows, int u0, int u1,
                                               float* slice, Sums& acc)
    {
        const int lane = threadIdx.x & 63;
        Place p;
        p.b = m.b;
        p.slice = slice;
        p.K = K;
        p.N = N;
        p.g = lane >> 4;
        p.c = stream_column<CPL>(n0, lane & 15, N);
#pragma unroll
        for (int i = 0; i < 8; ++i) p.off[i] = 2u * ((uint32_t)(8 * p.g + i) * (uint32_t)N + (uint32_t)p.c);
        if (u0 >= u1) return;
        Sums low;
        low.clear();
        if (N >= CPL) {
            stream_ring<Step>(
                u1 - u0, [&](Step& s, int i) { load(s, p, rows, u0 + i, u1); },
                [&](Step& s, int i) { multiply(s, p, rows, u0 + i, acc, low); });
        }
#pragma unroll 1
        for (int u = N >= CPL ? u1 : u0; u < u1; ++u) {  // fewer columns than a lane's: value by value
            Step s{};
#pragma unroll 1
            for (int i = 0; i < 8; ++i) {
                const int k = u * kStep + 8 * p.g + i;
                const u32x4 v = load8_first(p.b + (size_t)min(k, K - 1) * N + p.c, k < K ? N - p.c : 0);
#pragma unroll
                for (int x = 0; x < 8; ++x) s.b[x] = x == i ? v : s.b[x];
            }
            s.a[0] = rows.load(u * kStep + 8 * rows.run);
            if constexpr (SPLIT) s.a[1] = rows.load(rows.wide + u * kStep + 8 * rows.run);
            multiply(s, p, rows, u, acc, low);
        }
        // The second halves' sums apart: where a weight is infinite the first
        // halves' alone are the formula's (zero times infinity, and halves of
        // two signs, would make NaN of them).
        if constexpr (SPLIT)
#pragma unroll
            for (int j = 0; j < CPL; ++j)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc.v[j][r] = fmaf(fabsf(acc.v[j][r]) < __builtin_inff() ? low.v[j][r] : 0.0f, 1.0f / kRest, acc.v[j][r]);
    }
};

// ---- the sum over waves ---------------------------------------------------------
// Each of a workgroup's waves has a slice of LDS for its sums, 16 rows x CB
// columns, row-major.
constexpr int kStreamWaves = 8, kStreamThreads = kWave * kStreamWaves;

template <int CPL>
__device__ __forceinline__ void stream_put(float* slice, const StreamSums<CPL>& acc)
{
    const int lane = threadIdx.x & 63, l = lane & 15, g = lane >> 4;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        f32x4* to = (f32x4*)(slice + (4 * g + r) * 16 * CPL + CPL * l);
#pragma unroll
        for (int j = 0; j < CPL / 4; ++j)
            to[j] = f32x4{acc.v[4 * j][r], acc.v[4 * j + 1][r], acc.v[4 * j + 2][r], acc.v[4 * j + 3][r]};
    }
}

// Positions 4q .. 4q + 3 of row m, summed over `waves` slices in order from +0.
template <int CPL>
__device__ __forceinline__ f32x4 stream_sum(const float* slices, int waves, int m, int q)
{
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int w = 0; w < waves; ++w) s = add4(s, *(const f32x4*)(slices + (w * 16 + m) * 16 * CPL + 4 * q));
    return s;
}

// The column of position 4q of the block from n0 (three more lie behind it; those
// from N on are none), or -1 where the position or its lane lies past N.
template <int CPL>
__device__ __forceinline__ int stream_position(int n0, int q, int N)
{
    const int l = 4 * q / CPL, col = stream_column<CPL>(n0, l, N) + 4 * q % CPL;
    return n0 + CPL * l < N && col < N ? col : -1;
}

// Four fp16 values of a row of N from column `col` on (zeros past N), and back;
// one access where N is a multiple of four, as `col` is then too.
__device__ __forceinline__ f32x4 half4_at(const uint16_t* row, int col, int N)
{
    u32x2 w = {0u, 0u};
    if ((N & 3) == 0) {
        w = *(const u32x2_at2*)(row + col);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < N) w[i / 2] |= (uint32_t)row[col + i] << (16 * (i & 1));
    }
    const half4 h = __builtin_bit_cast(half4, w);
    return f32x4{(float)h[0], (float)h[1], (float)h[2], (float)h[3]};
}
__device__ __forceinline__ void put_half4(uint16_t* row, int col, int N, f32x4 v)
{
    const half4 h = {(_Float16)v[0], (_Float16)v[1], (_Float16)v[2], (_Float16)v[3]};
    const u32x2 w = __builtin_bit_cast(u32x2, h);
    if ((N & 3) == 0) {
        *(u32x2_at2*)(row + col) = w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (col + i < N) row[col + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
}

// ---- sums that meet in a workspace ---------------------------------------------------
// Written and read at device scope (the L2 of an XCD is not coherent with the
// others'): relaxed atomics at agent scope write through and do not take a
// stale line.  Whoever counts last has every other's sums: each wave waits for
// its stores before the barrier in front of the count, and reads only after the
// count has returned.
__device__ __forceinline__ void meet_store(float* to, f32x4 v)
{
    const u32x4 w = __builtin_bit_cast(u32x4, v);
    uint64_t* d = (uint64_t*)to;
    __hip_atomic_store(d, w[0] | (uint64_t)w[1] << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __hip_atomic_store(d + 1, w[2] | (uint64_t)w[3] << 32, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The sum of `n` quads `stride` values apart, in order from +0, eight in flight.
__device__ __forceinline__ f32x4 meet_sum(const float* from, int n, size_t stride)
{
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    for (int g = 0; g < n; g += 8) {
        uint64_t v[8][2];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint64_t* p = (const uint64_t*)(from + (size_t)min(g + i, n - 1) * stride);
            v[i][0] = __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            v[i][1] = __hip_atomic_load(p + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (g + i < n)
                s = add4(s, __builtin_bit_cast(f32x4, u32x4{(uint32_t)v[i][0], (uint32_t)(v[i][0] >> 32), (uint32_t)v[i][1],
                                                            (uint32_t)(v[i][1] >> 32)}));
    }
    return s;
}

// Counts this workgroup in; true in the one that completes `all`, whose counter
// it puts back to zero.
__device__ __forceinline__ bool meet_last(uint32_t* count, uint32_t all, int* flag)
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's sums have reached device scope
    __syncthreads();
    if (threadIdx.x == 0) {
        const uint32_t before = __hip_atomic_fetch_add(count, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        *flag = (int)(before == all - 1u);
        if (before == all - 1u) __hip_atomic_store(count, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    __syncthreads();
    return *flag != 0;
}

// Every workspace starts with 128 counters.
constexpr int kMeetCounters = 128;
constexpr int64_t kMeetBytes = 4 * kMeetCounters;

// act(y), SiLU = y / (1 + exp(-y)) too
enum : int { kActSilu = 3 };
__device__ __forceinline__ float stream_activate(float y, int act)
{
    if (act == kActSilu) return y * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.4426950408889634f * y));
    return activate(y, act);
}

__device__ __forceinline__ float half_at(const uint16_t* p) { return (float)__builtin_bit_cast(_Float16, *p); }
__device__ __forceinline__ uint16_t to_half(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

}  // namespace gsr
