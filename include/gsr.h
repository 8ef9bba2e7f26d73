/*
 * gsr.h -- C ABI of the fused fp16 GEMM + scale + ReLU library for AMD
 * Instinct MI355X (gfx950).
 *
 * The operation (PKUHPC scow-tutorial "Tutorial14: 使用TileLang语言编写attention
 * 算子", section 3 "算子介绍", display formula and symbol list; the kernel
 * listing in section 2 "编写算子" fixes the types and the epilogue order):
 *
 *     C[m,n] = ReLU( alpha * sum_{k<K} A[m,k] * B[k,n] ),  ReLU(x) = max(x, 0)
 *
 *   A  M x K, IEEE binary16, row-major (leading dimension K)
 *   B  K x N, IEEE binary16, row-major (leading dimension N)
 *   C  M x N, IEEE binary16, row-major (leading dimension N), written once
 *   alpha  binary32 scalar
 * Products are accumulated in binary32; the scale and the max(., 0) are applied
 * to the binary32 sum in registers and the result is narrowed to binary16 with
 * round-to-nearest-even on the single store.  Non-positive results are +0.
 *
 * Ownership and ordering.  A, B and C are device pointers owned by the caller
 * (any allocation the HIP runtime can address from the current device).  The
 * library allocates nothing and keeps no per-call state (the entry points
 * with a workspace keep theirs in the caller's workspace); it only enqueues
 * kernels on `stream` (a hipStream_t; NULL means the null stream) and returns
 * before they finish.  The caller synchronises.  Calls are thread-safe.
 *
 * Error behaviour.  Arguments are checked on the host before anything is
 * enqueued; a nonzero status means nothing was launched (except
 * GSR_ERROR_LAUNCH, which reports a failed launch).  No status aborts the
 * process.
 */
#ifndef GSR_H_
#define GSR_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum gsr_status {
    GSR_SUCCESS = 0,
    /* a dimension < 0; a null or odd-address pointer where the extent is
     * nonzero; C's byte range overlapping A's or B's; alpha not finite */
    GSR_ERROR_INVALID_VALUE = 1,
    /* a dimension >= 2^31, or a matrix of 2^31 bytes or more (the kernels
     * use 32-bit byte offsets), or so many tiles that a launch would have
     * 2^32 threads */
    GSR_ERROR_TOO_LARGE = 2,
    GSR_ERROR_NO_DEVICE = 3,          /* no HIP device is visible */
    GSR_ERROR_UNSUPPORTED_DEVICE = 4, /* the current device is not gfx950 */
    GSR_ERROR_LAUNCH = 5,             /* the runtime rejected the launch */
    GSR_ERROR_INVALID_CONFIG = 6      /* gemm_scale_relu_ex: unknown config id */
};

/* Activation of the epilogue variants. */
enum gsr_activation {
    GSR_ACT_RELU = 0, /* max(v, 0); non-positive results are +0 */
    GSR_ACT_GELU = 1, /* v/2 * (1 + tanh(sqrt(2/pi) * (v + 0.044715 v^3))) */
    GSR_ACT_NONE = 2, /* v itself */
    GSR_ACT_SILU = 3  /* v / (1 + exp(-v)); gsr_expert_mlp_few only */
};

/* One compiled tile configuration.  A workgroup of waves_m*waves_n wave64s
 * owns a block_m x block_n tile of C and walks K in steps of block_k through
 * `stages` LDS buffers (0 or 1: two per operand; configurations 28, 29 and
 * 31: two for A, three for B; 2 or more: a ring of that many buffers per
 * operand); each wave owns a (block_m/waves_m) x (block_n/waves_n) sub-tile
 * (configurations 31 and 32 add waves_m * waves_n waves that only copy
 * operands into LDS).  Configurations 25, 28, 29, 31 and 32 build that
 * sub-tile from 16x16x32 fp16 MFMAs, all others from 32x32x16 fp16 MFMAs.  (The K-split kinds, block_k
 * 128 with waves 1 x 1, give every wave the whole tile and a share of each
 * K-step instead.)  group_m is the number of tile rows in one group of the
 * grouped launch order; xcd_remap picks how workgroup ids map to tiles: 0 the
 * grouped order on the ids as dispatched, 1 the same on ids regrouped so that
 * neighbouring tiles run on the same XCD, 2 chip-wide rounds of 16 x 16 tiles
 * with a 4 x 8 part per XCD (grids whose tile rows and columns are multiples
 * of 16; others use 1; group_m unused).  Ids are stable across library
 * versions and not contiguous: gsr_config_ids lists the compiled ones. */
typedef struct gsr_config {
    int32_t id;
    int32_t block_m, block_n, block_k;
    int32_t waves_m, waves_n;
    int32_t stages;
    int32_t group_m;
    int32_t xcd_remap;
    int32_t lds_bytes;
} gsr_config;

/* The fused operation (the tutorial's kernel call: A, B, C, scale).
 * M, N, K >= 0.  M == 0 or N == 0: success, nothing enqueued.  K == 0: every
 * output is the empty sum, C is filled with +0.  Any pointer alignment of at
 * least 2 bytes is accepted; 16-byte aligned A and B with K and N multiples
 * of 8 take the 128-bit vector path (C written in the widest stores its own
 * alignment allows), anything else an element-wise path (a register-staged
 * kernel of the same tile, or of a 64x64 tile for the K-split kinds, reading
 * each operand in the widest unit its alignment allows).  Returns a gsr_status. */
int gemm_scale_relu(int64_t M, int64_t N, int64_t K,
                    const void* A, const void* B, void* C,
                    float alpha, void* stream);

/* As gemm_scale_relu with a forced tile configuration (an id from
 * gsr_config_ids; -1 = the selector's choice).  For sweeps and tests. */
int gemm_scale_relu_ex(int64_t M, int64_t N, int64_t K,
                       const void* A, const void* B, void* C,
                       float alpha, void* stream, int32_t config_id);

/* The epilogue variants (the aikraft.ru TileLang guide, section 4 "Слияние
 * эпилогов: GEMM + Bias + GELU": a bias and an exponent-based GELU applied to
 * the matmul result in registers before the single store):
 *
 *     C[m,n] = act( alpha * sum_{k<K} A[m,k] * B[k,n] + bias[n] )
 *
 *   bias  NULL, or N IEEE binary16 values on the device (one per output
 *         column, at least 2-byte aligned; 8-byte alignment keeps the 128-bit
 *         path), read-only, must not overlap C
 *   activation  a gsr_activation; GELU is the tanh form, evaluated in binary32
 *         as v / (1 + exp(-2u)), u = sqrt(2/pi) (v + 0.044715 v^3)
 * The sum, the scale, the bias and the activation are binary32; one
 * round-to-nearest-even narrowing to binary16.  With bias == NULL and
 * GSR_ACT_RELU this is exactly gemm_scale_relu; the guide's GEMM + Bias + GELU
 * is alpha = 1, GSR_ACT_GELU.  K == 0 gives act(bias[n]) (+0 without a bias).
 * Layout, alignment, ownership and errors as gemm_scale_relu; in addition
 * GSR_ERROR_INVALID_VALUE for an unknown activation, an odd bias address or
 * a bias overlapping C. */
int gemm_scale_bias_act(int64_t M, int64_t N, int64_t K,
                        const void* A, const void* B, const void* bias, void* C,
                        float alpha, int32_t activation, void* stream);

/* As gemm_scale_bias_act with a forced tile configuration (-1 = selector). */
int gemm_scale_bias_act_ex(int64_t M, int64_t N, int64_t K,
                           const void* A, const void* B, const void* bias, void* C,
                           float alpha, int32_t activation, void* stream, int32_t config_id);

/* As gemm_scale_bias_act with an explicit launch: cfg->id picks the compiled
 * tile configuration; cfg->group_m (1..4096, tile rows per group of the
 * launch order) and cfg->xcd_remap (0, 1 or 2) override that configuration's
 * launch order; the other fields are ignored.  The launch order changes only
 * which tiles run together, never a tile's arithmetic, so results are bit
 * for bit those of gemm_scale_bias_act_ex with the same id.  For tuning
 * sweeps.  GSR_ERROR_INVALID_CONFIG for an out-of-range field. */
int gemm_scale_bias_act_cfg(int64_t M, int64_t N, int64_t K,
                            const void* A, const void* B, const void* bias, void* C,
                            float alpha, int32_t activation, void* stream, const gsr_config* cfg);

/* The same operations with a workspace, so that K can be split across
 * workgroups.  The pages do not describe splitting K: the sum is still the
 * one the PKUHPC tutorial defines (section 3 display formula), taken over
 * runs of K and added, and the context is the aikraft.ru guide's section 3
 * (no schedule is best for every size) and the TileKernels article's section
 * one (memory bandwidth utilisation as the measure of a memory-bound
 * product).  It serves shapes whose output has too few tiles of the K-split
 * kinds (configurations 21 and 22) to occupy the chip, such as a few rows
 * against a 4096-wide weight: each tile's
 * K-steps are cut into `parts` runs, one workgroup each, whose fp32 sums meet
 * in the workspace, and the workgroup of a tile that finishes last adds them
 * in part order, applies the epilogue and stores C.  The sum of a part is
 * that of the unsplit kernel over its K range, so results differ from the
 * unsplit call only by the order of fp32 additions.
 *
 *   workspace  device memory owned by the caller, 16-byte aligned, not
 *              overlapping A, B, C or the bias.  Its first bytes hold one
 *              32-bit arrival counter per tile and must be zero before the
 *              first call (allocate it zero-filled); every call leaves them
 *              zero again (the first 512 bytes in all, what calls of up to
 *              128 tiles count in), so the same workspace serves any number
 *              of calls in stream order, of any shapes as long as none is
 *              forced to split over more than 128 tiles after another has
 *              split over fewer.  Calls that may run at the same time (other
 *              streams, other threads) need workspaces of their own.
 *   workspace_bytes  its size; gsr_workspace_bytes gives what the library's
 *              choice needs (at most 4 MiB + 512 bytes for any shape)
 *   splits     0: the library's choice (shapes of at most 128 such tiles
 *              and at least 32 K-steps of 128 whose unsplit call would not
 *              already stream near the read ceiling: up to four parts, at
 *              most one workgroup per CU and eight K-steps per part; fewer
 *              parts when the workspace is smaller, none without one);
 *              n >= 1: at most n parts (never
 *              more than one per K-step), GSR_ERROR_INVALID_VALUE if the
 *              workspace cannot hold them, GSR_ERROR_INVALID_CONFIG for n > 1
 *              with a configuration that cannot split.  1..16.
 * A call that does not split (other configurations, the element-wise path,
 * parts = 1) ignores the workspace.  Otherwise as gemm_scale_bias_act_ex and
 * gemm_scale_relu; GSR_ERROR_INVALID_VALUE also for a misaligned or
 * overlapping workspace, a negative size or splits outside 0..16. */
int gemm_scale_bias_act_ws(int64_t M, int64_t N, int64_t K,
                           const void* A, const void* B, const void* bias, void* C,
                           float alpha, int32_t activation,
                           void* workspace, int64_t workspace_bytes,
                           void* stream, int32_t config_id, int32_t splits);

/* gemm_scale_relu with a workspace: the selector's configuration and the
 * library's split. */
int gemm_scale_relu_ws(int64_t M, int64_t N, int64_t K,
                       const void* A, const void* B, void* C, float alpha,
                       void* workspace, int64_t workspace_bytes, void* stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc):
 * gemm_scale_bias_act_ws with the workspace taken from a scratch array that
 * the library keeps in every device's memory (4 MiB + 512 bytes per device,
 * present from the time the library's code object is loaded until the
 * process ends; its address is looked up once per device, on the first call
 * with that device current, so under graph capture make one call outside
 * the capture first).  The call itself allocates nothing.  Every call
 * on one device shares that device's array: calls that may overlap on one
 * device (other streams, other threads, other libraries' copies excepted)
 * race, and their results and the array's arrival counters are then
 * undefined.  Calls in stream order are safe: the counters start at zero and
 * every call leaves them zero.  A split that needs more than the array holds
 * (only a forced `splits` can) is GSR_ERROR_TOO_LARGE, with nothing
 * enqueued; the library's own choice always fits.  GSR_ERROR_LAUNCH also
 * when the runtime cannot give the array's address.  Otherwise as
 * gemm_scale_bias_act_ws. */
int gemm_scale_bias_act_noalloc(int64_t M, int64_t N, int64_t K,
                                const void* A, const void* B, const void* bias, void* C,
                                float alpha, int32_t activation,
                                void* stream, int32_t config_id, int32_t splits);

/* Workspace bytes the library's split needs for an M x N x K call on the
 * 128-bit path (the selector's or the tuning table's configuration); 0 when
 * that call does not split, -1 for a negative dimension.  Host only. */
int64_t gsr_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* ---- rows sorted by group and back ------------------------------------------
 * The rows around a product whose weights differ from row to row (routed
 * experts): T tokens, each with k choices among `groups` groups, give n = T k
 * slots; slot t k + j is token t's choice j.  A slot whose id is outside
 * [0, groups) is dropped.  Rows of fp16 values are row-major and contiguous,
 * `width` values each; any 2-byte alignment is accepted and the widest unit
 * (16, 8, 4 or 2 bytes) that the addresses and the width allow is used.
 * Counts are below 2^31 and widths below 2^30 (GSR_ERROR_TOO_LARGE), matrices may be larger than
 * 2^31 bytes.  Outputs must not overlap inputs or each other
 * (GSR_ERROR_INVALID_VALUE).  No kernel here uses atomics on memory: equal
 * inputs give equal bits.  Ownership, streams and errors as above. */

/* Slots sorted by group, in slot order within a group:
 *   ids        T x k ids, row-major, of id_bytes = 4 or 8 bytes each, signed
 *   offsets    groups + 1 values: group e has the sorted rows offsets[e] ..
 *              offsets[e + 1] - 1; offsets[groups] is the count of kept slots
 *   rows       n values: the token of each sorted row, -1 from
 *              offsets[groups] on
 *   positions  T x k values: the sorted row of each slot, -1 for a dropped one
 * groups is 1..1024.  workspace: gsr_group_workspace_bytes(T, k, groups) bytes
 * (0 up to 8192 slots), 16-byte aligned, any content, and one per call that
 * may run at the same time; GSR_ERROR_INVALID_VALUE if smaller.  T = 0 or
 * k = 0 writes the offsets only (zeros). */
int gsr_group_rows(int64_t tokens, int64_t k, int64_t groups, const void* ids, int32_t id_bytes,
                   int32_t* offsets, int32_t* rows, int32_t* positions,
                   void* workspace, int64_t workspace_bytes, void* stream);

/* The bytes gsr_group_rows needs; -1 for arguments it rejects.  Host only. */
int64_t gsr_group_workspace_bytes(int64_t tokens, int64_t k, int64_t groups);

/* out[p] = x[rows[p]] for p < rows_out; zeros where rows[p] is outside
 * [0, rows_in).  An index may occur any number of times. */
int gsr_gather_rows(int64_t rows_out, int64_t rows_in, int64_t width,
                    const void* x, const int32_t* rows, void* out, void* stream);

/* out[t] = sum over j of weights[t, j] * y[positions[t, j]], j ascending, in
 * binary32, one narrowing to binary16; choices whose position is outside
 * [0, rows_in) have no term (whatever lies in y).  weights: T x k binary32,
 * or NULL for ones, which makes this the gradient of gsr_gather_rows. */
int gsr_combine_rows(int64_t tokens, int64_t k, int64_t rows_in, int64_t width,
                     const void* y, const int32_t* positions, const float* weights,
                     void* out, void* stream);

/* The gradient of gsr_combine_rows for dout (T x width):
 *   dy        (rows_in x width): weights[t, j] * dout[t] in row
 *             positions[t, j]; zeros in the rows p with rows[p] outside
 *             [0, tokens).  With the rows and positions of gsr_group_rows
 *             every row is written; rows that neither names stay as they were.
 *             Positions inside [0, rows_in) must be distinct.
 *   dweights  (T x k binary32): the products <dout[t], y[positions[t, j]]>,
 *             0 for a choice without a position.
 * weights and dweights are both given or both NULL; without them dy = dout's
 * rows and y is not read (it may be NULL). */
int gsr_combine_rows_backward(int64_t tokens, int64_t k, int64_t rows_in, int64_t width,
                              const void* dout, const void* y, const int32_t* positions,
                              const float* weights, const int32_t* rows,
                              void* dy, float* dweights, void* stream);

/* Grouped products: every group of rows has a B (and bias) of its own, as the
 * experts of a routed layer do.  For group e and its rows
 * offsets[e] <= r < offsets[e + 1]:
 *
 *     C[r,n] = act( alpha * sum_{k<K} A[rows[r],k] * B[e,k,n] + bias[e,n] )
 *
 *   C        P x N; rows outside every group stay as they were
 *   A        a_rows x K with rows, P x K (row r itself) without (rows NULL,
 *            a_rows ignored)
 *   rows     NULL, or P row indices; an index outside [0, a_rows) is a row of
 *            zeros.  The copy of A's rows into group order is not made: the
 *            kernels fetch them where they are.
 *   B        groups x K x N; bias NULL or groups x N
 *   offsets  groups + 1 values on the device, not decreasing, in [0, P] (the
 *            offsets of gsr_group_rows); a group may be empty.  Other values
 *            make wrong or missing results, never an access outside.
 * Epilogue, precision, alignment, ownership and errors as gemm_scale_bias_act
 * (same sums per tile, so with a forced configuration a group's outputs are the
 * bits of that call on its rows with the same one; without one, operands off the
 * 128-bit path may be summed over four runs of K).  GSR_ERROR_TOO_LARGE for P >= 2^31,
 * more than 1024 groups, K or N >= 2^22, one group's B of 2^31 bytes or more,
 * or, with rows, an A of 2^31 bytes or more, and where a launch would have
 * 2^32 threads (a forced 64 x 64 tile: from P of about 2^29); P x N, P x K and
 * the whole B may be larger.  config_id: -1, or one of 21, 22, 28, 31 and 32
 * (forced tile; others GSR_ERROR_INVALID_CONFIG). */
int gemm_grouped_scale_bias_act(int64_t P, int64_t N, int64_t K, int64_t groups,
                                const void* A, int64_t a_rows, const int32_t* rows,
                                const void* B, const void* bias, void* C, const int32_t* offsets,
                                float alpha, int32_t activation, void* stream, int32_t config_id);

/* Low-rank adapters of many requests beside one product: row m uses the
 * weights B + scales[l] * La_l^T Lb_l^T of its own adapter l = ids[m],
 *
 *     C[m,n] = act( alpha * ( sum_k A[m,k] * B[k,n]
 *                   + scales[l] * sum_r ( sum_k A[m,k] * La[l,r,k] ) * Lb[l,n,r] ) + bias[n] )
 *
 *   La  adapters x rank x K, Lb  adapters x N x rank, IEEE binary16 (the
 *       layouts of a checkpoint's two factors; 16-byte aligned with K and
 *       rank multiples of 8 they are read in 16-byte units, else value by
 *       value); adapters of a smaller rank are padded with zeros
 *   ids  M adapter indices in any order; an index outside [0, adapters) is a
 *        row without an adapter
 *   scales  adapters binary32 values, or NULL (ones)
 * The inner sum is binary32 and enters the second product to within 2^-23 of
 * its row's largest value, whatever that is; both sums, the scale, the bias and
 * the activation are binary32, with one narrowing to binary16.  An adapter's
 * values reach its own rows only, whatever they are.  rank is at most 256
 * and M at most 2^27 - 16 (GSR_ERROR_TOO_LARGE); one adapter's La and Lb are
 * below 2^31 bytes each and the whole arrays may be larger.  adapters = 0 or
 * rank = 0 is the product alone (gemm_scale_bias_act_ws).  Two kernels are
 * enqueued, or, for at most 64 rows, one whose first workgroups make the inner
 * sums.
 *   workspace  as gemm_scale_bias_act_ws's, whose counters it shares (its
 *              first 512 bytes zero before the first call and again after
 *              each), of gsr_adapter_workspace_bytes(M, N, K, rank) bytes;
 *              with less GSR_ERROR_INVALID_VALUE, or no K split if only that
 *              does not fit
 *   config_id  -1, or one of 21, 22, 28, 31, 32; splits as
 *              gemm_scale_bias_act_ws's (at most 128 tiles split)
 *   looks  how often a workgroup of the one-kernel form looks for inner sums
 *          that are not there yet before it makes them itself, which gives
 *          the same bits; -1: the library's number (for tests)
 * Otherwise as gemm_scale_bias_act_ws. */
int gemm_adapters_scale_bias_act(int64_t M, int64_t N, int64_t K,
                                 const void* A, const void* B, const void* bias, void* C,
                                 int64_t adapters, int64_t rank, const void* la, const void* lb,
                                 const int32_t* ids, const float* scales, float alpha, int32_t activation,
                                 void* workspace, int64_t workspace_bytes,
                                 void* stream, int32_t config_id, int32_t splits, int32_t looks);

/* The bytes gemm_adapters_scale_bias_act needs (0: none); -1 for sizes it
 * rejects.  Host only. */
int64_t gsr_adapter_workspace_bytes(int64_t M, int64_t N, int64_t K, int64_t rank);

/* ---- a few rows against weights in 4 bits, and a whole layer for a few tokens ---
 * 4-bit weights of a K x N matrix (or `matrices` of them, one behind the other):
 *
 *     w[k,n] = (q[k,n] - zeros[k / group, n]) * scales[k / group, n]
 *
 *   codes   ceil(K / 8) x N 32-bit words (4-byte aligned): bits 4i .. 4i + 3 of
 *           word (r, n) are q[8r + i, n], 0..15; those of rows past K are ignored
 *   scales  ceil(K / group) x N binary16 values
 *   zeros   ceil(K / group) x N 8-bit values (0..255), or NULL: 8 everywhere
 *   group   a power of two from 32 to 2^30; the last group may be short
 * K and N are below 2^22 (GSR_ERROR_TOO_LARGE). */

/* codes, scales and (zeros not NULL) zeros of the binary16 values B, column by
 * column and group by group, in binary32:
 *   zeros NULL  scale = binary16(max|b| / 7), q = clamp(rint(b / scale), -8, 7) + 8
 *   else        lo = min(b, 0), hi = max(b, 0), scale = binary16((hi - lo) / 15),
 *               zero = clamp(rint(-lo / scale), 0, 15),
 *               q = clamp(rint(b / scale) + zero, 0, 15)
 * rint rounds ties to even.  A scale of zero has codes and zero 8; a group with
 * an infinity or a NaN gets the scale NaN.  Codes past K are those of zeros. */
int gsr_quantize_w4(int64_t matrices, int64_t K, int64_t N, int64_t group, const void* B,
                    uint32_t* codes, void* scales, uint8_t* zeros, void* stream);

/* B = the weights' values, each rounded once to binary16 (an infinity beyond its
 * range: 65504 in a group comes back as one, its scale 65504 / 7 being rounded up). */
int gsr_dequantize_w4(int64_t matrices, int64_t K, int64_t N, int64_t group,
                      const uint32_t* codes, const void* scales, const uint8_t* zeros, void* B,
                      void* stream);

/* The fused product with such weights, made for few rows:
 *
 *     C[m,n] = act( alpha * sum_k A[m,k] * w[k,n] + bias[n] )
 *
 * A, bias, C, alpha and the activation as gemm_scale_bias_act's, at any 2-byte
 * alignment; matrices may be larger than 2^31 bytes, M is below 2^31.  The
 * products A[m,k] (q - zero) are summed in binary32, group by group, and the
 * scale multiplies a group's sum: the weights are not rounded.  Where many rows
 * make it faster (more than 16, commonly from 200 on) and the workspace holds K x N
 * binary16 values (512 + 2 K N bytes, which have to be below 2^31), the weights are
 * first written there as gsr_dequantize_w4 gives them, each rounded once to
 * binary16, and multiplied by the dense kernels; a column with a group whose codes
 * could stand for 65520 or more in size, the first value past binary16, keeps its
 * weights unrounded there too.
 * A scale that is not finite makes its column's outputs not finite, before the
 * activation.
 *   workspace  as gemm_scale_bias_act_ws's, whose counters it shares (its first
 *              512 bytes zero before the first call and again after each), of
 *              gsr_w4_workspace_bytes(M, N, K) bytes; with less or NULL K is
 *              not split across workgroups, and the weights are not written out:
 *              fewer than 512 + 2 K N bytes keep them unrounded for any M
 * Ownership, streams and errors as gemm_scale_bias_act_ws. */
int gemm_w4_scale_bias_act(int64_t M, int64_t N, int64_t K, const void* A,
                           int64_t group, const uint32_t* codes, const void* scales, const uint8_t* zeros,
                           const void* bias, void* C, float alpha, int32_t activation,
                           void* workspace, int64_t workspace_bytes, void* stream);

/* The bytes gemm_w4_scale_bias_act can use (0: none); -1 for sizes it rejects.
 * Host only. */
int64_t gsr_w4_workspace_bytes(int64_t M, int64_t N, int64_t K);

/* One of a layer's matrices: `experts` of K x N binary16 values (group 0, scales
 * and zeros NULL) or of 4-bit weights (group as above, data the codes), and
 * experts x N binary16 values of bias, or NULL. */
typedef struct gsr_weights {
    const void* data;
    const void* scales;
    const uint8_t* zeros;
    const void* bias;
    int64_t group;
} gsr_weights;

/* A whole layer of routed experts for at most 64 tokens, in two launches.  With
 * e = ids[t,j] (T x k, 4 or 8 bytes each; an id outside [0, experts) has no
 * term, and an expert may be named more than once):
 *
 *     h[t,j,f] = act( sum_i x[t,i] * up[e,i,f] + bias_up[e,f] )               gate NULL
 *     h[t,j,f] = act( sum_i x[t,i] * gate[e,i,f] + bias_gate[e,f] )
 *                * ( sum_i x[t,i] * up[e,i,f] + bias_up[e,f] )                otherwise
 *     out[t,o] = sum_j weights[t,j] * ( sum_f h[t,j,f] * down[e,f,o] + bias_down[e,o] )
 *
 *   x        T x H;  up, gate  experts of H x F;  down  experts of F x O
 *   weights  T x k binary32, or NULL (ones)
 *   activation  any gsr_activation
 * Sums, biases, activation, gate and weights are binary32; between the launches
 * each h is kept to within 2^-22 of itself or 2^-35, whichever is more, and one that
 * is not zero keeps its sign beside an infinite weight (an h beyond binary16's range
 * is an infinity); out is rounded once.  weights[t,j] that are not finite make their
 * token's outputs not finite.  A token's choices are added in an order that the ids
 * alone decide: equal inputs give equal bits.  Either all matrices are binary16 or all are 4-bit, gate
 * and up of one group.  Values are row-major at any 2-byte alignment (codes 4).
 * T <= 64, T k <= 1024, experts <= 1024, widths below 2^22, T k F below 2^29 with F
 * in whole eights (GSR_ERROR_TOO_LARGE); for more tokens there are gsr_group_rows
 * and the grouped products.
 *   workspace  gsr_expert_few_workspace_bytes(T, k, experts, F, O) bytes,
 *              16-byte aligned, counters as gemm_scale_bias_act_ws's (its first
 *              512 bytes zero before the first call and again after each), one
 *              per call that may run at the same time; GSR_ERROR_INVALID_VALUE
 *              if smaller
 * out must not overlap anything else.  Ownership, streams and errors as above. */
int gsr_expert_mlp_few(int64_t tokens, int64_t k, int64_t experts, int64_t H, int64_t F, int64_t O,
                       const void* x, const void* ids, int32_t id_bytes, const float* weights,
                       const gsr_weights* up, const gsr_weights* gate, const gsr_weights* down,
                       int32_t activation, void* out, void* workspace, int64_t workspace_bytes, void* stream);

/* The bytes gsr_expert_mlp_few needs (with 4-bit weights or without); -1 for
 * sizes it rejects.  Host only. */
int64_t gsr_expert_few_workspace_bytes(int64_t tokens, int64_t k, int64_t experts, int64_t F, int64_t O);

/* Tuning table: exact problem shapes mapped to a launch, consulted before the
 * built-in selector (by every entry point called with config id -1, and by
 * gsr_select_config).  The file is text, one entry per line,
 *     M N K config_id group_m xcd_remap
 * with '#' starting a comment; tiled_dense_gemm_scale_amd/tune.py writes it
 * from measured sweeps (the aikraft.ru TileLang guide: section 3, a manual
 * sweep of tile, stage and swizzle knobs that finds no schedule best for
 * every size; section 7, an automatic search of that space per problem and
 * GPU).  gsr_load_tuning replaces the table, or returns
 * GSR_ERROR_INVALID_VALUE for an unreadable or malformed file and keeps the
 * previous one; gsr_clear_tuning empties it; gsr_tuning_entries counts it.
 * Host only, thread-safe. */
int gsr_load_tuning(const char* path);
int gsr_clear_tuning(void);
int gsr_tuning_entries(void);

/* The configuration the selector picks for an M x N x K problem (the tuning
 * table first, with its launch order in group_m / xcd_remap).  Host only;
 * touches no device.  Returns GSR_SUCCESS or GSR_ERROR_INVALID_VALUE. */
int gsr_select_config(int64_t M, int64_t N, int64_t K, gsr_config* out);

/* Number of compiled tile configurations; their ids (written to ids[0..],
 * at most `capacity` of them; returns the number of compiled configurations,
 * or -1 for capacity < 0 or a null ids with capacity > 0); the description of
 * one (GSR_ERROR_INVALID_CONFIG for an id that is not compiled).  Host only. */
int gsr_num_configs(void);
int gsr_config_ids(int32_t* ids, int32_t capacity);
int gsr_get_config(int32_t config_id, gsr_config* out);

/* A static, human-readable name for a status code. */
const char* gsr_status_string(int status);

/* Library version, as major*10000 + minor*100 + patch. */
int gsr_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GSR_H_ */
