/*
 * mxq — affine group-wise quantized matrix multiply for sm_103a (GB300).
 *
 * The operation (mlxcel issue #1536, Baseline section: weights stored as
 * "affine 4-bit / group 64", activations bf16; issue #1538, 4-bit vs 8-bit
 * section: 8-bit codes are unsigned bytes, and the product accumulates in
 * float at every width):
 *
 *   w^[n, k] = s[n, k/G] * q[n, k] + b[n, k/G]
 *   y[m, n]  = sum_k x[m, k] * w^[n, k]          (fp32 accumulation)
 *
 * G = group_size, the k values that share one scale/bias pair: 64 (the
 * stored format named above), 32 or 128 (issue #1536, Diagnosis item 4: the
 * tile choice there tests group_size <= 64, so the format also comes with
 * other group sizes; 32 and 128 are the sizes on either side of 64).
 *
 * Storage, all row-major and contiguous:
 *   x       bf16   [M, K]            activations
 *   w       uint32 [N, K*bits/32]    packed codes.  4-bit: eight codes per
 *                                    little-endian word, lowest k in the
 *                                    lowest nibble (integer_subbyte<4>, the
 *                                    qmm_naive kernel name in issue #1536's
 *                                    profile table).  8-bit: four codes per
 *                                    word, lowest k in the lowest byte.
 *                                    2-bit: sixteen codes per word, lowest k
 *                                    in the lowest two bits.  3- and 6-bit:
 *                                    the same little-endian bit stream per
 *                                    row, code k in bits [k*b, k*b + b), so
 *                                    a code may straddle two words (the bit
 *                                    width is a parameter of the kernels in
 *                                    issue #1536, Diagnosis item 3).
 *   scales  bf16   [N, K/G]          s per (output row, group of G k)
 *   biases  bf16   [N, K/G]          b per (output row, group of G k)
 *   y       bf16   [M, N]            output, rounded once from fp32 (RNE)
 *
 * All pointers except `stream` are DEVICE pointers owned by the caller; the
 * library allocates nothing and keeps no pointer after a call returns.  All
 * calls are asynchronous on `stream` (a cudaStream_t, NULL = legacy default
 * stream) and return after the launch.  Arguments are checked on the host
 * before anything is launched; a call that returns an error has launched
 * nothing and written nothing.  Inputs must be finite.
 *
 * Device requirement: compute capability 10.3 (sm_103a).
 */
#ifndef MXQ_H
#define MXQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MXQ_OK = 0,
    MXQ_ERR_INVALID_ARG = 1, /* bad size, bits, group size or null pointer   */
    MXQ_ERR_MISALIGNED = 2,  /* x, w or y not 16-byte aligned; or a scale /
                                bias / id pointer not aligned to its type     */
    MXQ_ERR_UNSUPPORTED = 3, /* a valid request this build does not implement */
    MXQ_ERR_ARCH = 4,        /* current device is not compute capability 10.3 */
    MXQ_ERR_CUDA = 5,        /* a CUDA runtime call or launch failed          */
    MXQ_ERR_WORKSPACE = 6,   /* workspace missing or smaller than required    */
    MXQ_ERR_SCRATCH_LIMIT = 7 /* mxq_gather_qmm_noalloc: the request needs more
                                 than MXQ_NOALLOC_SCRATCH_BYTES of scratch      */
} mxq_status;

/* Bits set in *dev_status (device memory, written by the kernels when the
 * caller passes a non-null pointer; the call first stores 0 there).        */
#define MXQ_DEV_BAD_EXPERT_ID   0x1 /* an expert id outside [0, E)             */
#define MXQ_DEV_UNSORTED_IDS    0x2 /* expert ids decrease somewhere           */
#define MXQ_DEV_BAD_ROW_SRC     0x4 /* a row_src entry outside [0, T)          */
#define MXQ_DEV_TIMEOUT         0x8 /* an on-chip pipeline wait gave up; the
                                       output is incomplete                   */
#define MXQ_DEV_BAD_SLOT       0x10 /* a cache slot at or past the last one    */
#define MXQ_DEV_BAD_PAGE       0x20 /* a page that a row sees is outside the
                                       cache; its tokens count as not visible */
#define MXQ_DEV_BAD_SEQUENCE   0x40 /* a sequence's length or rows are out of
                                       range                                  */

/* Decode GEMV, M = 1 (mlxcel issue #1536, Diagnosis item 3: the qmv kernel;
 * fp32 accumulation at every width is the fix that item names).
 *   x: bf16 [K]; y: bf16 [N]; w, scales, biases as above.
 *   dev_status: device int32 or NULL; receives 0 or MXQ_DEV_TIMEOUT.
 * Requirements: bits in {2, 3, 4, 6, 8}; group_size in {32, 64, 128}; K > 0,
 * K % 64 == 0 and K % group_size == 0 (K % 128 == 0 at 3 bits); N > 0;
 * x, w, y 16-byte aligned; scales, biases 2-byte aligned.  The streaming
 * kernel is used when K % 512 == 0, K <= 20480, K / group_size % 8 == 0 and
 * scales/biases are 16-byte aligned; other shapes take a direct-load kernel
 * (same result rule, different summation order).  The streaming kernel is
 * launched as a
 * programmatic dependent launch: its CTAs may be placed on SMs while the
 * kernel before it on the stream finishes, but they read and write nothing
 * until that kernel has completed, so stream order is kept.                 */
mxq_status mxq_qmv(const void* x, const uint32_t* w, const void* scales, const void* biases,
                   void* y, int K, int N, int bits, int group_size, int32_t* dev_status,
                   void* stream);

/* Decode GEMV for the other operand layout (mlxcel PR #1562, What changed:
 * the grouped GEMM is checked for both operand layouts): w is stored [K, N],
 * row k holding the codes of every output n as the same little-endian bit
 * stream (code n in bits [n*b, n*b + b) of row k), and each group is G
 * consecutive n of one row:
 *   w:      uint32 [K, N*bits/32]
 *   scales, biases: bf16 [K, N/G]
 *   y[n] = sum_k x[k] * (s[k, n/G] * q[k, n] + b[k, n/G])   (fp32 accumulation)
 *   x: bf16 [K]; y: bf16 [N].
 * Requirements: bits in {2, 4, 8} (3 and 6: MXQ_ERR_UNSUPPORTED); group_size
 * in {32, 64, 128}; K > 0; N > 0, N % 64 == 0 and N % group_size == 0;
 * x, w, y 16-byte aligned; scales, biases 2-byte aligned.  `dev_status`
 * (device int32, may be NULL) receives 0.  Up to 8 CTAs of a thread-block
 * cluster split K and add their partials in rank order: deterministic.     */
mxq_status mxq_qmv_kn(const void* x, const uint32_t* w, const void* scales, const void* biases,
                      void* y, int K, int N, int bits, int group_size, int32_t* dev_status,
                      void* stream);

/* Prefill GEMM for the [K, N] operand layout (mlxcel PR #1562, What
 * changed: both operand layouts), w, scales and biases as for mxq_qmv_kn:
 *   y[m, n] = sum_k x[m, k] * (s[k, n/G] * q[k, n] + b[k, n/G])
 *   x: bf16 [M, K]; y: bf16 [M, N].
 * M = 1 runs mxq_qmv_kn (the same operation).  Otherwise the tcgen05 tensor
 * cores: each code word dequantises (one bf16 rounding of s*q + b, as in
 * mxq_qmm) into 8 bf16 contiguous along n, stored as the MMA's MN-major A
 * operand in shared memory; fp32 accumulation in tensor memory.  With fewer
 * tiles than SMs, K is split over up to 8 CTAs of a cluster and the fp32
 * partials are added in a fixed order: deterministic.
 * Requirements: bits in {2, 4, 8} (3 and 6: MXQ_ERR_UNSUPPORTED);
 * group_size in {32, 64, 128}; M > 0; K > 0 (K % 8 == 0 when M > 1); N > 0,
 * N % 64 == 0, N % group_size == 0; x, w, y 16-byte aligned; scales,
 * biases 2-byte aligned.  `dev_status` (device int32, may be NULL) receives
 * 0 or MXQ_DEV_TIMEOUT.                                                     */
mxq_status mxq_qmm_kn(const void* x, const uint32_t* w, const void* scales, const void* biases,
                      void* y, int M, int K, int N, int bits, int group_size,
                      int32_t* dev_status, void* stream);

/* Prefill GEMM, y[M, N] = x[M, K] . w^[N, K]^T (mlxcel issue #1536, Baseline
 * profile table and Diagnosis item 4: the qmm_naive kernel).  M = 1 runs the
 * streaming GEMV of mxq_qmv (the same operation); M = 2 or 3 runs one such
 * GEMV per activation row where the shape allows (fewer rows than a tensor
 * tile's fill is worth).  Otherwise the tcgen05
 * tensor cores: codes are dequantised to bf16 into tensor memory (the MMA's
 * A operand) and the products accumulate in fp32 in tensor memory.  When M
 * and N give fewer 128 x 256 tiles than the GPU has SMs, K is split over up
 * to 8 CTAs of a thread-block cluster and the fp32 partials are added
 * through distributed shared memory in a fixed order; with enough tiles, one
 * persistent CTA per SM walks them.  Either way the result is deterministic
 * for a given shape.
 * Requirements as for mxq_qmv plus M > 0.  `dev_status` (device int32, may
 * be NULL) receives 0 or MXQ_DEV_TIMEOUT.                                   */
mxq_status mxq_qmm(const void* x, const uint32_t* w, const void* scales, const void* biases,
                   void* y, int M, int K, int N, int bits, int group_size, int32_t* dev_status,
                   void* stream);

/* Sorted mixture-of-experts grouped variant (mlxcel PR #1562, Summary: the
 * sorted-MoE prefill path that routes a quantized GatherQMM into a grouped
 * GEMM, B = tokens * top_k rows sorted by expert).
 *   x:          bf16 [T, K]  activation rows
 *   w:          uint32 [E, N, K*bits/32]; scales, biases: bf16 [E, N, K/G]
 *   expert_ids: int32 [B], non-decreasing: expert of sorted row r
 *   row_src:    int32 [B], row of x that feeds sorted row r; NULL means r
 *               (then T must equal B)
 *   y:          bf16 [B, N], in sorted row order
 *   workspace:  device scratch, 256-byte aligned, overwritten by the call:
 *               mxq_gather_workspace_bytes(B, E, K, N) bytes when row_src
 *               is given (it also holds the activation rows in sorted
 *               order), otherwise the smaller mxq_gather_workspace_bytes(B,
 *               E, 0, N) suffices.
 *   dev_status: device int32 or NULL; receives the MXQ_DEV_* bits.
 * Rows whose expert id lies outside [0, E), or whose row_src lies outside
 * [0, T), are skipped and their y rows set to zero.  If the ids are not
 * non-decreasing, nothing is computed, all of y is set to zero and
 * MXQ_DEV_UNSORTED_IDS is reported.  No invalid input makes the kernels
 * read or write out of bounds.
 * Calls with at most 32 rows (a decode step) run one GEMV per row against
 * its expert's matrix (the same result rule, another summation order) and
 * use no workspace memory, though the size check still applies.
 * Larger calls build a tile table on the GPU and run the tensor-core GEMM:
 * at 2 and 4 bits two persistent CTAs per SM take tiles from a counter; at
 * 3, 6 and 8 bits one CTA computes each tile.
 * Requirements: B, E, T, N > 0; K > 0, K % 64 == 0, K % group_size == 0;
 * bits in {2, 3, 4, 6, 8} (K % 128 == 0 at 3 bits); group_size in
 * {32, 64, 128}; x, w, y 16-byte aligned; the rest aligned to type.          */
mxq_status mxq_gather_qmm(const void* x, const uint32_t* w, const void* scales,
                          const void* biases, const int32_t* expert_ids,
                          const int32_t* row_src, void* y, int T, int B, int E, int K, int N,
                          int bits, int group_size, void* workspace, size_t workspace_bytes,
                          int32_t* dev_status, void* stream);

/* The sorted mixture-of-experts grouped GEMM for the [K, N] operand layout
 * (mlxcel PR #1562, What changed: the grouped GEMM is checked against the
 * dense per-expert reference in both operand layouts):
 *   w:      uint32 [E, K, N*bits/32]; scales, biases: bf16 [E, K, N/G]
 *   y[r, n] = sum_k x[src(r), k] * (s_e[k, n/G] * q_e[k, n] + b_e[k, n/G]),
 *             e = expert_ids[r]
 * Every other argument, the workspace (mxq_gather_workspace_bytes) and the
 * handling of invalid ids and rows are as for mxq_gather_qmm.  The call
 * builds the tile table on the GPU (tiles of at most 64 sorted rows of one
 * expert), copies routed rows into sorted order, and runs one CTA per (tile,
 * 128 columns) on the tensor cores, at every B.
 * Requirements: B, E, T > 0; bits in {2, 4, 8} (3 and 6:
 * MXQ_ERR_UNSUPPORTED); group_size in {32, 64, 128}; K > 0, K % 8 == 0;
 * N > 0, N % 64 == 0, N % group_size == 0; alignment as for mxq_gather_qmm. */
mxq_status mxq_gather_qmm_kn(const void* x, const uint32_t* w, const void* scales,
                             const void* biases, const int32_t* expert_ids,
                             const int32_t* row_src, void* y, int T, int B, int E, int K, int N,
                             int bits, int group_size, void* workspace, size_t workspace_bytes,
                             int32_t* dev_status, void* stream);

/* Workspace bytes mxq_gather_qmm (and mxq_gather_qmm_gateup) needs for B
 * rows over E experts with K-wide activation rows routed through row_src
 * (K = 0: no row_src). */
size_t mxq_gather_workspace_bytes(int B, int E, int K, int N);

/* The gate and up projections of a mixture-of-experts layer in one call
 * (mlxcel issue #1538, comment "Correction: MoE decode does not route to
 * qmm_naive": decode steps run fused per-expert gate/up kernels): the same
 * routed activation rows against two expert weight sets of one shape,
 *   y_gate[r, n] = sum_k x[src(r), k] * w^gate_{e(r)}[n, k]
 *   y_up[r, n]   = sum_k x[src(r), k] * w^up_{e(r)}[n, k]
 * with every argument as in mxq_gather_qmm (w_gate/w_up, scales_*,
 * biases_* each [E, N, ...] with the same shape; y_gate, y_up [B, N]; the
 * same workspace size).  No activation function is applied: the pages name
 * none; a caller combines the two outputs.  One launch computes both
 * projections: with at most 32 rows the per-row GEMVs of both sets (grid z
 * = the set); otherwise the routed rows are put in sorted order once and
 * the grouped GEMM takes the tiles of both sets (persistent CTAs at 2 and 4
 * bits, one CTA per tile and set otherwise).  Each output is bit for bit the
 * output mxq_gather_qmm gives for its set.  The status word reports the id
 * and row_src checks and timeouts of either set.                          */
mxq_status mxq_gather_qmm_gateup(const void* x, const uint32_t* w_gate, const void* scales_gate,
                                 const void* biases_gate, const uint32_t* w_up,
                                 const void* scales_up, const void* biases_up,
                                 const int32_t* expert_ids, const int32_t* row_src, void* y_gate,
                                 void* y_up, int T, int B, int E, int K, int N, int bits,
                                 int group_size, void* workspace, size_t workspace_bytes,
                                 int32_t* dev_status, void* stream);

/* Sorted mixture-of-experts GEMM without any allocation: the same operation,
 * arguments, results and checks as mxq_gather_qmm, but the scratch memory
 * comes from one fixed array inside the library instead of a caller-provided
 * workspace.  (The pages that define the operation have no counterpart to
 * this call; it exists for callers that cannot provide device memory.)
 *
 * Who needs it: callers that have no device allocator of their own (plain C
 * hosts), runtimes whose device memory is fully reserved before serving
 * starts, and loops that must not allocate between steps.  Nothing is
 * allocated at call time, by the caller or by the library: the scratch is
 * MXQ_NOALLOC_SCRATCH_BYTES of device memory reserved on each device when
 * the library's device code is loaded there.
 *
 * Limit: a request whose scratch, mxq_gather_workspace_bytes(B, E, K, N)
 * with row_src (or mxq_gather_workspace_bytes(B, E, 0, N) without), exceeds
 * MXQ_NOALLOC_SCRATCH_BYTES returns MXQ_ERR_SCRATCH_LIMIT before anything
 * touches the device.  32 MiB holds, for example, the tile table and the
 * sorted rows of 4584 routed rows of K = 2816.
 *
 * Set-up: the first call on each device looks up the scratch's device
 * address with that device current (this may load the library's device
 * code); make that first call before capturing a stream into a graph.  The
 * address is kept for the life of the process: do not use this entry point
 * on a device after cudaDeviceReset (or any other teardown of its primary
 * context), since the scratch may then live at another address.
 * Nothing in the scratch has to start at zero: every call writes all the
 * scratch it reads.
 *
 * Concurrency: all calls on one device share the scratch.  Two calls whose
 * execution overlaps (different streams, or different threads without
 * ordering between them) race on it and produce wrong results; order them,
 * for example by issuing every call on the same stream.                    */
#define MXQ_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)
mxq_status mxq_gather_qmm_noalloc(const void* x, const uint32_t* w, const void* scales,
                                  const void* biases, const int32_t* expert_ids,
                                  const int32_t* row_src, void* y, int T, int B, int E, int K,
                                  int N, int bits, int group_size, int32_t* dev_status,
                                  void* stream);

/* Affine group-wise encoder: the stored format from float weights (the
 * format of mlxcel issue #1536, Baseline section; the affine map read as
 * bias = group minimum, scale = group range / (2^bits - 1)).
 *   w:      float [N, K] row-major (finite), 16-byte aligned
 *   codes:  uint32 [N, K*bits/32], 16-byte aligned (output)
 *   scales, biases: bf16 [N, K/G] (output)
 * Per (row, group of G = group_size): mn, mx = min, max (-0 read as +0);
 * s = bf16(RN(RN(mx - mn) / (2^bits - 1))), b = bf16(mn), rounded to nearest
 * even; q = clamp(rint(RN(RN(w - b) / s)), 0, 2^bits - 1) with the stored
 * bf16 s and b, q = 0 when s == 0.  All decisions in binary32, so the codes
 * are reproducible bit for bit.  Requirements: bits in {2, 3, 4, 6, 8}
 * (K % 128 == 0 at 3 bits);
 * group_size in {32, 64, 128}; K > 0, K % 64 == 0, K % group_size == 0;
 * N > 0.                                                                    */
mxq_status mxq_quantize(const float* w, uint32_t* codes, void* scales, void* biases, int N,
                        int K, int bits, int group_size, void* stream);

/* ------------------------------------------------------------------------
 * A paged key/value cache held in 4 bits, and what a layer does between its
 * q/k/v projections and its output projection.  (The pages that define the
 * matrix products have no counterpart to these calls: they hold the format
 * of the weights, affine codes with a bf16 scale and bias per group, for the
 * keys and values of the attention.)
 *
 * The cache is one array of n_pages pages, uint8 [n_pages, Hkv, block bytes];
 * a page holds page_size tokens (16, 32, 64 or 128) of every key/value head,
 * and a slot is page * page_size + token.  Per (token, head) the D values
 * (64, 128 or 256) of the key and of the value are codes q of 4 bits and one
 * (scale, bias) pair of bf16 per group of G = group_size values (32, 64 or
 * 128, at most D): k^[d] = s[d/G] * q[d] + b[d/G].
 * Block of one page and head, mxq_kv_block_bytes(D, page_size, G) bytes:
 *   K codes  page_size * D/2 bytes
 *   K pairs  bf16 [page_size][D/G][2]: scale, bias
 *   V codes, V pairs likewise
 * Codes lie in slabs of 8 tokens x DS = min(D, 128) values, slab (t/8, d/DS)
 * after slab; a slab is 32 x DS/32 little-endian words, word (4 r + i) * DS/32
 * + u holding, lowest nibble first,
 *   K: token r of the 8, values 32 u + 8 i + 0 .. 7 of the DS
 *   V: tokens 2 i and 2 i + 1, values 32 u + r + 8 n, n = 0 .. 3: token 2 i
 *      in the low 16 bits, token 2 i + 1 in the high 16
 * Scales and biases may be any finite numbers of either sign.
 * Pages may be copied, shared by several page tables and reused freely: what
 * lies in slots that no row sees is never used, whatever bits it holds.
 * Strides are in values (elements), multiples of 8 and not negative; the D
 * values of a head are contiguous.  T = 0 (nothing to do) is valid.         */

/* Bytes of one page for one key/value head; 0 if the shape is not supported. */
size_t mxq_kv_block_bytes(int D, int page_size, int group_size);

/* RMS norm of query and key heads and the rotary position, in one pass:
 *   n = x * rsqrt(mean(x^2) + eps) * (weight + weight_offset)
 *   (n1, n2) -> (n1 c - n2 s, n2 c + n1 s),  c, s = rope_scale * cos, sin of
 *   positions[t] * inv_freq[j]
 * over the pairs (j, j + rot_dim/2), or (2 j, 2 j + 1) if interleaved, of the
 * first rot_dim values of each head; the rest keep n.  fp32 throughout (the
 * angle is reduced from the exact product), one rounding to bf16.
 *   q: bf16 [T, Hq, D], k: bf16 [T, Hk, D] (either count may be 0)
 *   positions: int32 [T], any sign; inv_freq: fp32 [rot_dim/2]
 *   q_weight, k_weight: bf16 [D]; NULL leaves that side without a norm
 *   q_out, k_out: bf16, may be q and k themselves (same strides)
 * rope_scale multiplies the rotation (the attention factor of position
 * scaling methods; 1 otherwise).
 * Requirements: D % 8 == 0, D <= 256; rot_dim % 16 == 0, rot_dim <= D (0: no
 * rotation; then at least one weight); pointers 16-byte aligned (positions
 * and inv_freq 4).                                                          */
mxq_status mxq_qk_norm_rope(const void* q, long long q_row_stride, long long q_head_stride,
                            const void* k, long long k_row_stride, long long k_head_stride,
                            const int32_t* positions, const float* inv_freq, const void* q_weight,
                            const void* k_weight, void* q_out, long long q_out_row_stride,
                            long long q_out_head_stride, void* k_out,
                            long long k_out_row_stride, long long k_out_head_stride, int T,
                            int Hq, int Hk, int D, int rot_dim, int interleaved, float eps,
                            float weight_offset, float rope_scale, void* stream);

/* Encode new rows and write them into the cache: row t goes to slots[t].
 * The rule is mxq_quantize's at 4 bits, with its binary32 decisions, so the
 * stored bits do not depend on the call that wrote them.
 *   k, v: bf16 [T, Hkv, D], finite, strided; pages 16-byte aligned
 *   slots: int32 [T]; a negative slot skips the row, one at or past
 *   n_pages * page_size is skipped and reported (MXQ_DEV_BAD_SLOT).  Two rows
 *   with one slot leave either's bits, not necessarily of one row.
 *   dev_status: device int32 or NULL.                                       */
mxq_status mxq_kv_append(const void* k, long long k_row_stride, long long k_head_stride,
                         const void* v, long long v_row_stride, long long v_head_stride,
                         void* pages, const int32_t* slots, int T, int Hkv, int D, int n_pages,
                         int page_size, int group_size, int32_t* dev_status, void* stream);

/* The rows of given slots: k_out, v_out bf16 [T, Hkv, D] contiguous, each
 * value s * q + b rounded once.  Rows of negative slots, and of slots past the
 * last one (reported), are zero.                                            */
mxq_status mxq_kv_read(const void* pages, const int32_t* slots, void* k_out, void* v_out, int T,
                       int Hkv, int D, int n_pages, int page_size, int group_size,
                       int32_t* dev_status, void* stream);

/* Attention over the cache.  Sequence i has ctx_lens[i] tokens in the cache
 * (its new ones already appended), in the pages page_table[i, 0 ...], and the
 * query rows q_starts[i] .. q_starts[i + 1] - 1, which are its last tokens:
 * row j of n has position p = ctx_lens[i] - n + j and sees the tokens
 *   t <= p, and with a window only t > p - window or t < sinks.
 *   out = softmax(scale * q . k^) . v^ over those, bf16 [T, Hq, D] contiguous;
 * query head h uses key/value head h / (Hq / Hkv).  A row that sees nothing
 * (ctx_lens[i] < n) is 0.
 *   q: bf16 [T, Hq, D], strided; q_starts: int32 [S + 1], or NULL: one row per
 *   sequence (T == S); page_table: int32 [S, max_pages], entries of pages that
 *   no row sees (behind a window, past the end) may hold anything
 *   lse: fp32 [T, Hq] or NULL: log sum exp of the scaled scores, -inf for a
 *   row that sees nothing, NaN for one whose scores are not numbers
 *   max_q_len: the most rows a sequence has, a host-side bound
 *   window: 0 for none; sinks: first tokens that stay visible
 *   workspace: mxq_kv_attention_workspace_bytes(T, S, Hq, Hkv, D, max_q_len)
 *   bytes, 256-byte aligned, overwritten
 * A page number outside [0, n_pages) where a row sees it makes its tokens
 * invisible and is reported (MXQ_DEV_BAD_PAGE).  A length outside [0, max_pages
 * * page_size] is clamped to it; a sequence whose rows are not within [0, T],
 * decrease or exceed max_q_len is left out (its rows of out are not written);
 * both are reported (MXQ_DEV_BAD_SEQUENCE).  Rows that belong to no sequence
 * are not written.  No invalid entry makes the kernels read or write out of
 * bounds.  The result is deterministic for given arguments.
 * Accuracy: scores, softmax and sums are fp32.  Sequences of one row, and of
 * several whose rows times query heads to a key/value head are up to 16: weights
 * times scales are rounded to 11 bits, keys and values are not; the output is
 * within 2^-8 of itself and 2^-11 of sum_t P_t (v^_t - b_t), in the 2-norm 1.9e-3
 * for values around zero at up to 131072 tokens, 1.7e-3 being the rounding to
 * bf16.  More rows: weights, keys and values are rounded to 11 bits, keys and values below
 * 2^-9 of the largest of their 32 tokens to 2^-20 of that.  In both, weights
 * times scales or values are kept down to 2^-31 of the largest.
 * Requirements: Hq % Hkv == 0; scale positive; q, pages, out 16-byte aligned;
 * max_pages * page_size at most 2^30 tokens.  Calls are counted in units of one
 * row tile and 32 to 128 tokens, in 32 bits; one that could have more of them for
 * its T, S and max_pages is refused (MXQ_ERR_UNSUPPORTED): some 10^13 rows times
 * tokens.                                                                     */
mxq_status mxq_kv_attention(const void* q, long long q_row_stride, long long q_head_stride,
                            const void* pages, const int32_t* page_table, const int32_t* ctx_lens,
                            const int32_t* q_starts, void* out, float* lse, int T, int S, int Hq,
                            int Hkv, int D, int n_pages, int max_pages, int page_size,
                            int group_size, int max_q_len, float scale, int window, int sinks,
                            void* workspace, size_t workspace_bytes, int32_t* dev_status,
                            void* stream);
size_t mxq_kv_attention_workspace_bytes(int T, int S, int Hq, int Hkv, int D, int max_q_len);

/* Attention over the cache for groups of sequences that begin with the same
 * tokens (several continuations of one prompt, conversations after one
 * instruction text): the keys and values of a group's prefix are read and
 * multiplied for all of its rows at once.
 *   Group g is the sequences group_starts[g] .. group_starts[g + 1] - 1 (NULL:
 * S / N each) and shares the prefix_lens[g] tokens in the pages prefix_table[g,
 * 0 ...].  Sequence i has ctx_lens[i] tokens of its own after them (its new ones
 * already appended), in the pages page_table[i, 0 ...], and the query rows
 * q_starts[i] .. q_starts[i + 1] - 1: row j of n sees its group's whole prefix
 * and the own tokens t <= ctx_lens[i] - n + j.  A sequence of no group has no
 * prefix.  A prefix need not end with a page: the own tokens begin in a page of
 * their own.
 *   out, lse, q, scale, pages, dev_status, workspace: as for mxq_kv_attention,
 *   mxq_kv_attention_shared_workspace_bytes(...) bytes; a row that sees nothing
 *   is 0 with lse -inf
 *   prefix_table: int32 [N, max_prefix_pages]; page_table: int32 [S, max_pages];
 *   group_starts: int32 [N + 1] or NULL; q_starts: int32 [S + 1], or NULL: one row
 *   per sequence (T == S)
 *   max_q_len, max_group: the most rows of a sequence and the most sequences of
 *   a group, host-side bounds
 * These bounds and the widths of the page tables decide how: a group's prefix for all of its
 * rows, or, where that takes no longer, for each sequence by itself.  Sequences with some tens of
 * rows of their own, or more, are faster by mxq_kv_attention over tables that name the prefix's pages.
 * Invalid entries as for mxq_kv_attention: pages outside [0, n_pages) are
 * invisible (MXQ_DEV_BAD_PAGE), lengths are clamped, a sequence or group whose
 * rows or sequences are out of range, decrease or exceed the bounds is left out
 * with its rows of out (MXQ_DEV_BAD_SEQUENCE).  Where group_starts or q_starts
 * decrease, so that groups or sequences overlap, that may be more of them, up to the
 * whole call: a value that is written then is that of one of the sequences that have
 * its row, after the prefix of one of the groups that have the sequence.  Otherwise the
 * result is deterministic for given arguments.
 * Accuracy: that of mxq_kv_attention for few rows in the own tokens and in
 * prefixes of up to 32 rows (times query heads to a key/value head) in a group,
 * at least that for more rows in the other prefixes.  There are no windows: a layer with
 * one reads few tokens of each sequence anyway.                              */
mxq_status mxq_kv_attention_shared(const void* q, long long q_row_stride, long long q_head_stride,
                                   const void* pages, const int32_t* prefix_table,
                                   const int32_t* prefix_lens, const int32_t* group_starts,
                                   const int32_t* page_table, const int32_t* ctx_lens,
                                   const int32_t* q_starts, void* out, float* lse, int T, int S, int N,
                                   int Hq, int Hkv, int D, int n_pages, int max_prefix_pages,
                                   int max_pages, int page_size, int group_size, int max_q_len,
                                   int max_group, float scale, void* workspace, size_t workspace_bytes,
                                   int32_t* dev_status, void* stream);
size_t mxq_kv_attention_shared_workspace_bytes(int T, int S, int N, int Hq, int Hkv, int D,
                                               int max_q_len, int max_group);

/* The best continuations of N prompts with W beams each (beam search):
 *   cand(w, v) = scores[w] + x[w, v] - log sum_u exp x[w, u]
 * over a prompt's W beams and V tokens, x their logits; the K best, the best
 * first, equal ones in the order of w V + v.
 *   logits: bf16 or (fp32 != 0) fp32 [N W, V], row_stride values from row to row
 *   (>= 0), any alignment of its type; scores: fp32 [N, W]
 *   done: uint8 [N, W] or NULL: beams that have ended; such a one has the single
 *   candidate end_token with its score as it is, and its logits are not read
 *   out_scores: fp32, parents (w): int32, tokens (v): int32, all [N, K]
 *   out_done: uint8 [N, K] or NULL: the parent had ended or the token is end_token
 *   (with K == W out_scores and out_done may be scores and done themselves)
 *   workspace: mxq_beam_select_workspace_bytes(N, W, V, K, fp32) bytes, 256-byte
 *   aligned, overwritten
 * A beam whose score is not finite is not in use: all its candidates, and any that
 * are not a number (a row with a logit that is +inf or not a number has no
 * others), count as -inf, which is a score like another: where there are fewer than K
 * above it the lowest w V + v of those follow.  -inf logits are tokens that are not
 * allowed.
 * Candidates are compared in 48 bits and none past the 53rd: tokens whose logits are
 * very low (-1e30, the type's lowest number) are level for all beams of a prompt.  Sums
 * over a row are fp32 in parts, which are added in 64 bits (scores are within 2^-18 and
 * their rounding, of rows of up to 2^20 tokens).  The result is deterministic, and equal
 * rows with equal scores have equal candidates.
 * Requirements: 1 <= W <= 64, 1 <= K <= 64, K <= W V; V > 0, W V < 2^31 - 65536;
 * 0 <= end_token < V where done or out_done is given.                        */
mxq_status mxq_beam_select(const void* logits, long long row_stride, int fp32, const float* scores,
                           const uint8_t* done, float* out_scores, int32_t* parents, int32_t* tokens,
                           uint8_t* out_done, int N, int W, int V, int K, int end_token, void* workspace,
                           size_t workspace_bytes, void* stream);
size_t mxq_beam_select_workspace_bytes(int N, int W, int V, int K, int fp32);

/* The cache after a selection of beams.  Sequences g W .. g W + W - 1 are group g;
 * sequence i of a group goes on from sequence parents[i] of it (0 .. W - 1), the
 * tokens of a prefix that the group shares (mxq_kv_attention_shared) aside.
 *   Every sequence has pages of its own, home_table int32 [S, max_pages], which
 * never changes; page_table starts as a copy of it, and in each column holds
 * pages out of the group's W home pages of that column.  Pages that are full are
 * then shared by the sequences that go on from them; the page that is being written
 * and those after it stay with the lowest of those sequences, and each other one
 * gets the lowest home page (in the order of the group's sequences) that nobody
 * keeps, into which the tokens are copied, in whole slabs of 8.
 *   pages: uint8 [layers, n_pages, Hkv, block bytes]: layers whose caches have the
 *   same page numbers are copied together
 *   page_table, ctx_lens -> table_out int32 [S, max_pages], lens_out int32 [S],
 *   which may be page_table and ctx_lens themselves; table_out[i, c], lens_out[i]
 *   are those of the sequence it goes on from but for the pages above
 *   parents: int32 [S]
 *   workspace: mxq_kv_reorder_workspace_bytes(S) bytes, 256-byte aligned
 * Sequences of a group may have different lengths.  A group with a parent outside
 * 0 .. W - 1 or a length outside its pages stays as it is (MXQ_DEV_BAD_SEQUENCE),
 * a column with pages that are not the group's home pages, or are outside the cache
 * where tokens are copied, likewise (MXQ_DEV_BAD_PAGE).  Columns in which no sequence
 * of a group has been given a page (negative in home_table) stay as they are.
 * Requirements: 1 <= W <= 64, S % W == 0; pages 16-byte aligned.             */
mxq_status mxq_kv_reorder(void* pages, const int32_t* page_table, const int32_t* home_table,
                          const int32_t* ctx_lens, const int32_t* parents, int32_t* table_out,
                          int32_t* lens_out, int S, int W, int layers, int n_pages, int Hkv, int D,
                          int max_pages, int page_size, int group_size, void* workspace,
                          size_t workspace_bytes, int32_t* dev_status, void* stream);
size_t mxq_kv_reorder_workspace_bytes(int S);

/* Static description of a status code. */
const char* mxq_status_string(mxq_status status);

/* Library version, major * 10000 + minor * 100 + patch. */
int mxq_version(void);

/* Testing aid; the pages have no counterpart.  Every on-chip pipeline wait
 * (a warp waiting for a copy, a stage or an accumulator) gives up after a
 * budget of SM clock cycles, after which the kernel winds down, the call's
 * dev_status receives MXQ_DEV_TIMEOUT and the output is incomplete.  This
 * sets that budget for kernels launched from now on by any thread of the
 * process (kernels already launched keep theirs) and returns the budget now
 * in force.  cycles <= 0 restores the default, 2e9 cycles (about one second
 * at 2 GHz); larger values are clamped to it.  The environment variable
 * MXQ_DEBUG_WAIT_BUDGET, read at the first launch, gives the initial value.
 * A CTA's waits for the copies and MMAs it issued itself, before it exits or
 * frees tensor memory, always take the default budget, so a short budget
 * leaves no asynchronous write behind a finished kernel, and a call after it
 * runs normally.                                                             */
long long mxq_debug_set_wait_budget(long long cycles);

#ifdef __cplusplus
}
#endif

#endif /* MXQ_H */
