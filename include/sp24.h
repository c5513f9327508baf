/*
 * sp24.h - C ABI of the transposable 2:4 sparse FFN kernels for MI355X (gfx950).
 *
 * Method: "Accelerating Transformer Pre-training with 2:4 Sparsity" (Hu, Zhao,
 * Huang, Chen, Zhu; ICML 2024).  Citations below name the part of that paper's
 * pages that defines each operation:
 *   [Alg.1]    Algorithm 1, "transposable mask search" (reproducibility table,
 *              "Pseudocode" row): |W|, a stride-4 correlation with the mask
 *              patterns, argmax over patterns.
 *   [Abstract] the abstract: transposable 2:4 masks computed by convolution,
 *              2:4 sparse matrix multiplication for the FFN layers.
 *   [SW]       reproducibility table, "Software Dependencies" row: separate
 *              mask-search and pruning kernels, and 2:4 sparse MMs.
 *   [Decay]    the abstract's modified sparse-refined straight-through
 *              estimator, which applies the masked decay term on gradients,
 *              and the "Software Dependencies" row's masked-decay kernel.
 *              The pages give no formula; the library adds
 *              decay * (1 - M) * W to the straight-through weight gradient.
 *   [GEGLU]    the abstract's acceleration of gated activation functions and
 *              the "Software Dependencies" row's GEGLU kernel (no formula
 *              on the pages).
 *   [MVUE]     the "Software Dependencies" row's MVUE kernel (name only).
 *              The library's reading: the minimum-variance unbiased
 *              estimator that keeps 2 of 4 entries of a gradient.
 *   [Flip]     the abstract's "flip rate", a monitor of the stability of 2:4
 *              training.  The pages give no formula; the library counts the
 *              mask entries (of the R*C) whose kept/pruned state differs
 *              between two masks, and the rate is that count over R*C.
 *
 * Conventions shared by every entry point:
 *   - W is the fp16 weight [R, C], row-major, PyTorch Linear layout [out, in].
 *   - Every pointer argument except `stream` is a DEVICE pointer owned by the
 *     caller.  The library allocates nothing, keeps no per-call state and never
 *     frees caller memory.  Buffers are contiguous and row-major, except the
 *     compressed 2:4 forms, which use the blocked order defined below.
 *   - Every device pointer must be 16-byte aligned (SP24_ERR_ALIGN otherwise).
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Calls enqueue their kernels on that stream and return at once; nothing
 *     is synchronised.  A fault inside a kernel surfaces at the caller's next
 *     synchronisation of that stream.  The stream and every buffer belong to
 *     the calling thread's current device (hipSetDevice), whose CU count
 *     picks the tiling.
 *   - Arguments are checked on the host before any HIP call, so every
 *     validation error is returned without touching the device.  A zero-sized
 *     problem (R, C or T equal to 0) is valid, launches nothing and may pass
 *     NULL for its buffers.
 *   - Calls are reentrant and thread-safe.
 *   - Inputs are expected to be finite.  +-Inf is handled deterministically
 *     (Inf scores tie and the first such pattern wins); NaN inputs give
 *     unspecified (but in-bounds) results.
 *
 * Pattern index: the 90 transposable 4x4 patterns (two kept entries in every
 * row and every column of the block) are numbered by the tuple (a, b, c, d) of
 * row-pair codes of rows 0..3, in lexicographic order, a slowest, with codes
 * 0:{0,1} 1:{0,2} 2:{0,3} 3:{1,2} 4:{1,3} 5:{2,3}.
 *
 * Compressed 2:4 storage (the pages leave the format open; this is the
 * library's fixed layout):
 *   row form     vals_row fp16 [R, C/2], meta_row uint16 [R, C/16].  Row i,
 *                group g (columns 4g..4g+3) keeps in-group positions i0 < i1:
 *                vals_row[i][2g] = W[i][4g+i0], vals_row[i][2g+1] = W[i][4g+i1]
 *                (bit copies), and the nibble (i0 | i1 << 2) sits at bits
 *                4*(g%4) .. 4*(g%4)+3 of meta_row[i][g/4].
 *   column form  vals_col fp16 [C, R/2], meta_col uint16 [C, R/16]: the same
 *                layout applied to the transpose of the pruned W (groups of 4
 *                along R).  It exists because the masks are transposable, so
 *                every column group keeps exactly two entries [Abstract].
 * The bracketed shapes above give the logical matrices; in memory each is
 * stored in BLOCKED ORDER (every vals and meta buffer of this library, in and
 * out), a permutation of the same number of elements:
 *   An n x m matrix (vals: m = C/2 halves per row, block width b = 32; meta:
 *   m = C/16 words per row, b = 4) is cut into bands of 64 rows (the last
 *   band has h = n - 64*(n/64) rows when n is not a multiple of 64).  Band k
 *   occupies elements [64*k*m, 64*k*m + h_k*m) and holds its column blocks
 *   of width b one after the other, each block row-major (h_k rows of its
 *   width; the last block of a row is m - b*(m/b) wide when b does not
 *   divide m).  So element (r, c) sits at
 *     64*k*m + b*(c/b)*h_k + (r - 64*k)*w + c%b,   k = r/64,
 *   with w = min(b, m - b*(c/b)).  One block holds the operands of 64
 *   columns of W (64 of the reduction) for 64 output rows, so a sparse
 *   product reads each of its stages as whole contiguous blocks.
 */
#ifndef SP24_H
#define SP24_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point. */
enum {
  SP24_OK = 0,
  SP24_ERR_NULL = 1,        /* a required pointer is NULL                        */
  SP24_ERR_SHAPE = 2,       /* negative size, or not a required multiple         */
  SP24_ERR_ALIGN = 3,       /* a device pointer is not 16-byte aligned           */
  SP24_ERR_LAUNCH = 4,      /* the HIP runtime rejected a kernel launch          */
  SP24_ERR_UNSUPPORTED = 5, /* not available on this device / build              */
  SP24_ERR_TOO_LARGE = 6,   /* a size exceeds the kernels' index range           */
  SP24_ERR_WORKSPACE = 7    /* the workspace is smaller than the call needs      */
};

/*
 * Transposable 2:4 mask search [Alg.1].
 *
 * For each 4x4 block (bi, bj) of |W| (rows 4bi..4bi+3, columns 4bj..4bj+3),
 * scores every pattern p as the fp32 sum of the 8 kept magnitudes added in
 * row-major order starting from +0, and writes the index of the first maximum
 * (strict >) to idx[bi * (C/4) + bj].  fp16 subnormals are kept exactly.
 *
 *   W    in   fp16 [R, C]
 *   R, C      R >= 0 and C >= 0, both multiples of 4 (a stride-4 window with
 *             no padding would drop a remainder; the call refuses it instead)
 *   idx  out  uint8 [R/4, C/4], values 0..89
 * Errors: NULL, SHAPE, ALIGN, TOO_LARGE (R*C >= 2^40), LAUNCH.
 */
int sp24_mask_search(const void* W, int64_t R, int64_t C, uint8_t* idx, void* stream);

/*
 * Prune W with the given masks and store both compressed forms [SW, Abstract].
 *
 *   W         in   fp16 [R, C]
 *   idx       in   uint8 [R/4, C/4] pattern indices (values >= 90 give
 *                  unspecified but in-bounds output)
 *   R, C           >= 0, both multiples of 16 (a meta word covers 4 groups)
 *   vals_row  out  fp16 [R, C/2]     meta_row  out  uint16 [R, C/16]
 *   vals_col  out  fp16 [C, R/2]     meta_col  out  uint16 [C, R/16]
 * Either (vals, meta) pair may be NULL to skip that form, but not both, and
 * not one pointer of a pair.
 * Errors: NULL, SHAPE, ALIGN, TOO_LARGE, LAUNCH.
 */
int sp24_compress(const void* W, const uint8_t* idx, int64_t R, int64_t C,
                  void* vals_row, uint16_t* meta_row,
                  void* vals_col, uint16_t* meta_col, void* stream);

/*
 * Mask search and compression in one pass over W [Alg.1, SW]: the same
 * results as sp24_mask_search followed by sp24_compress, with W read once.
 * idx may be NULL (not written).  Either (vals, meta) pair may be NULL, as in
 * sp24_compress.  R, C: >= 0, multiples of 16.
 * Errors: NULL, SHAPE, ALIGN, TOO_LARGE, LAUNCH.
 */
int sp24_search_compress(const void* W, int64_t R, int64_t C, uint8_t* idx,
                         void* vals_row, uint16_t* meta_row,
                         void* vals_col, uint16_t* meta_col, void* stream);

/*
 * One weight of a batched search + compression call.  W .. meta_col mean
 * what the arguments of sp24_search_compress mean; idx and either (vals,
 * meta) pair may be NULL, as there.
 *
 * Flip counting [Flip] (optional; both NULL to skip, both set to count):
 *   idx_prev  in   uint8 [R/4, C/4], the masks of the previous search (values
 *                  >= 90 are read as pattern 0).  It may be the same buffer as
 *                  idx, which is then updated in place (each block's previous
 *                  index is read before its new one is written), but it must
 *                  not overlap any other buffer of the call.
 *   flips     in/out  one uint64 in device memory, 8-byte aligned.  The call
 *                  ADDS the number of mask entries whose kept/pruned state
 *                  differs from idx_prev (an even number, at most R*C); the
 *                  caller clears it when it wants a fresh count, and several
 *                  jobs or calls may add into one counter.  The additions are
 *                  device atomics, so the total does not depend on order.
 */
typedef struct sp24_sc_job {
  const void* W;
  int64_t R;
  int64_t C;
  uint8_t* idx;
  void* vals_row;
  uint16_t* meta_row;
  void* vals_col;
  uint16_t* meta_col;
  const uint8_t* idx_prev;
  uint64_t* flips;
} sp24_sc_job;

#define SP24_MAX_BATCH 8

/*
 * sp24_search_compress for `count` weights (1..SP24_MAX_BATCH) in a single
 * kernel launch [Alg.1, SW]: an FFN layer re-searches both of its weights
 * every step, and one launch keeps the whole GPU streaming both.  `jobs` is a
 * HOST array, read during the call only.  Every job is validated first; on
 * any error nothing is launched and the first failing job's status is
 * returned.  Results are identical to separate sp24_search_compress calls.
 * Errors: NULL (jobs NULL, a job as in sp24_search_compress, or only one of
 * idx_prev and flips given), SHAPE (also count outside 1..SP24_MAX_BATCH),
 * ALIGN (flips needs 8 bytes, every other pointer 16), TOO_LARGE, LAUNCH.
 */
int sp24_search_compress_batch(const sp24_sc_job* jobs, int count, void* stream);

/*
 * Flip count between two mask-index arrays [Flip]: ADDS to *flips the number
 * of mask entries whose kept/pruned state differs between pattern idx_prev[i]
 * and pattern idx_new[i], summed over i in [0, nblocks).  Indices >= 90 are
 * read as pattern 0.  Dividing by 16*nblocks gives the flip rate.  The fused
 * form inside sp24_search_compress_batch saves this extra pass.
 *
 *   idx_prev, idx_new  in   uint8 [nblocks], 16-byte aligned
 *   nblocks                 >= 0, below 2^40
 *   flips     in/out  one uint64 in device memory, 8-byte aligned (as for
 *                     sp24_sc_job: the call adds, the caller clears)
 * Errors: NULL, SHAPE (negative nblocks), ALIGN, TOO_LARGE, LAUNCH.
 */
int sp24_flip_count(const uint8_t* idx_prev, const uint8_t* idx_new, int64_t nblocks,
                    uint64_t* flips, void* stream);

/*
 * Forward 2:4 sparse GEMM  Y = X * Ws^T  [Abstract, SW].
 *
 *   X         in   fp16 [T, C] activations
 *   vals_row, meta_row   in   row form of the pruned W [R, C]
 *   T, R, C        T >= 0; R, C >= 0 and multiples of 16
 *   Y         out  fp16 [T, R]; fp32 accumulation, rounded to nearest even
 * No bias, no activation.  Errors: NULL, SHAPE, ALIGN, TOO_LARGE, LAUNCH.
 */
int sp24_spmm_fwd(const void* X, const void* vals_row, const uint16_t* meta_row,
                  int64_t T, int64_t R, int64_t C, void* Y, void* stream);

/*
 * Forward 2:4 sparse GEMM of a gated FFN's first linear with GEGLU fused
 * into its epilogue [Abstract, SW, GEGLU]:
 *     U = X * Ws^T (fp16, as sp24_spmm_fwd), out = value * GELU(gate) of U
 * The rows of W (the output features of U) come in blocks of 32: rows
 * 32b .. 32b+15 are the value units 16b .. 16b+15 and rows 32b+16 .. 32b+31
 * their gate units, so U has sp24_geglu_fwd's layout with group 16.  `out`
 * is GEGLU of the fp16 products with the same fp32 GELU code as
 * sp24_geglu_fwd (the same inlined functions, no fp contraction), so it
 * equals sp24_geglu_fwd of U bit for bit.
 * Each value meets its gate in the same lane's accumulators, so U need not
 * be stored or read back.
 *
 *   X         in   fp16 [T, C]
 *   vals_row, meta_row   in   row form of the pruned W [R, C]
 *   T, R, C        as sp24_spmm_fwd, and R a multiple of 32
 *   U         out  fp16 [T, R], the products (for the backward), or NULL
 *   out       out  fp16 [T, R/2]
 * When C is not a multiple of 64, C is 4M or more, or an operand exceeds
 * 2 GiB, the library stores U and runs the GEGLU kernel on it; U must then be
 * given, else SP24_ERR_UNSUPPORTED.
 * Errors: NULL, SHAPE, ALIGN, UNSUPPORTED, LAUNCH; TOO_LARGE as for
 * sp24_spmm_fwd, and when T*R/16 > 2^32 - 256 (the GEGLU kernel's launch).
 */
int sp24_spmm_fwd_geglu(const void* X, const void* vals_row, const uint16_t* meta_row,
                        int64_t T, int64_t R, int64_t C, void* U, void* out, void* stream);

/*
 * Input-gradient 2:4 sparse GEMM  dX = dY * Ws  [Abstract, SW].  Uses the
 * column form, which exists because the mask is transposable.
 *
 *   dY        in   fp16 [T, R]
 *   vals_col, meta_col   in   column form of the pruned W [R, C]
 *   T, R, C        as for sp24_spmm_fwd
 *   dX        out  fp16 [T, C]; fp32 accumulation, rounded to nearest even
 * Errors: NULL, SHAPE, ALIGN, TOO_LARGE, LAUNCH.
 */
int sp24_spmm_bwd_input(const void* dY, const void* vals_col, const uint16_t* meta_col,
                        int64_t T, int64_t R, int64_t C, void* dX, void* stream);

/*
 * Several independent 2:4 sparse GEMMs in one launch [Abstract, SW]: for
 * each entry g of gemms[0..count),
 *     out[T][N] = A[T][K] * S^T,
 * S the [N, K] matrix whose 2:4 row form (groups of 4 along K) is
 * (vals, meta).  The forward product of a layer is {A = X, (vals, meta) =
 * its row form, N = R, K = C}; its input gradient is {A = dY, (vals, meta) =
 * its column form, N = C, K = R}.  Each output equals the corresponding
 * sp24_spmm_fwd / sp24_spmm_bwd_input result bit for bit.
 * One persistent launch serves every product whose K is a multiple of 64
 * and at least 192 (and whose operands each stay below 2 GiB): its
 * workgroups take 256 x 256 output tiles from per-XCD queues, the
 * products with the longest K first, so the tiles of all products share
 * the GPU without a partly filled last round per product.  Other products
 * run as single launches before it.
 *
 *   gemms     in   host array of `count` descriptors (1..SP24_MAX_GROUP)
 *   workspace in   device memory of SP24_GROUP_WORKSPACE_BYTES bytes that
 *                  must be all zero before the first call (e.g. from
 *                  hipMemset); every call that completes leaves it all zero
 *                  again.  Calls that overlap in time must use different
 *                  workspaces.
 * The products must be independent: no output may overlap any input or
 * another output.  Per product: N, K multiples of 16, T >= 0, the buffers as
 * for sp24_spmm_fwd; an empty product (T or N zero) is skipped.
 * Errors: NULL, SHAPE (also count outside 1..SP24_MAX_GROUP), ALIGN,
 * TOO_LARGE, LAUNCH.
 */
typedef struct sp24_gemm {
  const void* A;           /* fp16 [T, K] */
  const void* vals;        /* fp16 [N, K/2] */
  const uint16_t* meta;    /* uint16 [N, K/16] */
  void* out;               /* fp16 [T, N] */
  int64_t T, N, K;
} sp24_gemm;

#define SP24_MAX_GROUP 8
#define SP24_GROUP_WORKSPACE_BYTES 64

int sp24_spmm_group(const sp24_gemm* gemms, int count, void* workspace, void* stream);

/*
 * sp24_spmm_group without a workspace argument, for callers that cannot
 * allocate device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc).  The queue counters live in the
 * library's own device array of SP24_GROUP_WORKSPACE_BYTES bytes, one copy
 * per GPU, held until the process ends: zero when the library is loaded,
 * and left zero by every call that completes.  Its device address is looked
 * up (hipGetSymbolAddress) on a device's first call.  The call allocates and
 * frees nothing.  Every call on a GPU shares that GPU's array, so calls that
 * overlap in time on one GPU (on different streams) race and must not be
 * made.  Same products, results (bit for bit) and limits as
 * sp24_spmm_group: up to SP24_MAX_GROUP products, SP24_ERR_SHAPE beyond.
 * Errors: as sp24_spmm_group; LAUNCH also when the array's address cannot be
 * had.
 */
int sp24_spmm_group_noalloc(const sp24_gemm* gemms, int count, void* stream);

/*
 * Weight gradient of a 2:4 FFN linear layer with the masked decay term
 * [Decay]:
 *     dW[r][c] = sum_t dY[t][r] * X[t][c]  +  decay * (1 - M[r][c]) * W[r][c]
 * The straight-through gradient reaches the dense weight W as the dense
 * product dY^T X (fp16 products, fp32 accumulation); M is the transposable
 * mask (1 where kept) given by idx.
 *
 *   dY        in   fp16 [T, R] output gradient of the layer
 *   X         in   fp16 [T, C] input of the layer
 *   W         in   fp16 [R, C] dense weight, or NULL (no decay term)
 *   idx       in   uint8 [R/4, C/4] pattern indices (values >= 90 read as 0),
 *                  NULL exactly when W is NULL
 *   decay          the decay factor (fp32)
 *   T, R, C        T >= 0; R, C >= 0, multiples of 16; T*R and T*C < 2^30
 *   dW        out  fp32 [R, C] (written, not accumulated).  T == 0 gives the
 *                  decay term alone (zeros without W).
 * Results are deterministic.  Every output element is reduced in a fixed
 * order by one workgroup, or, when the weight has too few tiles to fill the
 * GPU (a GPT-2-1.5B FFN weight), by two: each sums one half of the tokens in
 * a fixed order, and the second half's sum, stored in dW and announced by a
 * flag, is added to the first half's (fp32 addition of two terms does not
 * depend on their order).  The flags are library memory on each GPU (64
 * sets, taken in turn by the calls that split, each left clear); up to 64
 * such calls may overlap in time on one GPU.
 * Errors: NULL (also exactly one of W and idx given), SHAPE, ALIGN,
 * TOO_LARGE, LAUNCH (also when the flags' address cannot be had).
 */
int sp24_weight_grad(const void* dY, const void* X, const void* W, const uint8_t* idx, float decay,
                     int64_t T, int64_t R, int64_t C, float* dW, void* stream);

/*
 * GEGLU forward [GEGLU]: out[t][j] = value[t][j] * GELU(gate[t][j]), GELU the
 * exact x * Phi(x) = x/2 * (1 + erf(x / sqrt 2)), fp32 arithmetic, fp16
 * result rounded to nearest even.  Phi is evaluated within 7e-7 relative of
 * its exact value; gates of +-inf give what x * Phi(x) gives in IEEE
 * arithmetic (+inf, and NaN for -inf).
 *
 *   U      in   fp16 [T, 2h], the first linear's output.  Its columns come in
 *               blocks of `group` value columns followed by the `group`
 *               matching gate columns: value j is column
 *               2*group*(j/group) + j%group, its gate is `group` columns
 *               later.  group = h is the two-halves layout [value | gate].
 *   T, h, group  T >= 0; h >= 0 and group > 0, multiples of 8; h % group == 0
 *   out    out  fp16 [T, h]
 * Errors: NULL, SHAPE, ALIGN, LAUNCH; TOO_LARGE when T*2h >= 2^40 or when
 * T*h/8 > 2^32 - 256 (one work-item per 8 units, the most one launch takes).
 */
int sp24_geglu_fwd(const void* U, int64_t T, int64_t h, int64_t group, void* out, void* stream);

/*
 * GEGLU backward [GEGLU]: dU in U's layout, with
 *   d value = dout * GELU(gate),  d gate = dout * value * GELU'(gate),
 *   GELU'(x) = Phi(x) + x * phi(x).
 *   U      in   fp16 [T, 2h] as for sp24_geglu_fwd
 *   dout   in   fp16 [T, h]
 *   dU     out  fp16 [T, 2h] (may not overlap U or dout)
 * Errors: as sp24_geglu_fwd.
 */
int sp24_geglu_bwd(const void* U, const void* dout, int64_t T, int64_t h, int64_t group,
                   void* dU, void* stream);

/*
 * MVUE 2:4 estimate of a gradient [MVUE]: every group of 4 consecutive
 * entries a_0..a_3 of a row keeps exactly two, chosen at random so that the
 * estimate is unbiased with the least summed variance.
 *   - Keep probabilities: p_i = 2|a_i| / S with S = sum |a_i|, summed left to
 *     right.  If some p_k > 1, p_k = 1 and the others are |a_j| / (S - |a_k|).
 *   - Sampling: the cumulative sums C_0 = p_0, C_1 = C_0 + p_1,
 *     C_2 = C_1 + p_2 split [0, 2).  The picks are i = #{C_j <= u} and
 *     k = #{C_j <= u + 1}.  Rounding can put u in the last interval
 *     (i == 3, which exact arithmetic never does, as u < 1 <= C_2); u + 1 is
 *     then there too, and the picks are (i, k) = (2, 3).  Before the last
 *     interval, u + 1 always lies past u's: every p_j <= 1, and the fp32
 *     evaluation below keeps that order.
 *   - Kept values are a_i / p_i (0 where p_i == 0).  A group with fewer than
 *     two non-zero entries keeps its non-zero entry (if any) and the lowest
 *     other index, unchanged.
 * Evaluation, all fp32, in this order, without division: with D = S/2
 * (uncapped) or D = S - |a_k| (capped k, the first with 2|a_k| > S; the sum of
 * the other three left to right), masses w_j = |a_j| (w_k = D) and their
 * running sums W_0..W_2, the test C_j <= u is W_j <= u*D and C_j <= u + 1 is
 * W_j <= u*D + D.  A kept value is a_k for the capped entry and +-D (the sign
 * of a_j) for any other non-zero entry: a_j / p_j in exact arithmetic.
 * Values are rounded to nearest even in fp16, so results are reproducible bit
 * for bit.  An estimate beyond the fp16 range (|D| > 65504) becomes +-inf.
 *
 *   M      in   fp16 [rows, cols], the gradient (finite)
 *   U      in   fp32 [rows, cols/4], one uniform u in [0, 1) per group,
 *               supplied by the caller
 *   rows, cols   >= 0, cols a multiple of 16
 *   vals   out  fp16 [rows, cols/2]    meta  out  uint16 [rows, cols/16]
 *               The library's 2:4 row form in blocked order: the kept pair
 *               of group g in order, and its nibble i | k << 2.  The sparse
 *               GEMMs accept it as their sparse operand.
 * Errors: NULL, SHAPE, ALIGN, LAUNCH; TOO_LARGE when a dimension reaches
 * 2^31, rows*cols reaches 2^40, or ceil(rows/64) * ceil(cols/256) > 2^24 - 1
 * (one workgroup of 256 work-items per 64 x 256 panel; one launch takes at
 * most 2^32 - 256 work-items).
 */
int sp24_mvue(const void* M, const float* U, int64_t rows, int64_t cols, void* vals, uint16_t* meta,
              void* stream);

/* Element types of the calls below that take more than one. */
enum {
  SP24_F16 = 0,
  SP24_F32 = 1,
  SP24_I32 = 2,
  SP24_I64 = 3,
  SP24_BF16 = 4,
  SP24_STATE8 = 5   /* sp24_adamw_step's states in 8 bits */
};

/* May be added to sp24_orthogonalize's out_type: products of fp16 operands. */
enum { SP24_FP16_OPERANDS = 16 };

/*
 * Token embedding: out[t] = scale * table[ids[t]], rounded to nearest even in
 * fp16.  It makes the FFN path's input from token ids.  An id outside [0, V)
 * is padding and gives a row of zeros.
 *
 *   ids     in   [T], SP24_I32 or SP24_I64 (id_type)
 *   table   in   [V, d], SP24_F16 or SP24_F32 (table_type)
 *   T, V, d      >= 0, of any size
 *   out     out  fp16 [T, d] (may not overlap the table)
 * Errors: NULL (the table may be NULL when V is 0), SHAPE, ALIGN, LAUNCH;
 * UNSUPPORTED for another type; TOO_LARGE when T, V or d reaches 2^31, a
 * matrix 2^40 entries, or the output about 2^34 chunks of 8 entries of a row
 * (of 1 entry where d is below 8).
 */
int sp24_embed_fwd(const void* ids, int id_type, int64_t T, const void* table, int table_type, int64_t V, int64_t d,
                   float scale, void* out, void* stream);

/*
 * Gradient of sp24_embed_fwd with respect to the table:
 *   dtable[v] = scale * sum over t with ids[t] == v of dout[t]
 * summed in fp32 in an order that the token positions fix (tokens of one id
 * in order, in parts of up to 64), so the same inputs give the same bits.
 * accumulate != 0 adds the sums to dtable, whose other rows are left as they
 * are (a table tied to an output layer has a gradient there already);
 * otherwise every row is written, those of absent ids with zeros.  Padding
 * ids add nothing.
 *
 *   ids        in      [T], SP24_I32 or SP24_I64 (id_type)
 *   dout       in      fp16 [T, d]
 *   dtable     out     fp32 [V, d] (in/out with accumulate)
 *   workspace  scratch device memory of sp24_embed_bwd_workspace bytes
 * Errors: NULL, SHAPE, ALIGN, LAUNCH; UNSUPPORTED for another id type;
 * WORKSPACE when workspace_bytes is too few; TOO_LARGE when T reaches 2^28, V
 * 2^27, d 2^24 - 256, or a matrix 2^40 entries.
 */
int sp24_embed_bwd(const void* ids, int id_type, int64_t T, const void* dout, int64_t V, int64_t d, float scale,
                   int accumulate, float* dtable, void* workspace, int64_t workspace_bytes, void* stream);

/* Host only: the workspace bytes of such a call; -1 for sizes it refuses. */
int64_t sp24_embed_bwd_workspace(int64_t T, int64_t V, int64_t d);

/*
 * Orthogonalises up to SP24_MAX_BATCH weight updates by Newton-Schulz
 * products.  With X [m, n] the update G or its transpose, m <= n:
 *   X_0 = G / (|G|_F + eps),   A = X X^T,   X <- a X + (b A + c A A) X
 * `steps` times, each step with its own (a, b, c).  A step maps every
 * singular value s to a s + b s^3 + c s^5 and leaves the singular vectors;
 * the usual (3.4445, -4.7750, 2.0315), five times, brings all but the
 * smallest to about 1.  A zero update gives zeros (for eps > 0).
 *
 * The products' operands are held in two fp16 parts, three products each with
 * fp32 sums, for results to about fp32's own accuracy; of out_type SP24_F16
 * they are rounded once at the end.  With the usual coefficients an update of
 * full rank comes within about 1e-5 of exact arithmetic in five steps,
 * normwise.  In directions that an update lacks, a step multiplies rounding
 * errors by a, here as in fp32 arithmetic: updates of any rank come within
 * about 3e-6 a^(steps - 1) (4e-4 in five steps, 2e-2 in eight), those whose
 * entries or rows are all alike, and so are their sums' roundings, within six
 * times that.
 *
 * With SP24_FP16_OPERANDS added to out_type the products' operands are rounded
 * to fp16 (at a scale that keeps their full precision; X itself keeps two
 * parts), for a third of the matrix work.  A result of either type is then off
 * by up to 6e-4 more a step, normwise, where the update's short side is 128 or
 * more (3e-3 in five steps), and by up to 3e-3 a step where few roundings
 * average out: with a shorter side, or with many entries alike or zero.
 *
 * The same call gives the same bits.  How the work is dealt out is chosen for
 * all weights of a call and the GPU's number of CUs, and fp32 sums with it: a
 * weight's last bits may differ between calls with other weights beside it.
 *
 * X is held to 2^-36 in absolute terms.  Smaller entries of X_0 vanish: an
 * update whose norm is far below eps loses its last bits, and in the end all.
 *
 * The weights of a call are worked on side by side: the buffers of one may not
 * overlap those of another.
 *
 *   jobs       in    host array: G [R, C] of g_type, out [R, C] of out_type
 *                    (may be G's own memory when the types agree)
 *   coef       in    host array of 3 * steps floats: a, b, c of each step.
 *                    X, A and B must stay within fp16's range: for all s that
 *                    the steps reach from [0, 1], before a step s^2, in it
 *                    b s^2 + c s^4 (with a added unless SP24_FP16_OPERANDS)
 *                    and after the last s have magnitudes up to 15.5
 *   steps            1..SP24_MAX_NS_STEPS
 *   eps              >= 0
 *   workspace        device memory of sp24_orthogonalize_workspace bytes (the
 *                    pointers in jobs do not matter to it)
 * Errors: NULL, SHAPE (also count or steps out of range), ALIGN, LAUNCH;
 * UNSUPPORTED for another type, a negative eps or coefficients that leave the
 * range (checked on the host, before anything is written); WORKSPACE;
 * TOO_LARGE when a job's (min(R, C) + 128) * (max(R, C) + 128) reaches 2^29.
 */
typedef struct sp24_ortho_job {
  const void* G;
  void* out;
  int64_t R;
  int64_t C;
} sp24_ortho_job;

#define SP24_MAX_NS_STEPS 32

int sp24_orthogonalize(const sp24_ortho_job* jobs, int count, int g_type, int out_type, const float* coef, int steps,
                       float eps, void* workspace, int64_t workspace_bytes, void* stream);

/* Host only: the workspace bytes of such a call; -1 for sizes it refuses. */
int64_t sp24_orthogonalize_workspace(const sp24_ortho_job* jobs, int count);

/*
 * One optimiser step of up to SP24_MAX_BATCH weights with momentum and an
 * orthogonalised update (sp24_orthogonalize's), in place:
 *   M <- momentum M + G
 *   U  = G + momentum M if nesterov, else M
 *   P <- (1 - decay) P - lr * orthogonalised U
 *   W  = fp16(P)
 * The last product's epilogue applies the update, so it is never written.
 * sp24_weight_grad's dW is such a G; W is the weight that
 * sp24_search_compress then searches.
 *
 *   jobs  in  host array, one per weight:
 *     G       in      fp32 [R, C]
 *     M, P    in/out  fp32 [R, C]
 *     W       out     fp16 [R, C], or NULL
 *     lr, decay       the update's factor (with any factor for the weight's
 *                     shape) and the part of P that is taken off (lr times
 *                     the weight decay)
 *   precise != 0: operands in two parts; 0: fp16 ones, as SP24_FP16_OPERANDS
 *                 says
 *   coef, steps, eps, workspace, errors: as sp24_orthogonalize
 */
typedef struct sp24_muon_job {
  const float* G;
  float* M;
  float* P;
  void* W;
  int64_t R;
  int64_t C;
  float lr;
  float decay;
} sp24_muon_job;

int sp24_muon_step(const sp24_muon_job* jobs, int count, float momentum, int nesterov, int precise, const float* coef,
                   int steps, float eps, void* workspace, int64_t workspace_bytes, void* stream);

/* Host only: the workspace bytes of such a call; -1 for sizes it refuses. */
int64_t sp24_muon_workspace(const sp24_muon_job* jobs, int count);

/* Activations of the products below, act(u) in fp32:
 *   RELU max(u, 0), RELU2 max(u, 0)^2, GELU u Phi(u), SILU u / (1 + exp(-u)),
 *   GELU_TANH u/2 (1 + tanh(sqrt(2 / pi) (u + 0.044715 u^3))). */
enum {
  SP24_ACT_NONE = 0,
  SP24_ACT_RELU = 1,
  SP24_ACT_RELU2 = 2,
  SP24_ACT_GELU = 3,
  SP24_ACT_GELU_TANH = 4,
  SP24_ACT_SILU = 5
};

/*
 * Forward 2:4 sparse GEMM of a plain layer with what follows it in the same
 * pass [Abstract, SW]:
 *     U = X * Ws^T + bias,   Y = act(U) + residual
 * fp32 throughout; U (for the backward) and Y are each rounded once, Y from
 * the unrounded U.  Made for one token as for a training batch.
 *
 *   X         in   fp16 [T, C]
 *   vals_row, meta_row   in   row form of the pruned W [R, C]
 *   T, R, C        T >= 0; R, C >= 0 and multiples of 16
 *   bias      in   fp32 [R], or NULL
 *   act            SP24_ACT_*
 *   residual  in   fp16 [T, R], or NULL
 *   U         out  fp16 [T, R], or NULL
 *   Y         out  fp16 [T, R]; may be the residual's own memory (if that is not
 *             X's too: other rows' products read X).  Apart from that U and Y
 *             share no memory with each other or with what the call reads.
 *   workspace scratch device memory of sp24_spmm_fwd_act_workspace bytes (NULL
 *             where those are 0)
 * U of +inf gives +inf; of -inf 0 with RELU, RELU2 and GELU, NaN with GELU_TANH
 * and SILU (-inf * 0); NaN gives NaN.
 * Errors: NULL, SHAPE, ALIGN, WORKSPACE, LAUNCH; UNSUPPORTED for another act;
 * TOO_LARGE as for sp24_spmm_fwd, and when R reaches 2^27.
 */
int sp24_spmm_fwd_act(const void* X, const void* vals_row, const uint16_t* meta_row, int64_t T, int64_t R, int64_t C,
                      const float* bias, int act, const void* residual, void* U, void* Y, void* workspace,
                      int64_t workspace_bytes, void* stream);

/* Host only: the workspace bytes of such a call; -1 for sizes it refuses. */
int64_t sp24_spmm_fwd_act_workspace(int64_t T, int64_t R, int64_t C);

/*
 * Input-gradient 2:4 sparse GEMM through the activation before the layer, with
 * the gradient of that activation's bias [Abstract, SW]:
 *     dU = (dY * Ws) * act'(U),   dbias[c] = sum over t of dU[t][c]
 * The layer's input is act(U), U = its predecessor's products with their bias:
 * dU is the gradient that the predecessor's weight and input gradients take.
 * RELU's and RELU2's slope at 0 is 0, and where U <= 0 they give 0 whatever the
 * product is, infinite and NaN ones too; where U is NaN so is dU, but RELU's is the
 * product alone.  U of an infinity: RELU, RELU2 and GELU have their limits, GELU_TANH
 * and SILU NaN.  fp32 throughout; the sums are of the
 * unrounded values, in an order that T, R and C fix, so the same call gives
 * the same bits.
 *
 *   dY        in   fp16 [T, R]
 *   vals_col, meta_col   in   column form of the pruned W [R, C]
 *   T, R, C        as sp24_spmm_fwd_act
 *   act            SP24_ACT_*; U may be NULL with SP24_ACT_NONE
 *   U         in   fp16 [T, C]
 *   dU        out  fp16 [T, C]; may be U's own memory (if that is not dY's too).
 *             Apart from that dU and dbias share no memory with each other or
 *             with what the call reads.
 *   dbias     out  fp32 [C], or NULL.  Written, not accumulated (zeros if T is 0).
 *   workspace scratch device memory of sp24_spmm_bwd_input_act_workspace bytes
 *             (NULL where those are 0)
 * Errors: as sp24_spmm_fwd_act (C reaching 2^27).
 */
int sp24_spmm_bwd_input_act(const void* dY, const void* vals_col, const uint16_t* meta_col, int64_t T, int64_t R,
                            int64_t C, int act, const void* U, void* dU, float* dbias, void* workspace,
                            int64_t workspace_bytes, void* stream);

/* Host only: the workspace bytes of such a call; -1 for sizes it refuses. */
int64_t sp24_spmm_bwd_input_act_workspace(int64_t T, int64_t R, int64_t C);

/*
 * Bias gradient of a layer that no activation follows: dbias[r] = sum over t of
 * dY[t][r], in fp32 in an order that T and R fix.
 *
 *   dY        in   fp16 [T, R]
 *   T, R           >= 0, R a multiple of 16
 *   dbias     out  fp32 [R], written (zeros if T is 0)
 *   workspace scratch device memory of sp24_bias_grad_workspace bytes (NULL where
 *             those are 0)
 * Errors: NULL, SHAPE, ALIGN, WORKSPACE, LAUNCH; TOO_LARGE when T reaches 2^31,
 * R 2^27 or dY 2^40 entries.
 */
int sp24_bias_grad(const void* dY, int64_t T, int64_t R, float* dbias, void* workspace, int64_t workspace_bytes,
                   void* stream);

/* Host only: the workspace bytes of such a call; -1 for sizes it refuses. */
int64_t sp24_bias_grad_workspace(int64_t T, int64_t R);

/*
 * What a training step's optimiser goes by, in device memory, so that no call
 * waits for the host: sp24_grad_norm writes it, sp24_adamw_step reads it.  All
 * zeros before the first step.
 */
typedef struct sp24_step_control {
  int64_t step;     /* steps taken, this one included: bias correction's t  */
  float norm;       /* of the scaled gradients, before clipping             */
  float factor;     /* what the gradients are multiplied with               */
  int32_t skip;     /* 1: some gradient is not finite; the step is left out */
  int32_t unused[3];
} sp24_step_control;

/*
 * The norm of all gradients of a step together:
 *     norm = scale * sqrt(sum of squares),  factor = scale * min(1, max_norm / norm)
 * into *control.  If some gradient is not finite, skip becomes 1, factor 0 and
 * step stays; otherwise skip becomes 0 and step grows by 1.  Squares are summed
 * in fp64, in an order that the sizes fix.
 *
 *   grads     in   host array of `count` device pointers, all of g_type
 *   sizes     in   host array: the number of entries of each, >= 0
 *   count          >= 0
 *   g_type         SP24_F16 or SP24_F32
 *   scale          > 0, finite: what a loss scale left in the gradients is taken off with
 *   max_norm       > 0; infinity: gradients are not clipped
 *   control   in/out  one sp24_step_control in device memory
 *   workspace scratch device memory of sp24_grad_norm_workspace bytes
 * Errors: NULL, SHAPE, ALIGN, WORKSPACE, LAUNCH; UNSUPPORTED for another type,
 * scale or max_norm; TOO_LARGE when a size reaches 2^34.
 */
int sp24_grad_norm(const void* const* grads, const int64_t* sizes, int64_t count, int g_type, float scale,
                   float max_norm, sp24_step_control* control, void* workspace, int64_t workspace_bytes, void* stream);

/* Host only: the workspace bytes of such a call; -1 for sizes it refuses. */
int64_t sp24_grad_norm_workspace(const int64_t* sizes, int64_t count);

/*
 * One AdamW step of `count` tensors, in place.  With g = factor * G (factor and
 * the step t from `control`; 1 and `step` without one):
 *   M <- beta1 M + (1 - beta1) g,   V <- beta2 V + (1 - beta2) g^2
 *   P <- (1 - decay) P - lr * (M / (1 - beta1^t)) / (sqrt(V / (1 - beta2^t)) + eps)
 *   W  = fp16(P)
 * Where control->skip is set, or no step was counted yet, nothing is written.
 *
 * State type SP24_F32: M and V are fp32 [n].  SP24_STATE8: M and V are 8-bit
 * codes [n] with one exponent byte for every 64 consecutive entries, M_exps and
 * V_exps [ceil(n / 64)]; all zeros stand for zeros.  An M entry has a sign and
 * 3 fraction bits, the root of a V entry, which is what is held, 4; both have 4
 * exponent bits below their group's exponent.  The step uses this step's M and
 * V before they are rounded; rounded they go up or down at random (unbiased),
 * by a hash of seed, t, the tensor's place in the call and the entry's in the
 * tensor, so the same call gives the same bits; a root above zero stays above
 * zero.  A group in which some entry is not finite turns to NaN.
 *
 *   jobs  in  host array, one per tensor:
 *     G       in      [n] of g_type (SP24_F16 or SP24_F32)
 *     P       in/out  fp32 [n]
 *     M, V    in/out  fp32 [n], or codes
 *     M_exps, V_exps  in/out  uint8 [ceil(n / 64)] (SP24_STATE8; otherwise not read)
 *     W       out     fp16 [n], or NULL
 *     n               >= 0
 *     lr, decay       the update's factor and the part of P that is taken off
 *                     (lr times the weight decay)
 *   beta1, beta2      0 <= beta < 1;  eps >= 0, rounded to fp32: if it is 0 there
 *                     an entry whose V is 0 in fp32 is divided by 0
 *   step              t >= 1 (not read with a control)
 *   control   in      one sp24_step_control in device memory, or NULL
 * What the jobs hold, beta1, beta2, eps and seed are taken as the call is made: a
 * captured call replays them, lr and decay too.
 * Pointers are 16-byte aligned, the exponents' at any byte.  The buffers of a
 * call may not overlap.
 * Errors: NULL, SHAPE (also step below 1), ALIGN, LAUNCH; UNSUPPORTED for
 * another type, beta or eps; TOO_LARGE when an n reaches 2^34.
 */
typedef struct sp24_adamw_job {
  const void* G;
  float* P;
  void* M;
  void* V;
  uint8_t* M_exps;
  uint8_t* V_exps;
  void* W;
  int64_t n;
  float lr;
  float decay;
} sp24_adamw_job;

int sp24_adamw_step(const sp24_adamw_job* jobs, int64_t count, int g_type, int state_type, double beta1, double beta2,
                    double eps, int64_t step, const sp24_step_control* control, uint32_t seed, void* stream);

/*
 * The values that an 8-bit state stands for: M's entries, or with root != 0 the
 * roots of V's.
 *   codes  in   uint8 [n]     exps  in  uint8 [ceil(n / 64)], at any byte
 *   n           >= 0
 *   out    out  [n] of out_type: SP24_F32, or SP24_BF16, which holds such values
 *               whole unless their group's largest is below 2^-110
 * Errors: NULL, SHAPE, ALIGN, LAUNCH; UNSUPPORTED for another type; TOO_LARGE
 * when n reaches 2^34 - 1024.
 */
int sp24_state8_values(const uint8_t* codes, const uint8_t* exps, int64_t n, int root, int out_type, void* out,
                       void* stream);

/* Host only: a static, human-readable name for a status code. */
const char* sp24_status_str(int status);

/*
 * Host only: writes the 90 patterns in index order to out[0..89] (host
 * memory).  Bit 4r+c of out[p] is set when pattern p keeps entry (r, c) of
 * the block.  Returns SP24_OK, or SP24_ERR_NULL for a NULL out.
 */
int sp24_pattern_table(uint16_t* out);

/* Host only: the library's ABI version (8 for this header). */
int sp24_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SP24_H */
