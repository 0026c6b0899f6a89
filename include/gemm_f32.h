/*
 * gemm_f32.h -- C ABI of the MI355X (gfx950) fp32 matrix-product library.
 *
 * The operation is the dense product C = A x B of the pages on shared-memory
 * tiling ("03 CUDA Shared Memory: Tiling, Bank Conflicts, and Reduction",
 * section "Shared Memory와 Tiling"; PMPP chapter 5 notes
 * "메모리 계층과 데이터 지역성", sections 5.4 and 5.5): every output element is
 * the dot product of one row of A with one column of B, matrices are stored
 * row by row, sizes need not be multiples of the tile because out-of-range
 * tile slots hold zero, and only the final store is range checked.  The pages
 * state it for square Width x Width matrices; this interface takes the
 * general M x K times K x N case with BLAS-style leading dimensions (an
 * offset sub-matrix view is a base pointer plus a leading dimension, as in
 * the first page's "Global Memory와 Coalescing" section).
 *
 * Layout (all three matrices row-major, binary32):
 *   A is M x K,  element (i, k) at A[i*lda + k],  lda >= max(1, K)
 *   B is K x N,  element (k, j) at B[k*ldb + j],  ldb >= max(1, N)
 *   C is M x N,  element (i, j) at C[i*ldc + j],  ldc >= max(1, N)
 *
 * Result: C[i*ldc + j] = sum_{k<K} A[i*lda + k] * B[k*ldb + j] for i < M,
 * j < N, rounded in binary32 (summation order and fused multiply-adds vary
 * by kernel; see the accuracy note below).  C is OVERWRITTEN (no alpha, no
 * beta, C is never read).  Entries of C outside the M x N window -- the
 * padding between N and ldc -- are never written.  K == 0 writes +0 to the
 * whole window.  M == 0 or N == 0 is a no-op that returns GEMM_F32_OK.
 *
 * Memory and ownership: A, B and C are DEVICE pointers on the current HIP
 * device, owned by the caller; the library allocates nothing, keeps no
 * pointer after returning and holds no state (the one exception is the
 * fixed 1 MiB scratch array of reduce_sum_f32_variant_noalloc, a static
 * device variable, and its address per device).  A and B are read only.  C
 * must not overlap A or B (the result is undefined otherwise).  Pointers need
 * 4-byte alignment only; 16-byte alignment is not required.
 *
 * Streams and errors: `stream` is a hipStream_t (NULL = the null stream).
 * Every call only enqueues work: it returns before the product is computed,
 * and the caller synchronises the stream to see the result.  Argument errors
 * are detected synchronously, before anything is enqueued, and are returned
 * as a nonzero status with no launch.  GEMM_F32_ERR_LAUNCH reports a launch
 * rejected by the HIP runtime; a fault during execution surfaces at the
 * caller's next synchronisation, as for any HIP kernel.  All entry points are
 * thread safe.
 *
 * Accuracy: the result of every kernel satisfies, per element,
 *   |C - C_exact| <= 1e-5 * sum_k |A_ik| |B_kj|
 * on the workloads the library is tested on, and is bit exact whenever every
 * product and partial sum is an integer below 2^24 in magnitude (for
 * instance small-integer inputs).
 */
#ifndef GEMM_F32_H
#define GEMM_F32_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes.  Every entry point returns one, synchronously, before it
 * enqueues anything: the host-program habit of the one-volume PMPP notes
 * ("PMPP 단권화", chapter 2, host program structure), which checks the
 * status of every runtime call and reports it by name, carried over to the
 * library's own argument checks.  The codes and their texts
 * (gemm_f32_status_string) are this library's own. */
#define GEMM_F32_OK                  0
#define GEMM_F32_ERR_INVALID_DIM     1  /* M, N or K negative                       */
#define GEMM_F32_ERR_INVALID_LD      2  /* lda < max(1,K), ldb or ldc < max(1,N)     */
#define GEMM_F32_ERR_NULL_PTR        3  /* a pointer is NULL while its matrix is non-empty */
#define GEMM_F32_ERR_MISALIGNED      4  /* a pointer is not 4-byte aligned           */
#define GEMM_F32_ERR_INVALID_VARIANT 5  /* unknown kernel variant                    */
#define GEMM_F32_ERR_TOO_LARGE       6  /* M, N or K >= 2^31, or the grid would not fit */
#define GEMM_F32_ERR_LAUNCH          7  /* the HIP runtime rejected the launch       */
#define GEMM_F32_ERR_DEVICE          8  /* no usable current HIP device              */
#define GEMM_F32_ERR_INVALID_OP      9  /* op_a or op_b is neither N nor T           */
#define GEMM_F32_ERR_WORKSPACE      10  /* workspace smaller than required            */
#define GEMM_F32_ERR_INVALID_FORMAT 11  /* 16-bit input format unknown                */
#define GEMM_F32_ERR_SCRATCH        12  /* partials would exceed the fixed scratch      */
#define GEMM_F32_ERR_INVALID_TYPE   13  /* a stored type the entry point does not take */
#define GEMM_F32_ERR_INVALID_ACTIVATION 14 /* activation unknown                       */
#define GEMM_F32_ERR_INVALID_EPILOGUE 15 /* an epilogue field its mode does not take   */
#define GEMM_F32_ERR_INVALID_SCALAR 16  /* eps, a coefficient or a step count out of range */
#define GEMM_F32_ERR_OVERLAP        17  /* an output overlaps another tensor of its call  */

/* Kernel ladder.  Each rung computes the same product; each is tested against
 * the oracle and against the rung below it.
 *   0  naive: one thread per output element, 16 x 16 workgroups, operands read
 *      straight from global memory (PMPP one-volume notes, naive matrix
 *      product; first page, naive kernel)
 *   1  LDS-tiled: the pages' tiled kernel with T = 32 -- 32 x 32 A and B tiles
 *      staged cooperatively in LDS with ghost zeros, two barriers per phase,
 *      rows padded by 4 words, 128-bit coalesced global loads
 *   2  register-blocked, double-buffered: 128 x 128 workgroup tile, 8 x 8
 *      outputs per thread in registers, two LDS buffers and one barrier per
 *      phase, next tile prefetched into registers during the current phase
 *   3  MFMA: v_mfma_f32_32x32x2_f32 matrix-core contraction on double-
 *      buffered LDS tiles (the default).  The tile follows from how full the
 *      last round of 256 workgroups would run: 256 x 256 tiles with direct
 *      global-to-LDS copies into an XOR-swizzled layout (on four waves with
 *      a fixed instruction order when K, M and N are multiples of 4
 *      and each stored factor is under 2 GiB, else on eight waves; both give
 *      the same bits), else 128 x 128 tiles, else 64 x 64 tiles whose phases
 *      are split over four groups of four waves.  With K, M and N multiples
 *      of 4, 64 x 64 tiles whose four waves each run the whole tile over
 *      every fourth phase (partial tiles added in wave order, so results are
 *      deterministic and the same for every op pair) replace that choice
 *      where a cost model of rounds, per-kernel efficiency and fixed cost
 *      per tile gives them the shorter time (K >= 448), or in place of the
 *      split-phase tiles (K >= 384); then 96 x 96 tiles of the same kind
 *      (16-deep phases) where the model gives them the shorter time (K >=
 *      448), and, from K = 256, 64 x 64 tiles of four waves with one 32 x
 *      32 block each over the whole K (three blocks sharing a CU) where the
 *      model, charging their fixed cost once per launch, does.  Products of at most 1024 output tiles
 *      of 16 x 16 take small tiles instead (16 x 16 on 8 waves up to 512 of
 *      them, else 32 x 32 on 4 waves), whose K is split over the waves of
 *      each block, operands loaded straight into registers for
 *      v_mfma_f32_16x16x4_f32, partial tiles added in wave order.
 *      gemm_f32_default_variant() names the configuration a shape runs.
 * Variants numbered from 16 up are diagnostic layouts of the same rungs, kept
 * so that their hardware counters can be compared; see
 * gemm_f32_variant_name().
 */
#define GEMM_F32_VARIANT_NAIVE    0
#define GEMM_F32_VARIANT_TILED    1
#define GEMM_F32_VARIANT_REGBLOCK 2
#define GEMM_F32_VARIANT_MFMA     3

/* C = A x B with the library's best kernel for the shape (the MFMA rung). */
int gemm_f32(int64_t M, int64_t N, int64_t K,
             const float *A, int64_t lda,
             const float *B, int64_t ldb,
             float *C, int64_t ldc,
             void *stream);

/* Same contract, with the kernel chosen by `variant` (see above).
 * Returns GEMM_F32_ERR_INVALID_VARIANT for an unknown number. */
int gemm_f32_variant(int variant,
                     int64_t M, int64_t N, int64_t K,
                     const float *A, int64_t lda,
                     const float *B, int64_t ldb,
                     float *C, int64_t ldc,
                     void *stream);

/* Products with a transposed factor: C = op(A) x op(B), C still M x N.
 *
 * The one-volume PMPP notes (deep-learning chapter, backward pass) need the
 * weight gradient X^T dY and the input gradient dY W^T besides the forward
 * product, and run all three on the same tile kernel; so does this entry
 * point (the MFMA rung, with each factor's LDS tile kept in the orientation
 * in which it is stored).
 *   op_a == GEMM_F32_OP_N: A is stored M x K, element (i,k) at A[i*lda + k],
 *                          lda >= max(1, K)
 *   op_a == GEMM_F32_OP_T: A is stored K x M, element (i,k) of op(A) at
 *                          A[k*lda + i], lda >= max(1, M)
 *   op_b == GEMM_F32_OP_N: B is stored K x N, element (k,j) at B[k*ldb + j],
 *                          ldb >= max(1, N)
 *   op_b == GEMM_F32_OP_T: B is stored N x K, element (k,j) of op(B) at
 *                          B[j*ldb + k], ldb >= max(1, K)
 * C, ownership, streams, errors and accuracy are as for gemm_f32; an op
 * other than N or T returns GEMM_F32_ERR_INVALID_OP.  For a given M, N, K
 * the k-summation order does not depend on the ops, so op(A) = A^T gives
 * the same bits as gemm_f32 on an explicitly transposed copy.
 */
#define GEMM_F32_OP_N 0
#define GEMM_F32_OP_T 1
int gemm_f32_op(int op_a, int op_b,
                int64_t M, int64_t N, int64_t K,
                const float *A, int64_t lda,
                const float *B, int64_t ldb,
                float *C, int64_t ldc,
                void *stream);

/* Introspection.  These calls are this library's own (the pages define no
 * such interface): they launch nothing, need no device, and exist so that
 * tests, benchmarks and counter runs can name the kernels they measure.
 *
 * Number of ladder rungs (variants 0 .. n-1). */
int gemm_f32_num_variants(void);

/* Static, NUL-terminated name of a variant, or NULL if it does not exist.
 * Valid numbers are 0 .. gemm_f32_num_variants()-1 and the diagnostic
 * numbers 16 .. 16 + gemm_f32_num_diagnostic_variants() - 1. */
const char *gemm_f32_variant_name(int variant);

/* Number of diagnostic variants (numbered from 16). */
int gemm_f32_num_diagnostic_variants(void);

/* The diagnostic variant whose configuration gemm_f32 and gemm_f32_op run
 * for an M x N x K product (the choice depends on the sizes only; the
 * four-wave configuration hands a stored factor of 2 GiB or more to the
 * eight-wave kernel), or -1 for sizes that are
 * negative or above INT_MAX.  Launches nothing, needs no device; for callers
 * that want to know which kernel a call will use. */
int gemm_f32_default_variant(int64_t M, int64_t N, int64_t K);

/* Measurement helper, this library's own (not part of the product): a loop
 * of non-packed binary32 fused multiply-adds on the vector ALU -- the
 * register-blocked rung's instruction -- whose time, measured by the caller,
 * gives that instruction's issue rate on the device.
 *   form    0: one operand in a scalar register; 1: all operands in vector
 *           registers, 16 independent accumulators per lane; 2: an 8 x 8
 *           outer product of vector registers (the rung's inner step)
 *   blocks  workgroups of 256 threads (4 waves) to launch, >= 1
 *   iters   loop trips: each lane does iters x 16 FMAs (forms 0 and 1) or
 *           (iters / 4) x 64 (form 2)
 *   out     device pointer to blocks x 256 floats, overwritten (keeps the
 *           results live)
 *   stamps  device pointer to blocks x 4 x 4 uint64_t (8-byte aligned): for
 *           wave w, stamps[4w .. 4w+3] = shader clock counter and 100 MHz
 *           counter at the start, then at the end of its loop
 * Enqueue-only on `stream`; statuses as for gemm_f32 (an unknown form gives
 * GEMM_F32_ERR_INVALID_VARIANT). */
int gemm_f32_valu_probe(int form, int64_t blocks, int iters, float *out, uint64_t *stamps,
                        void *stream);

/* Measurement helper, this library's own (not part of the product): one
 * wave (a single workgroup of 64 threads) reads LDS, lane l at byte offset
 * offsets[l] of a 64 KB array (masked into it and aligned down to the read's
 * width), `iters` times; with a profiler's LDS bank-conflict counter per
 * dispatch, a chosen set of offsets shows which lanes one read cycle serves.
 *   form     0 ds_read_b32, 1 ds_read_b64, 2 ds_read_b128,
 *            3 ds_read_b64_tr_b16
 *   offsets  device pointer to 64 int32 byte offsets (4-byte aligned)
 *   out      device pointer to 64 uint32, overwritten (keeps the reads live)
 * Enqueue-only on `stream`; statuses as for gemm_f32 (an unknown form gives
 * GEMM_F32_ERR_INVALID_VARIANT, iters < 0 GEMM_F32_ERR_INVALID_DIM). */
int gemm_f32_lds_probe(int form, const int32_t *offsets, int iters, uint32_t *out, void *stream);

/* Measurement helper, this library's own (not part of the product): the
 * rate at which a CU brings 1 KB wave loads (16 bytes a lane, as the 16-bit
 * kernels' copies) from an L2-resident buffer, into LDS or into registers.
 * Each workgroup (4 waves) reads its own 64 KB of src, wave w the 16 KB at
 * 16 KB w, cycling through it `iters` x 8 times with 8 to 16 loads in flight.
 *   mode    0: buffer loads into LDS; 1: buffer loads into vector registers
 *   blocks  workgroups of 256 threads, >= 1 (one per CU for a per-CU rate)
 *   iters   loop trips, even, >= 0
 *   src     device pointer, 16-byte aligned, to blocks x 65536 bytes
 *           (blocks x 64 KB should fit the L2 caches)
 *   out     device pointer to blocks x 256 uint32, overwritten
 *   cycles  device pointer to blocks x 4 uint64 (8-byte aligned): each
 *           wave's shader clock cycles for its loop
 * Enqueue-only on `stream`; statuses as for gemm_f32 (an unknown mode gives
 * GEMM_F32_ERR_INVALID_VARIANT, odd or negative iters
 * GEMM_F32_ERR_INVALID_DIM). */
int gemm_f32_copy_probe(int mode, int64_t blocks, int iters, const void *src, uint32_t *out, uint64_t *cycles,
                        void *stream);

/* Measurement helper, this library's own (no page defines it): gemm_f32's
 * k-split kernel (64 x 64 tiles whose four waves each take every fourth
 * phase of the tile; gemm_f32 runs it for square1000-sized products) on an
 * instantiation that also records when each wave passes five points.  A, B,
 * C and every size, leading dimension and status as for gemm_f32 with both
 * factors as stored; C receives the same bits as gemm_f32 gives with the
 * k-split kernel.  The problem must be one that kernel takes (M, N, K
 * multiples of 4, K > 0, M and N > 0), else GEMM_F32_ERR_INVALID_DIM.
 *   timeline        device buffer of timeline_words uint32 words, 4-byte
 *                   aligned; timeline_words a positive multiple of 32
 *                   (GEMM_F32_ERR_INVALID_DIM otherwise)
 * Block b < timeline_words / 32 (in launch order), wave w, writes words
 * 8 (4 b + w) .. + 7: the 100 MHz real-time counter at the wave's start,
 * when its first phase has landed in LDS, after its last matrix instruction
 * is issued, after the barrier before the partial tiles are added, and after
 * its stores have completed; its shader-clock cycles between the first and
 * the last; its phase count; b.  Other words are not written.  The
 * instantiation waits for its stores before the last stamp, which the
 * product kernel does not.  Enqueue-only on `stream`. */
int gemm_f32_ksplit_timeline(int64_t M, int64_t N, int64_t K, const float *A, int64_t lda, const float *B,
                             int64_t ldb, float *C, int64_t ldc, uint32_t *timeline, int64_t timeline_words,
                             void *stream);

/* Static, NUL-terminated description of a status code (the by-name report
 * of the chapter 2 error check cited with the codes above); "unknown status"
 * for any other number. */
const char *gemm_f32_status_string(int status);

/* Shared-tile transpose: out = in^T, binary32, row-major.
 *
 * The first page's "Bank Conflict" section transposes through a tile held
 * in shared memory -- read rows of `in` and write rows of `out`, both
 * coalesced, reading the tile by columns in between -- and uses it to show
 * bank conflicts and their cures (padding, XOR swizzle).
 *   in  is rows x cols, element (r, c) at in[r*ld_in + c],   ld_in  >= max(1, cols)
 *   out is cols x rows, element (c, r) at out[c*ld_out + r], ld_out >= max(1, rows)
 * out[c*ld_out + r] = in[r*ld_in + c] exactly; words of out outside the
 * cols x rows window are never written.  Device pointers, caller-owned, 4-byte
 * aligned; out must not overlap in.  rows or cols == 0 is a no-op.  Status
 * codes, streams and asynchrony as for gemm_f32 (GEMM_F32_ERR_INVALID_LD for
 * a too-small leading dimension, GEMM_F32_ERR_INVALID_VARIANT for an unknown
 * variant).
 * Variants: 0 naive (no LDS), 1 [32][32] tile (the page's kernel), 2 [32][33]
 * padded tile, 3 XOR-swizzled [32][32] tile, 4 64 x 64 tile with 128-bit
 * global and LDS accesses and an LDS layout conflict free on gfx950, 5 the
 * same with 128 x 128 tiles, 6 variant 4 with tiles handed out in diagonal
 * order, 7 and 8 variants 6 and 4 with nontemporal global loads and stores,
 * 9 and 10 variant 6 and its 128 x 128 form with nontemporal stores only.
 * transpose_f32 uses 9 when the 64 x 64 tile grid is square or the input
 * holds 128 MiB or more, else 6 (diagonal order: with leading dimensions
 * near a multiple of 4 KB, tiles handed out row by row crowd the same memory
 * channels; nontemporal stores keep the caches for the input);
 * transpose_f32_default_variant names that choice (-1 for negative sizes or
 * sizes above INT_MAX), launching nothing.
 */
int transpose_f32(int64_t rows, int64_t cols, const float *in, int64_t ld_in,
                  float *out, int64_t ld_out, void *stream);
int transpose_f32_variant(int variant, int64_t rows, int64_t cols, const float *in,
                          int64_t ld_in, float *out, int64_t ld_out, void *stream);
int transpose_f32_num_variants(void);
const char *transpose_f32_variant_name(int variant);   /* NULL if unknown */
int transpose_f32_default_variant(int64_t rows, int64_t cols, int64_t ld_in, int64_t ld_out);

/* Sum reduction: *out = x[0] + ... + x[n-1], binary32.
 *
 * The first page's "Reduction" section folds an array into one value with a
 * tree in shared memory, improves the tree step by step (interleaved, then
 * sequential addressing, then warp shuffles for the last steps, then one
 * atomic per block), and reduces large arrays in several passes (each block
 * folds its values to one partial, then the partials are folded again).
 *   x          device pointer to n floats (4-byte aligned), read only
 *   out        device pointer to one float, overwritten (+0 when n == 0)
 *   workspace  device memory of at least reduce_sum_f32_workspace_size()
 *              bytes for the partials (NULL allowed when that size is 0);
 *              owned by the caller, contents undefined after the call; it
 *              must not overlap x or out
 * The summation order depends on the variant and on n only, except for
 * variant 3, whose block sums are added by float atomics in arrival order:
 * its last bits may vary from run to run.  The error is bounded by
 * (longest sequential chain + tree depth) * 2^-24 * sum |x_i|; the result is
 * exact when every partial sum is an integer below 2^24 in magnitude.
 * Variants: 0 interleaved pairs (the thread owning a pair's left slot adds),
 * 1 sequential addressing (the lowest-numbered threads add), 2 sequential +
 * wave shuffles for the last six steps, 3 one atomic add per block, 4
 * grid-stride 128-bit loads + wave shuffles + a one-block second pass (the
 * default).  Statuses as for gemm_f32, plus GEMM_F32_ERR_WORKSPACE.
 */
int64_t reduce_sum_f32_workspace_size(int variant, int64_t n);   /* bytes; -1 if invalid */
int reduce_sum_f32(int64_t n, const float *x, float *out,
                   void *workspace, int64_t workspace_bytes, void *stream);
int reduce_sum_f32_variant(int variant, int64_t n, const float *x, float *out,
                           void *workspace, int64_t workspace_bytes, void *stream);
int reduce_sum_f32_num_variants(void);
const char *reduce_sum_f32_variant_name(int variant);  /* NULL if unknown */

/* reduce_sum_f32_variant without a workspace, for callers that cannot
 * allocate device memory: code under HIP stream capture, serving loops that
 * must not call the allocator, harnesses that forbid it.  It calls no
 * allocator (the library's, HIP's or torch's) at any point.
 *   The partials go to a fixed array of REDUCE_SUM_F32_SCRATCH_BYTES (1 MiB)
 * that the library holds in the device memory of every GPU it runs on, for
 * the life of the process.  Its address on a device is looked up on the
 * first call with that device current.
 *   Limit: a problem whose partials need more than that scratch, i.e. whose
 * reduce_sum_f32_workspace_size(variant, n) exceeds
 * REDUCE_SUM_F32_SCRATCH_BYTES, is rejected with GEMM_F32_ERR_SCRATCH
 * before anything is enqueued.  Variants 3 and 4 fit for any n; variants
 * 0-2 need about 4 n / 255 bytes, so they take n up to about 6.7e7.
 *   Sharing: every call on one GPU uses that GPU's one scratch array, which
 * keeps the last call's contents.  Calls that overlap on one GPU -- on two
 * streams, or from two host threads without ordering -- race and give
 * undefined results.  Calls on one stream are ordered and safe.
 *   Arguments, results, summation order (the same bits as
 * reduce_sum_f32_variant for variants 0-2 and 4), statuses and asynchrony
 * are as for reduce_sum_f32_variant. */
#define REDUCE_SUM_F32_SCRATCH_BYTES (1 << 20)
int reduce_sum_f32_variant_noalloc(int variant, int64_t n, const float *x, float *out,
                                   void *stream);

/* Mixed-precision product: C (binary32) = A x B with A and B in a 16-bit
 * format, accumulated in binary32.
 *
 * The one-volume PMPP notes ("PMPP 단권화", deep-learning chapter, "FC Layer
 * = GEMM" and "Mixed Precision") run the fully connected layer as a matrix
 * product on matrix units that take FP16 or BF16 inputs and accumulate in
 * FP32; BF16 keeps FP32's exponent range, FP16 does not.
 *   format   GEMM_MIXED_BF16 (bfloat16: 1 sign, 8 exponent, 7 fraction bits)
 *            or GEMM_MIXED_F16 (IEEE binary16: 1 sign, 5 exponent, 10
 *            fraction bits); both factors use the same format
 *   A        M x K, element (i, k) at A[i*lda + k], lda >= max(1, K), 16-bit
 *            patterns, 2-byte aligned
 *   B        K x N, element (k, j) at B[k*ldb + j], ldb >= max(1, N), same
 *   C        M x N binary32, element (i, j) at C[i*ldc + j], ldc >= max(1, N),
 *            4-byte aligned
 * Leading dimensions count elements.  C[i*ldc + j] = sum_k a_ik b_kj: every
 * product of two 16-bit values is exact in binary32, the sum is accumulated
 * in binary32 (the accuracy bound of gemm_f32 applies, measured against the
 * exact product of the 16-bit values), and the result is bit exact whenever
 * every partial sum is an integer below 2^24 in magnitude.  Rounding binary32
 * data to 16 bits is the caller's step, before the call.  Overwrite, window,
 * K == 0, empty-size, ownership, stream and error rules as for gemm_f32; an
 * unknown format returns GEMM_F32_ERR_INVALID_FORMAT.  Operands whose bases
 * are 4-byte aligned with even leading dimensions use vector loads; others
 * are served by element-wise loads (correct, slower).
 * gemm_mixed picks the tile shape for the problem; gemm_mixed_variant runs
 * tile configuration `variant` (0 .. gemm_mixed_num_variants() - 1, named by
 * gemm_mixed_variant_name).  Below 128 tiles of 128 x 128 (and below 128 of
 * 256 x 256) with K a multiple of 8, gemm_mixed and gemm_mixed_op take
 * 64 x 64 tiles whose four waves each run the whole tile over every fourth
 * 32-deep phase (mixed64x64_bk32_w4_ksplit, v_mfma_f32_16x16x32; partial
 * tiles added in wave order, so every op pair gives the same bits); it needs
 * what the scheduled configurations need (below), and a problem it does not
 * take runs the element-wise 64 x 64 kernel.  With 128 to 256 tiles of
 * 128 x 128 and K >= 1024 (a multiple of 8) they take the same split on
 * 128 x 128 tiles (mixed128x128_bk32_w4_ksplit), with the same needs; a
 * problem it does not take runs mixed128x128_bk64_w2x2_directAB (aligned) or
 * the element-wise 128 x 128 kernel.  The scheduled configurations
 * -- mixed256x256_bk64_w4_wide (v_mfma_f32_16x16x32; gemm_mixed's and
 * gemm_mixed_op's choice once there are 128 tiles of 256 x 256),
 * mixed192x192_bk64_w4_wide (the same kernel on 192 x 192 tiles; their
 * choice, with K even, where its tiles need fewer rounds of the 256 CUs at
 * 0.8 of a 256 tile's time each, or, below 128 tiles of 256 x 256, with at
 * least 140 of 192 x 192 or, for K % 8 != 0, 32 of them with K < 1536 (or
 * K % 4 == 2 and fewer than 128 tiles of 128 x 128)),
 * mixed160x160_bk64_w4_wide (the same kernel on 160 x 160 tiles; their
 * choice wherever 192 x 192 tiles would be, if the 160 x 160 ones need no
 * more rounds of the 256 CUs),
 * mixed256x256_rowsplit (their choice, with K a multiple of 8, where the
 * last round of 256 x 256 tiles would be under 40 % full: the rows filling
 * the other rounds on the 256 x 256 kernel, the remaining rows on k-split
 * 128 x 128 tiles if at most 256 of them, else on 160 x 160 tiles if they
 * need no more rounds of the 256 CUs than 192 x 192 ones, else on 192 x 192
 * tiles; two launches in stream order),
 * mixed256x256_bk64_w4_sched (the same schedule on v_mfma_f32_32x32x16) and
 * mixed256x256_bk32_w4_wide4stage (16x16x32 with four 32-deep LDS stages) --
 * take K a multiple of 8 (the 16x16x32 wide ones on 256, 192 and 160 tiles: K even), N even (M
 * too for A stored transposed in gemm_mixed_op, and not N for B stored
 * transposed), 4-byte aligned operands with even leading dimensions and
 * operands under 2^31 bytes; edge tiles run whole and store only inside C,
 * and k positions past K contribute zeros.  Other
 * problems given to them run mixed256x256_bk64_w2x4_directAB (for the
 * 32 x 32 x 16 configuration the same tiles and summation order, the same
 * bits; for the 16 x 16 x 32 ones another instruction, other bits within the
 * same bound).
 */
#define GEMM_MIXED_BF16 0
#define GEMM_MIXED_F16  1

int gemm_mixed(int format, int64_t M, int64_t N, int64_t K,
               const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
               float *C, int64_t ldc, void *stream);
int gemm_mixed_variant(int variant, int format, int64_t M, int64_t N, int64_t K,
                       const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                       float *C, int64_t ldc, void *stream);
int gemm_mixed_num_variants(void);
const char *gemm_mixed_variant_name(int variant);   /* NULL if unknown */
/* The configuration gemm_mixed runs for an M x N x K product (the scheduled
 * configurations hand problems they do not take to
 * the 8-wave fallback, as described above), or -1 for sizes that are negative
 * or above INT_MAX.  Launches nothing, needs no device. */
int gemm_mixed_default_variant(int64_t M, int64_t N, int64_t K);

/* C (binary32) = op(A) x op(B) for 16-bit factors, either one stored
 * transposed: the backward-pass products X^T dY and dY W^T of the same
 * deep-learning chapter ("Backward"), in mixed precision.
 *   op_a = GEMM_F32_OP_N: A stored M x K (lda >= max(1, K));
 *   op_a = GEMM_F32_OP_T: A stored K x M (lda >= max(1, M)), op(A) = A^T;
 *   op_b = GEMM_F32_OP_N: B stored K x N (ldb >= max(1, N));
 *   op_b = GEMM_F32_OP_T: B stored N x K (ldb >= max(1, K)), op(B) = B^T.
 * Everything else as for gemm_mixed (formats, alignment, accuracy, errors;
 * GEMM_F32_ERR_INVALID_OP for another op value).  The factors are read in
 * place; for a given M, N and K the result has the same bits whichever way
 * the factors are stored, as long as each storage meets the conditions of
 * the configuration gemm_mixed picks: from 128 tiles of 256 x 256 on, a
 * storage that does not (an odd M for A stored transposed, an odd N for B
 * as stored, an odd leading dimension, a 2-byte aligned base) runs the
 * 8-wave fallback on v_mfma_f32_32x32x16, whose bits differ within the same
 * bound. */
int gemm_mixed_op(int op_a, int op_b, int format, int64_t M, int64_t N, int64_t K,
                  const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                  float *C, int64_t ldc, void *stream);

/* Stored types of the entry points below: the 16-bit formats' numbers, and
 * binary32. */
#define GEMM_MIXED_F32 2

/* Activations.  At infinities each takes its limit, -0 or +0 and +inf, and so
 * does its derivative, 0 and 1: a kept pre-activation past binary16's range is
 * infinite.  NaN stays NaN. */
#define GEMM_ACT_NONE      0
#define GEMM_ACT_RELU      1  /* max(z, 0), NaN stays NaN; derivative 0 at 0            */
#define GEMM_ACT_GELU      2  /* z Phi(z), Phi the normal distribution function         */
#define GEMM_ACT_GELU_TANH 3  /* z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2         */
#define GEMM_ACT_SILU      4  /* z / (1 + e^-z)                                         */

/* What a product's entries pass through before they are stored.
 *   gradient == 0, the layer's forward pass:
 *     Z = op(A) op(B) + bias          (bias added to every row)
 *     C = act(Z) + residual
 *     preact, if not NULL, receives Z rounded to the factors' format
 *   gradient == 1, the backward pass through an activation that comes before
 *   the product in the network:
 *     C = (op(A) op(B) + residual) * act'(Z), Z read from preact
 *     bias_grad, if not NULL, receives the N column sums of C, added in
 *     binary32 before C's rounding, in a fixed order
 * Fields: */
typedef struct gemm_epilogue {
    int c_type;           /* type of C and residual: the factors' format or GEMM_MIXED_F32  */
    int activation;       /* GEMM_ACT_*                                                     */
    int gradient;         /* 0 or 1                                                         */
    int bias_type;        /* type of bias: the factors' format or GEMM_MIXED_F32            */
    const void *bias;     /* N values, or NULL; NULL in gradient mode                       */
    const void *residual; /* M x N, or NULL; may be C itself (same pointer, leading dimension) */
    int64_t ld_residual;  /* >= max(1, N) where residual is set                             */
    void *preact;         /* M x N of the factors' format, or NULL; needed in gradient mode
                             unless the activation is GEMM_ACT_NONE                         */
    int64_t ld_preact;    /* >= max(1, N) where preact is used                              */
    float *bias_grad;     /* N sums, or NULL; NULL in forward mode                          */
} gemm_epilogue;

/* The 16-bit product with its epilogue: the fully connected layer of the
 * same deep-learning chapter ("FC Layer = GEMM", "Backward"), the epilogue in
 * the product's kernel.  A product of few tiles whose K is split over blocks
 * (and one of operands past 2 GiB, or of K == 0) passes through binary32
 * planes in the workspace.
 *   op_a, op_b, format, M, N, K, A, lda, B, ldb   as for gemm_mixed_op; any
 *            alignment of 2 bytes and any leading dimension are taken
 *   C        M x N of epilogue->c_type, element (i, j) at C[i*ldc + j];
 *            aligned to its type's size, as are bias, residual and preact
 *   workspace, workspace_bytes   device memory of at least
 *            gemm_mixed_epilogue_workspace_size() bytes for the same
 *            arguments (NULL allowed when that is 0), 16-byte aligned, owned
 *            by the caller until the call has run; contents undefined after
 *            it.  Two calls that may overlap need a workspace each.
 * Products and sums are accumulated in binary32 and every stored value is
 * rounded once.  C must not overlap A, B or preact, nor residual unless it
 * is residual (the same pointer with another leading dimension is refused with
 * GEMM_F32_ERR_INVALID_LD, here and below).  K == 0 leaves a product of zeros to the epilogue; M == 0
 * writes +0 to bias_grad; N == 0 is a no-op.  Statuses as for gemm_mixed,
 * with GEMM_F32_ERR_INVALID_TYPE, _ACTIVATION and _EPILOGUE for the
 * epilogue's fields and GEMM_F32_ERR_WORKSPACE.  Enqueue-only on `stream`;
 * calls no allocator and may be captured into a graph. */
int64_t gemm_mixed_epilogue_workspace_size(int op_a, int op_b, int format, int64_t M, int64_t N, int64_t K,
                                           const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                                           const gemm_epilogue *epilogue);   /* bytes; -1 if invalid */
int gemm_mixed_epilogue(int op_a, int op_b, int format, int64_t M, int64_t N, int64_t K,
                        const uint16_t *A, int64_t lda, const uint16_t *B, int64_t ldb,
                        void *C, int64_t ldc, const gemm_epilogue *epilogue,
                        void *workspace, int64_t workspace_bytes, void *stream);

/* The layer's forward pass with a weight held in 4 bits, for a decoder's few
 * rows: the product of gemm_mixed_epilogue (op_b T) with
 *   W[n][k] = scales[n][k / group] (q[n][k] - zeros[n][k / group])
 * which is never formed: whole numbers meet A in the matrix units, and a group's
 * binary32 sum meets the scale.
 *   format     of A, scales and zeros (16-bit values)
 *   Q          N rows of (K + 1) / 2 bytes: q[n][k], 0 .. 15, in the low half of
 *              byte n*ldq + k / 2 for an even k, in the high half for an odd
 *              one; any alignment, ldq >= max(1, (K + 1) / 2)
 *   group      k per scale: 32, 64 or a multiple of 128 (a whole row's: any
 *              multiple not below K); the last group may be cut off by K
 *   scales     N rows of ceil(K / group), ld_scales >= max(1, that)
 *   zeros      likewise, any values; or NULL: 8 throughout
 *   epilogue   forward mode only
 * Any number of rows is taken; the weight is expanded once for every 64 of
 * them, so that past a few hundred a 16-bit weight is the better choice.  Sums
 * are binary32, of x (16 + q) with 16 + zero times the sum of x taken off: their
 * error is that of binary32 sums of the terms scale |x| (16 + q + 16 + |zero|),
 * not of scale |x (q - zero)|, which are 12 (values spread evenly, zero 8) to 24
 * times smaller in all (normal weights) and may be 0.  A 16-bit product of
 * the same whole numbers is up to 6 times closer in binary32, which a 16-bit
 * result does not show.  For the same reason finite bfloat16 x give infinities
 * or NaN where such a sum over up to 128 k passes binary32's range (not below |x|
 * of 2^116 with zeros of -15 .. 15), and an infinity in A gives NaN.  The workspace, of
 * gemm_w4_epilogue_workspace_size() bytes, and the rest as for
 * gemm_mixed_epilogue; M at most 65535 * 64, N at most 2^25. */
int64_t gemm_w4_epilogue_workspace_size(int64_t M, int64_t N, int64_t K);   /* bytes; -1 if invalid */
int gemm_w4_epilogue(int format, int64_t M, int64_t N, int64_t K, const uint16_t* A, int64_t lda, const uint8_t* Q,
                     int64_t ldq, int64_t group, const uint16_t* scales, int64_t ld_scales, const uint16_t* zeros,
                     int64_t ld_zeros, void* C, int64_t ldc, const gemm_epilogue* epilogue, void* workspace,
                     int64_t workspace_bytes, void* stream);

/* The gradient mode without a product, for a gradient dY that is already
 * there: dZ = dY * act'(Z), and the bias gradient, dZ's column sums.
 *   format      GEMM_MIXED_BF16 or GEMM_MIXED_F16, of dY, preact and dZ
 *   dY          M x N, ld_dy >= max(1, N)
 *   preact      Z, M x N, ld_preact >= max(1, N); may be NULL if the
 *               activation is GEMM_ACT_NONE
 *   dZ          M x N, ld_dz >= max(1, N), may be dY itself (same pointer and
 *               leading dimension), or NULL for the sums alone
 *   bias_grad   N binary32 sums (of dZ before its rounding, in a fixed
 *               order), or NULL; needs the workspace
 * Rules as for gemm_mixed_epilogue. */
int64_t activation_grad_workspace_size(int64_t M, int64_t N);   /* bytes; -1 if invalid */
int activation_grad(int activation, int format, int64_t M, int64_t N, const uint16_t *dY, int64_t ld_dy,
                    const uint16_t *preact, int64_t ld_preact, uint16_t *dZ, int64_t ld_dz, float *bias_grad,
                    void *workspace, int64_t workspace_bytes, void *stream);

/* The layer whose rows belong to groups with a weight each: the experts of a
 * mixture, each with the rows that were sent to it, sorted by expert.  Group
 * g has the rows offsets[g] .. offsets[g + 1] - 1 of A, C, residual and preact:
 *   Z = A op(B_g) + bias_g,  C = act(Z) + residual     for the rows of group g
 * in one launch over all groups.  With B the weights in their other
 * orientation it is also the backward pass's input gradient, dX = dZ W_g^T.
 *   groups    0 .. 65535; a group may be empty
 *   M         rows of A and C (those of all groups, and others)
 *   B         group g's K x N matrix (op_b N; N x K for T) at B + g*stride_b,
 *             leading dimension ldb; stride_b >= 0 elements
 *   offsets   DEVICE pointer to groups + 1 int32 (4-byte aligned), read when
 *             the call runs: not decreasing, 0 <= offsets[0], offsets[groups]
 *             <= M.  The library cannot check them; others give undefined
 *             values in C and preact, but no access outside the matrices.
 *   epilogue  forward mode only (GEMM_F32_ERR_INVALID_EPILOGUE); bias_g at
 *             bias + g*ld_bias elements, ld_bias >= 0
 * Rows of no group (before offsets[0], from offsets[groups] on) are neither
 * read nor written: C and preact keep what they held there.  Everything else
 * as for gemm_mixed_epilogue: types, alignment of one element, any leading
 * dimension, roundings, workspaces, graphs, statuses. */
int64_t gemm_mixed_grouped_workspace_size(int op_b, int format, int64_t groups, int64_t M, int64_t N, int64_t K,
                                          const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb,
                                          int64_t stride_b, const int32_t* offsets, const gemm_epilogue* epilogue,
                                          int64_t ld_bias);   /* bytes; -1 if invalid */
int gemm_mixed_grouped(int op_b, int format, int64_t groups, int64_t M, int64_t N, int64_t K, const uint16_t* A,
                       int64_t lda, const uint16_t* B, int64_t ldb, int64_t stride_b, const int32_t* offsets, void* C,
                       int64_t ldc, const gemm_epilogue* epilogue, int64_t ld_bias, void* workspace,
                       int64_t workspace_bytes, void* stream);

/* The weights' gradients of the same layer: C_g = A_g^T B_g, M x N, summed over
 * the rows of group g (A = X, B = dZ for weights stored K x N; A = dZ, B = X for
 * N x K).  An empty group's gradient is +0.
 *   A, B      rows x M and rows x N, as stored
 *   C         group g's at C + g*stride_c, of c_type (format or
 *             GEMM_MIXED_F32), stride_c >= (M - 1) ldc + N if groups > 1
 * Sums are binary32; the rest as above. */
int64_t gemm_mixed_grouped_grad_workspace_size(int format, int64_t groups, int64_t rows, int64_t M, int64_t N,
                                               const uint16_t* A, int64_t lda, const uint16_t* B, int64_t ldb,
                                               const int32_t* offsets, int c_type);   /* bytes; -1 if invalid */
int gemm_mixed_grouped_grad(int format, int64_t groups, int64_t rows, int64_t M, int64_t N, const uint16_t* A,
                            int64_t lda, const uint16_t* B, int64_t ldb, const int32_t* offsets, int c_type, void* C,
                            int64_t ldc, int64_t stride_c, void* workspace, int64_t workspace_bytes, void* stream);

/* activation_grad for the same layer: dZ = dY * act'(Z) on the groups' rows
 * (dZ keeps what it held on others), and bias_grad, groups x N binary32 sums of
 * dZ over each group's rows, before its rounding, in a fixed order (+0 for an
 * empty group). */
int64_t activation_grad_grouped_workspace_size(int64_t groups, int64_t M, int64_t N);   /* bytes; -1 if invalid */
int activation_grad_grouped(int activation, int format, int64_t groups, int64_t M, int64_t N, const uint16_t* dY,
                            int64_t ld_dy, const uint16_t* preact, int64_t ld_preact, const int32_t* offsets,
                            uint16_t* dZ, int64_t ld_dz, float* bias_grad, void* workspace, int64_t workspace_bytes,
                            void* stream);

/* Layer norm over the rows of a rows x cols matrix (cols >= 1).
 *   mean = <x>, rstd = 1 / sqrt(<(x - mean)^2> + eps), <.> over a row
 *   y = (x - mean) rstd gamma + beta
 *   type         of x and y: GEMM_MIXED_BF16, _F16 or _F32
 *   x, y         element (r, c) at x[r*ldx + c], ldx >= cols; y may be x with
 *                the same leading dimension
 *   gamma, beta  cols values of param_type (any of the three), or NULL (1, 0)
 *   eps          >= 0, finite
 *   mean, rstd   rows binary32 values for the backward pass, or NULL
 * Statistics are binary32; the variance is the mean of the squared
 * deviations.  rows == 0 is a no-op.  Statuses, streams and alignment (each
 * pointer to its type's size) as above. */
int layer_norm(int type, int64_t rows, int64_t cols, const void *x, int64_t ldx, int param_type, const void *gamma,
               const void *beta, float eps, void *y, int64_t ldy, float *mean, float *rstd, void *stream);

/* Its backward pass, with xhat = (x - mean) rstd and g = dy gamma:
 *   dx     = rstd (g - <g> - xhat <g xhat>) + residual_grad
 *   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
 *   dy, x, dx      of type, with leading dimensions >= cols; dx may be dy or
 *                  residual_grad, with the same leading dimension
 *   mean, rstd     as the forward pass wrote them
 *   gamma          cols values of param_type, or NULL (1)
 *   residual_grad  the gradient that reaches x past the layer, of type, or NULL
 *   dgamma, dbeta  cols binary32 sums, added in a fixed order, or NULL;
 *                  +0 when rows == 0
 *   workspace      as for gemm_mixed_epilogue; none is needed with dgamma and
 *                  dbeta both NULL */
int64_t layer_norm_backward_workspace_size(int type, int64_t rows, int64_t cols);   /* bytes; -1 if invalid */
int layer_norm_backward(int type, int64_t rows, int64_t cols, const void *dy, int64_t lddy, const void *x,
                        int64_t ldx, const float *mean, const float *rstd, int param_type, const void *gamma,
                        const void *residual_grad, int64_t ld_residual, void *dx, int64_t lddx, float *dgamma,
                        float *dbeta, void *workspace, int64_t workspace_bytes, void *stream);

/* The norm over all of a model's gradients, and their clipping.
 *   norm = sqrt(sum over the tensors and their values of g^2)
 *   out  = g min(1, max_norm / (norm + eps))
 *   count     tensors; grads, out, sizes and types are HOST arrays of that
 *             length, read before the call returns
 *   grads     device pointers to sizes[i] values each, in one run of memory, of
 *             types[i]: GEMM_MIXED_BF16, _F16 or _F32, mixed as they come;
 *             aligned to the type's size.  A size of 0 is skipped, and its
 *             pointer may be NULL
 *   out       likewise; out[i] may be grads[i].  Outputs must overlap nothing
 *             else in the lists (GEMM_F32_ERR_OVERLAP): a tensor listed twice
 *             counts twice in grad_norm and is refused in place
 *   norm      device pointer to one binary32 value: written by grad_norm and
 *             grad_clip_norm, read by grad_clip (so that the norms of shards
 *             can be joined in between); in both calls of clipping no part of
 *             an output, in grad_clip_norm of a gradient neither
 *             (GEMM_F32_ERR_OVERLAP)
 *   max_norm  >= 0, finite;  eps > 0, finite
 *   workspace of grad_norm_workspace_size() bytes, as for gemm_mixed_epilogue
 * Squares are added in binary64 in a fixed order, so that no binary32 value is
 * too large or too small to count; the norm is rounded to binary32, the factor
 * is computed from it and rounded to binary32, and every value times the factor
 * to binary32 and then to its type.  In place with a factor of 1 nothing is
 * written.  A norm that is infinite (an infinity among the values, or finite ones
 * whose norm passes binary32) gives a factor of 0 (0, and NaN in place of
 * infinities), a NaN gives NaN: look at the norm before the update.  Without
 * tensors the norm is +0.  Statuses, streams and graphs as above; a captured
 * graph holds the lists as they were. */
int64_t grad_norm_workspace_size(int64_t count, const int64_t *sizes);   /* bytes; -1 if invalid */
int grad_norm(int64_t count, const void *const *grads, const int64_t *sizes, const int *types, float *norm,
              void *workspace, int64_t workspace_bytes, void *stream);
int grad_clip(int64_t count, const void *const *grads, void *const *out, const int64_t *sizes, const int *types,
              const float *norm, float max_norm, float eps, void *stream);
/* Both; of up to 128 tensors in a launch less. */
int grad_clip_norm(int64_t count, const void *const *grads, void *const *out, const int64_t *sizes, const int *types,
                   float max_norm, float eps, float *norm, void *workspace, int64_t workspace_bytes, void *stream);

/* Orthogonalisation of `batch` rows x cols matrices by Newton-Schulz
 * products (the update step of the Muon optimiser).  Per matrix,
 *   X <- G / (|G|_F + eps), then `steps` times
 *   X <- a X + (b S + c S^2) X with S = X X^T          (rows <= cols)
 *   X <- a X + X (b S + c S^2) with S = X^T X          (rows > cols)
 * so that every singular value s of X goes to a s + b s^3 + c s^5.
 *   type        of G and out: GEMM_MIXED_BF16, _F16 or _F32
 *   batch       at most 65535
 *   rows, cols  4 (rows + 256) (cols + 256) below 2^31, each first rounded up
 *               to a multiple of 64 (22848 x 22848, 16384 x 32000)
 *   G           matrix z's element (r, c) at G[z*stride_g + r*ldg + c], ldg >=
 *               cols, stride_g >= 0
 *   out         likewise with ldo, stride_o; matrices must not overlap
 *               (stride_o >= (rows - 1) ldo + cols when batch > 1); may be G
 *               with the same strides
 *   steps       0 .. 100
 *   a, b, c     finite; refused (GEMM_F32_ERR_INVALID_SCALAR) if singular
 *               values of at most 1 could pass 2^40 within the steps
 *   eps         >= 0, finite; with eps > 0 a matrix of zeros gives zeros
 *   workspace   of newton_schulz_workspace_size() bytes, as for
 *               gemm_mixed_epilogue
 * Accuracy is that of the matrix as a whole, not of each entry: X is kept to 22
 * bits of entries above 2^-16 of its norm, smaller ones lose bits one by one,
 * and below 2^-39 (1.8e-12) they are 0, so that singular values and rows that
 * small stay 0 however many steps follow.  Five default steps of binary32
 * matrices whose rows or columns are scaled over 1 .. 1e-9 (1000 x 600): 1e-6 or
 * less of a row's root mean square down to 1e-3 of the largest, 1.4e-4 at 1e-6,
 * 0.13 at 1e-9; bfloat16 results 2e-3, 2e-3, 0.13.  Products of a binary32
 * result take 22-bit factors, those of a bfloat16 one past 64 x 64 11-bit
 * factors (error 1.7e-3 to 2e-3 of the result's root mean square, 1.66e-3 of it
 * the rounding of the result).
 * A matrix with a NaN or an infinity gives NaN throughout; the other
 * matrices of the batch do not see it.  Statuses as above. */
int64_t newton_schulz_workspace_size(int type, int64_t batch, int64_t rows, int64_t cols);   /* bytes; -1 if invalid */
int newton_schulz(int type, int64_t batch, int64_t rows, int64_t cols, const void *G, int64_t ldg, int64_t stride_g,
                  int steps, float a, float b, float c, float eps, void *out, int64_t ldo, int64_t stride_o,
                  void *workspace, int64_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F32_H */
