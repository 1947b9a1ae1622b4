/*
 * gemm_f32.h -- C ABI of libgemmf32.so, single-precision dense matrix
 * multiply C = A * B for one NVIDIA GB300 (sm_103a).
 *
 * Operation ("Lecture 12: final project", runguoli.com ECE408 notes l12,
 * section 2, the general M/N/K kernel tiledMatMulKernel, and section 3, the
 * CPU golden reference):
 *
 *     C[i][j] = sum_{k < K} A[i][k] * B[k][j]      0 <= i < M, 0 <= j < N
 *
 * Layout: A is M x K, B is K x N, C is M x N, all packed row-major
 * (leading dimensions K, N and N elements).  There is no alpha, beta or
 * transpose: C is overwritten.  All three are 4-byte floats in DEVICE memory
 * of the current CUDA device; any alignment is accepted (4-byte aligned
 * pointers that are not 16-byte aligned, and row strides that are not a
 * multiple of 16 bytes, are served through an internal padded copy).
 *
 * Accuracy: every algorithm is checked against the double-accumulating CPU
 * reference within |C - C_ref| <= 1e-3 + 1e-3 |C_ref| elementwise (the
 * section 4 atol/rtol of the same page).  Results are run-to-run
 * deterministic for a given (shape, algo, splits) on a given device.
 *
 * Edge semantics (same page, section 7, the early exits of main): a negative
 * dimension is an error; M == 0 or N == 0 returns success and launches
 * nothing; K == 0 writes C = 0.  Elements of memory outside C are never
 * written (out-of-range rows and columns of a boundary tile are skipped, the
 * lecture-5 coarsened kernel's predicated store).
 *
 * Ownership and ordering: the caller owns A, B and C; the library reads A
 * and B, writes C and its own workspace, and keeps no reference to any of
 * them after the call returns.  Every call is asynchronous on `stream`
 * (enqueue and return; no implicit synchronisation).  The library owns a
 * workspace per (device, stream), grown on demand: a call that must grow it
 * synchronises that stream first.  cudaStreamPerThread counts as a stream of
 * each host thread (whose workspace goes once the thread has ended and another
 * thread's is made).  gemm_f32_release() frees all of it.  The entry points
 * are thread-safe.
 *
 * CUDA graphs: the calls that take a stream can be captured from it
 * (cudaStreamBeginCapture) and replayed; the graph keeps the pointers,
 * shapes and plan of the capture and reads what the buffers hold at replay.
 * The first call on a device sets it up, and a call may have to grow the
 * stream's workspace (or the host entry's device copies); neither is done
 * during a capture, so such a call returns GEMM_F32_ERR_CAPTURE without
 * enqueuing anything.  Issue each captured call once on the same stream
 * before capturing it.  A captured call does not use the stream's workspace
 * and device copies: it gets some that belong to its graph, shared by the
 * calls that the capture takes from one stream, so graphs may be replayed on
 * any streams, at the same time as one another and as calls on the stream of
 * the capture (gemm_f32_noalloc's scratch is one for all calls: see there).
 * When the graph and the executables made from it are
 * destroyed, that memory serves later captures; gemm_f32_release() frees it:
 * do not release while a graph that holds such a call may still be replayed.
 *
 * Errors: 0 is success.  Negative values are library errors (GEMM_F32_ERR_*),
 * positive values are the cudaError_t of the failing CUDA runtime call.  No
 * entry point exits or aborts the process.  Nothing runs on the host CPU:
 * there is no CPU fallback, and a device other than sm_103 is rejected.
 */
#ifndef GEMM_F32_H
#define GEMM_F32_H

#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- status codes ------------------------------------------------------ */
#define GEMM_F32_SUCCESS                 0
/* negative dimension; NULL pointer with a nonzero extent; unknown algo;
 * splits out of range; C overlapping A or B; a size product that overflows */
#define GEMM_F32_ERR_INVALID_VALUE      (-1)
/* no CUDA device, or the current device is not compute capability 10.3 */
#define GEMM_F32_ERR_UNSUPPORTED_DEVICE (-2)
/* the workspace could not be allocated */
#define GEMM_F32_ERR_WORKSPACE          (-3)
/* a kernel gave up waiting on one of its own pipeline barriers (watchdog) */
#define GEMM_F32_ERR_DEVICE_TIMEOUT     (-4)
/* the driver rejected a tensor-memory-access descriptor */
#define GEMM_F32_ERR_DESCRIPTOR         (-5)
/* the stream is being captured into a CUDA graph and the call would first
 * have to set up this device or the stream's buffers (a larger workspace, the
 * host entry's device copies), which is not done during a capture: issue the
 * same call once on the stream before capturing it.  Nothing was enqueued. */
#define GEMM_F32_ERR_CAPTURE            (-6)

/* ---- algorithms -------------------------------------------------------- */
/* Choose by shape: the tensor-core 3xTF32 kernels, except the CUDA-core
 * kernel for tiny problems (under 5e7 multiply-adds); among the tensor-core
 * kernels, those that split A and B in shared memory when staging them
 * would cost more than it saves (few flops per operand element). */
#define GEMM_F32_ALGO_AUTO    0
/* CUDA-core FFMA kernel: TMA-fed, swizzled shared-memory tiles, mbarrier
 * pipeline, 8x8 or 8x16 register tile per thread. */
#define GEMM_F32_ALGO_FFMA    1
/* Tensor-core kernel: each operand x split into a TF32 high part trunc(x)
 * (the fp32 word itself, which the tensor core reads truncated) and a TF32
 * low part tf32(x - trunc(x)); three tcgen05 products hi*hi + hi*lo + lo*hi
 * accumulated in tensor memory in fp32, promoted every 128 K into fp32
 * registers.  Non-finite operands: an Inf's low part is Inf - Inf = NaN, so
 * an output that is +-Inf in exact arithmetic may come back NaN; NaN inputs
 * still give NaN, and outputs whose row of op(A) and column of op(B) are
 * finite are unaffected.  The FFMA kernel follows IEEE fp32 there. */
#define GEMM_F32_ALGO_3XTF32  2

/* Largest explicit split-K factor accepted by gemm_f32_algo_splitk. */
#define GEMM_F32_MAX_SPLITS   256

/*
 * gemm_f32 -- C = A * B with the algorithm the library picks for the shape.
 * Same as gemm_f32_algo(A, B, C, M, N, K, GEMM_F32_ALGO_AUTO, stream).
 * A: M*K floats, B: K*N floats, C: M*N floats, device pointers, row-major.
 */
int gemm_f32(const float* A, const float* B, float* C, int M, int N, int K,
             cudaStream_t stream);

/*
 * gemm_f32_algo -- as gemm_f32 with an explicit per-call algorithm
 * (GEMM_F32_ALGO_*).  There is no global state: the choice applies to this
 * call only.  The split-K factor is chosen by the library.
 */
int gemm_f32_algo(const float* A, const float* B, float* C, int M, int N, int K,
                  int algo, cudaStream_t stream);

/*
 * gemm_f32_algo_splitk -- as gemm_f32_algo with an explicit split of the
 * K dimension.  splits == 0 lets the library choose; 1 disables splitting;
 * 2..GEMM_F32_MAX_SPLITS computes that many partial products over disjoint
 * K ranges into the workspace and adds them in a fixed order (split 0 first)
 * in a separate kernel, so the result is deterministic.  A split count
 * larger than the number of K blocks is reduced to it.
 */
int gemm_f32_algo_splitk(const float* A, const float* B, float* C, int M, int N, int K,
                         int algo, int splits, cudaStream_t stream);

/*
 * gemm_f32_ex -- the general row-major form
 *
 *     C = alpha * op(A) * op(B) + beta * C
 *
 * op(A) is M x K: element (i, k) is A[i*lda + k] (transa == 0, A stored
 * M x K, lda >= K) or A[k*lda + i] (transa == 1, A stored K x M, lda >= M).
 * op(B) is K x N: element (k, j) is B[k*ldb + j] (transb == 0, ldb >= N) or
 * B[j*ldb + k] (transb == 1, B stored N x K, ldb >= K).  C[i][j] is
 * C[i*ldc + j], ldc >= N.  Leading dimensions are in elements.  With
 * beta == 0 the old C is not read (NaN or garbage there is harmless); with
 * alpha == 0 or K == 0 A and B are not read and C = beta * C.  algo and
 * splits as for gemm_f32_algo_splitk.  Operands that TMA cannot read in
 * place (transposed for the CUDA-core kernel, or a row stride / base not
 * 16-byte aligned) are first copied into the workspace.  The pages have only
 * the packed alpha = 1, beta = 0 form; this is the same product with the
 * interface a BLAS-style caller expects.  transa or transb other than 0 or
 * 1, or a leading dimension below its minimum, is GEMM_F32_ERR_INVALID_VALUE.
 */
int gemm_f32_ex(int transa, int transb, int M, int N, int K, float alpha, const float* A,
                long long lda, const float* B, long long ldb, float beta, float* C,
                long long ldc, int algo, int splits, cudaStream_t stream);

/*
 * gemm_f32_algo_splitk_ev -- as gemm_f32_algo_splitk, and, for profiling,
 * records `main_begin` on `stream` just before the main GEMM kernel is
 * launched and `main_end` just after it (either may be NULL).  The events
 * must belong to the current device.  Staging copies and the split-K
 * reduction, when a call has them, fall outside the pair.
 */
int gemm_f32_algo_splitk_ev(const float* A, const float* B, float* C, int M, int N, int K,
                            int algo, int splits, cudaStream_t stream,
                            cudaEvent_t main_begin, cudaEvent_t main_end);

/*
 * gemm_f32_host -- C = A * B where A, B and C are HOST pointers (row-major,
 * same shapes as gemm_f32).  The library copies B to the device, then walks
 * row panels of A and C: the copy of panel i+1 of A, the GEMM of panel i
 * and the copy back of panel i-1 of C run at the same time on the call's
 * stream and two internal streams.  For deep K with M <= 4096 it walks K
 * panels instead (each accumulates into C, the first GEMM starts after one
 * panel of A and B has arrived, the last panel returns C by row blocks).  Page-locked host memory is needed for
 * that overlap (pageable memory works, serialised).  Asynchronous on
 * `stream`: the host buffers must stay valid, and C is complete, only when
 * `stream` has reached the end of the call.  Device copies of A, B and C
 * are kept in a library buffer per (device, stream), grown on demand like
 * the workspace; gemm_f32_release() frees them.  Same status codes.
 */
int gemm_f32_host(const float* A, const float* B, float* C, int M, int N, int K, int algo,
                  cudaStream_t stream);

/*
 * gemm_f32_plan_info / gemm_f32_plan -- what a call with these arguments
 * would launch, without launching anything.  Needs a device (it reads the
 * SM count); returns a status code like the compute entry points.
 */
typedef struct gemm_f32_plan_info {
    int algo;            /* resolved GEMM_F32_ALGO_FFMA or _3XTF32 (0 if no launch) */
    int splits;          /* resolved split-K factor (1 = none) */
    int tile_m;          /* output tile rows per CTA */
    int tile_n;          /* output tile columns per CTA */
    int tile_k;          /* K depth of one pipeline stage */
    int stages;          /* pipeline stages in shared memory */
    int ctas;            /* CTAs in the main kernel's grid */
    int stage_a;         /* 1 if A goes through a staging copy */
    int stage_b;         /* 1 if B goes through a staging copy */
    int kernels;         /* kernel launches the call makes */
    long long workspace_bytes; /* workspace the call needs */
    int split_in_kernel; /* 1 if the 3XTF32 TF32 split happens inside the GEMM kernel */
    int cluster_reduce;  /* 1 if split-K partials are added inside thread-block clusters
                            (no workspace, no reduction kernel) */
    int ctas_per_sm;     /* CTAs of the main kernel one SM holds at once (occupancy
                            calculator; 0 if it could not be asked) */
    int threads_per_cta; /* threads of one CTA of the main kernel */
    int b_in_tmem;       /* 1 if the 3XTF32 kernel holds B's split in tensor memory
                            (GEMM_F32_TILE_128x128_TMEM, _256x256_TMEM or
                            _256x128_TMEM) */
    int reduce_in_kernel; /* 1 if that kernel adds its split-K partials itself, in
                             split order (no reduction kernel): from 16 splits,
                             with one unit per CTA (or CTA pair) */
} gemm_f32_plan_info;

int gemm_f32_plan(int M, int N, int K, int algo, int splits,
                  const float* A, const float* B, const float* C,
                  gemm_f32_plan_info* out);

/*
 * gemm_f32_plan_ex -- the plan gemm_f32_ex would run for the same transa,
 * transb, sizes, leading dimensions, algo and splits (alpha and beta do not
 * change it), without running it.  A, B, C are optional (NULL): like the
 * leading dimensions they only decide which operands need a padded or
 * transposed copy.  Returns GEMM_F32_SUCCESS or GEMM_F32_ERR_INVALID_VALUE.
 */
int gemm_f32_plan_ex(int transa, int transb, int M, int N, int K, const float* A, long long lda,
                     const float* B, long long ldb, const float* C, long long ldc, int algo,
                     int splits, gemm_f32_plan_info* out);

/*
 * gemm_f32_config / gemm_f32_configured / gemm_f32_plan_config -- run (or
 * plan) C = A * B with a forced kernel configuration instead of the
 * library's choice: the tool behind design-space sweeps ("Lecture 12: final
 * project", the sweep program: try every configuration, check it, time it,
 * rank it).  Arguments as for gemm_f32; the config fields:
 *   algo    GEMM_F32_ALGO_FFMA or _3XTF32 (AUTO only with tile = AUTO)
 *   tile    GEMM_F32_TILE_* below; 0 lets the library choose
 *   splits  as for gemm_f32_algo_splitk (0 = choose)
 * The 256 x 256 CTA-pair tiles exist for 3XTF32 only: _PAIR reads TF32
 * hi/lo copies of A and B written by staging kernels, _PAIR_SPLIT reads A
 * and B as stored and splits each tile in shared memory (same products, no
 * staging pass).  _128x128_SPLIT is the single-CTA 128 x 128 tile that
 * likewise reads A and B as stored and splits them in shared memory (no
 * staging launch: for small calls, where that launch is a large part of
 * the call).  _128x128_TMEM reads A and B as stored too; it splits A in
 * shared memory and B into tensor memory, where the MMA takes B^T as its
 * operand, and computes each 128 x 128 tile transposed (no staging pass and
 * no transpose in shared memory).  _256x256_TMEM is its CTA-pair form
 * (256 x 256 tiles, N = 256 MMAs), and _256x128_TMEM its wide single-CTA
 * form (256 rows by 128 columns, N = 256 MMAs, 16-deep stages).  AUTO
 * takes one of these for row-major A and B (after padded copies where a
 * row stride or base is not 16-byte aligned; for transposed operands, after
 * transposed copies, once C has at least 3M elements), the one a fitted time
 * model finds shorter (the wide form only for operands read in place).
 * Split-K partials are added in split order: by the 128 x 128 forms (staged,
 * _SPLIT and _TMEM) inside a thread-block cluster when 2..8 splits give
 * every CTA one unit and the clusters all fit at once (cluster_reduce = 1:
 * no workspace for them, no reduction launch); by the _TMEM forms inside the
 * kernel from 16 splits (reduce_in_kernel = 1); otherwise by a reduction
 * kernel over a workspace.
 * Invalid combinations return GEMM_F32_ERR_INVALID_VALUE.
 */
#define GEMM_F32_TILE_AUTO          0
#define GEMM_F32_TILE_128x128       1
#define GEMM_F32_TILE_128x256       2
#define GEMM_F32_TILE_256x256_PAIR  3
#define GEMM_F32_TILE_256x256_PAIR_SPLIT 4
#define GEMM_F32_TILE_128x128_SPLIT 5
#define GEMM_F32_TILE_128x128_TMEM  6
#define GEMM_F32_TILE_256x256_TMEM  7
#define GEMM_F32_TILE_256x128_TMEM  8
typedef struct gemm_f32_config {
    int algo;
    int tile;
    int splits;
} gemm_f32_config;

int gemm_f32_configured(const float* A, const float* B, float* C, int M, int N, int K,
                        const gemm_f32_config* cfg, cudaStream_t stream);
int gemm_f32_plan_config(int M, int N, int K, const gemm_f32_config* cfg, const float* A,
                         const float* B, const float* C, gemm_f32_plan_info* out);

/*
 * gemm_f32_device_status -- read (and with clear != 0, reset) the fault
 * words that kernels set on the current device when a bounded wait on one of
 * their pipeline barriers runs out: the library's own word and, once
 * gemm_f32_noalloc has run on the device, the word at the head of that entry
 * point's fixed array.  Synchronises the current device.  Allocates nothing
 * and sets nothing up (a device no call has used reports 0).  Returns 0, or
 * GEMM_F32_ERR_DEVICE_TIMEOUT if a kernel reported a timeout since the last
 * clear, GEMM_F32_ERR_UNSUPPORTED_DEVICE, or a positive cudaError_t.
 */
int gemm_f32_device_status(int clear);

/*
 * gemm_f32_selftest_watchdog -- launch on `stream` one kernel that waits on
 * a shared-memory barrier that nothing ever completes, with a wait limit of
 * timeout_ns nanoseconds (1e3 .. 1e10), then synchronise the stream and
 * return gemm_f32_device_status(1).  A working watchdog returns
 * GEMM_F32_ERR_DEVICE_TIMEOUT and leaves the context usable.
 */
int gemm_f32_selftest_watchdog(long long timeout_ns, cudaStream_t stream);

/*
 * gemm_f32_noalloc -- C = A * B on the CUDA-core FFMA kernel (with split-K
 * when it helps) without allocating any memory.  The pages have no
 * counterpart: this entry point exists for callers that cannot let a library
 * allocate while they run -- programs that reserve their whole device memory
 * budget up front and hand it out from their own pool, and latency-critical
 * loops that cannot absorb the device-wide synchronisation of cudaFree.
 * A, B, C, M, N, K and the result are exactly as for gemm_f32; `splits` is
 * as for gemm_f32_algo_splitk (0 = choose, limited to what fits).
 *
 * Scratch (split-K partial sums, and padded copies of A or B when a row
 * stride or base address is not 16-byte aligned) comes from one fixed
 * device array of GEMM_F32_NOALLOC_SCRATCH_BYTES, compiled into the library
 * and held by every GPU that loads it until the process exits.  A problem
 * whose padded copies, or whose explicitly requested split partials
 * (splits x M x roundup(N, 4) floats), do not fit returns
 * GEMM_F32_ERR_INVALID_VALUE and launches nothing.  The first call on each
 * device looks up the array's device address and clears its fault word (a
 * kernel-side watchdog flag at the start of the array), waiting on `stream`
 * for the clear; make that first call before any stream capture begins (made
 * on a capturing stream it returns GEMM_F32_ERR_CAPTURE and enqueues
 * nothing).  A kernel of this entry point whose bounded wait runs out sets
 * that word and returns; the call itself has already returned 0, so, as with
 * gemm_f32, the timeout is seen through gemm_f32_device_status, which reads
 * and clears this word too.  Every call uses the same array, so
 * calls whose work overlaps on the GPU (other streams, other host threads)
 * race on it: serialise them.  No cudaMalloc, cudaFree or allocating
 * library routine is called.
 */
#define GEMM_F32_NOALLOC_SCRATCH_BYTES (16u << 20)
int gemm_f32_noalloc(const float* A, const float* B, float* C, int M, int N, int K,
                     int splits, cudaStream_t stream);

/*
 * gemm_f32_noalloc_selftest_watchdog -- the watchdog self-test of
 * gemm_f32_selftest_watchdog, aimed at gemm_f32_noalloc's fault word instead
 * of the library's: one kernel on `stream` waits on a barrier nothing
 * completes, with a limit of timeout_ns nanoseconds (1e3 .. 1e10), and the
 * stream is synchronised.  Returns GEMM_F32_ERR_DEVICE_TIMEOUT when the wait
 * gave up and set the word (the working outcome), 0 if it did not.  The bit
 * is left set, as after a real timeout, for gemm_f32_device_status to report
 * and clear.  Allocates nothing; the pages have no counterpart.
 */
int gemm_f32_noalloc_selftest_watchdog(long long timeout_ns, cudaStream_t stream);

/* ---- 8-bit activation checkpoints -------------------------------------- */
/*
 * What a training step keeps of a layer between its forward and its backward
 * pass, in 8 bits an element, and the operators of the backward pass that
 * read it in that form: the weight gradient of a linear layer and the
 * derivative of a gated unit.  The pages have no counterpart: these serve the
 * callers that use the product above to train.
 *
 * The form: rows x cols elements, a code byte each, and for each block of 32
 * consecutive columns of a row (the last may be shorter) one exponent byte E,
 * the power-of-two scale of the OCP microscaling formats:
 *   GEMM_F32_Q8_INT8   value = code * 2^(E - 133), code in -127 .. 127
 *   GEMM_F32_Q8_E4M3   value = code * 2^(E - 127), code an 8-bit float with 4
 *                      exponent and 3 mantissa bits, at most 448
 * E is the smallest exponent at which the block's largest magnitude fits
 * (INT8: at most 127 * 2^(E-133); E4M3: at most 448 * 2^(E-127)), but at
 * least 7 (10 for E4M3), so that every nonzero value is a normal float, and
 * for INT8 at most 254.  Codes are rounded to nearest, ties to even.  A block
 * that holds a NaN or an infinity gets E = 255 and codes 0, and all of it
 * restores to NaN.  An E below its least value reads as a scale of zero.
 * Every value is exactly representable in bf16.  (E4M3 rounds finite
 * magnitudes of 248 * 2^120 = 3.296e38 and more to 2^128, which both types
 * restore as an infinity.)
 *
 * Layout: row i's codes are at codes + i * ldcodes, its exponents at scales +
 * i * ldscales (bytes).  Both arrays are in device memory, 16-byte aligned,
 * with row strides that are multiples of 16, ldcodes >= cols and ldscales >=
 * ceil(cols / 32).  Bytes beyond a row's last column or block are neither
 * read for their value nor written.  The caller owns them.
 *
 * For all five entry points: matrices are row-major with leading dimensions
 * in elements, any 4-byte (bf16: 2-byte) alignment and any leading dimension
 * at least the row; an output may not share an element with an input or
 * another output (matrices side by side in one buffer, with equal leading
 * dimensions, are apart; with different ones they count as sharing wherever
 * their address ranges meet), else GEMM_F32_ERR_INVALID_VALUE; a matrix without
 * elements is a successful no-op; asynchronous on `stream`, with the status
 * codes, workspace and graph-capture rules above.  Results are deterministic.
 */
#define GEMM_F32_Q8_INT8   0
#define GEMM_F32_Q8_E4M3   1
#define GEMM_F32_Q8_BLOCK  32
typedef struct gemm_f32_q8 {
    unsigned char* codes;
    unsigned char* scales;
    long long ldcodes;
    long long ldscales;
    int rows;
    int cols;
    int format; /* GEMM_F32_Q8_INT8 or _E4M3 */
} gemm_f32_q8;

/* gemm_f32_q8_store -- write the 8-bit form of X (q->rows x q->cols floats,
 * row stride ldx) into q's arrays. */
int gemm_f32_q8_store(const float* X, long long ldx, const gemm_f32_q8* q, cudaStream_t stream);

/* gemm_f32_q8_restore -- write the values that q stands for to X (row stride
 * ldx elements), as floats or, also exactly, as bf16. */
#define GEMM_F32_Q8_TO_F32   0
#define GEMM_F32_Q8_TO_BF16  1
int gemm_f32_q8_restore(const gemm_f32_q8* q, void* X, long long ldx, int type,
                        cudaStream_t stream);

/*
 * gemm_f32_q8_wgrad -- the weight gradient of a linear layer Y = X W from
 * the 8-bit form x of its input (x->rows tokens, x->cols features):
 *
 *     dW = alpha * x^T * dY + beta * dW
 *
 * dY is x->rows x N (row stride lddy), dW x->cols x N (row stride lddw).
 * x's values enter exactly and products are summed in fp32.  algo:
 * GEMM_F32_ALGO_FFMA, the CUDA-core kernel; GEMM_F32_ALGO_3XBF16 (this entry
 * point's alone), the tensor-core kernel, which splits each float of dY
 * exactly into three bf16 parts, with its tiles (256 x 256 by a CTA pair or
 * 256 x 128 by one CTA) chosen by size or, _PAIR and _SINGLE, forced;
 * GEMM_F32_ALGO_AUTO, all of this chosen by size.  splits:
 * for the tensor-core kernel, over how many ranges the tokens are split, as
 * for gemm_f32_algo_splitk (0: the library chooses).
 * The split of dY is exact down to 2^-110; what a smaller element has below
 * 2^-133 is cut off (the CUDA-core kernel takes all of it).
 * The tensor-core kernel's running sums are truncated, the CUDA-core kernel's
 * rounded to nearest: measured 2-norm errors 2e-7 to 4e-7 (a unit of work of up
 * to 512 tokens) or 7e-7 to 8e-7 (beyond), of which 1.5e-7 to 3e-7 or 6e-7
 * towards zero, against 1e-7 to 4e-7 without a direction.
 * With beta == 0 the old dW is not read; with alpha ==
 * 0 or no rows, x and dY are not read and dW = beta * dW.  A NaN or infinity
 * in dY or a block of x that restores to NaN gives non-finite outputs in the
 * columns or rows of dW it enters.
 */
#define GEMM_F32_ALGO_3XBF16        3
#define GEMM_F32_ALGO_3XBF16_PAIR   4
#define GEMM_F32_ALGO_3XBF16_SINGLE 5
int gemm_f32_q8_wgrad(const gemm_f32_q8* x, const float* dY, long long lddy, int N, float alpha,
                      float beta, float* dW, long long lddw, int algo, int splits,
                      cudaStream_t stream);

/*
 * gemm_f32_q8_gated -- the forward pass of a gated unit, H = act(G) * U
 * elementwise, which also stores G and U in gq and uq (equal rows, cols and
 * format) for the backward pass.  H comes from G and U as given, not from
 * their 8-bit form.  act: GEMM_F32_ACT_SILU (z / (1 + e^-z)) or
 * GEMM_F32_ACT_GELU (z times the normal distribution function of z).
 *
 * gemm_f32_q8_gated_backward -- from those and dH:
 *     dU = dH * act(G^),   dG = dH * U^ * act'(G^)
 * and, with hq not NULL, the 8-bit form of act(G^) * U^, the input of the
 * layer that follows, for its weight gradient: H need not be kept.
 */
#define GEMM_F32_ACT_SILU 0
#define GEMM_F32_ACT_GELU 1
int gemm_f32_q8_gated(int act, const float* G, long long ldg, const float* U, long long ldu,
                      float* H, long long ldh, const gemm_f32_q8* gq, const gemm_f32_q8* uq,
                      cudaStream_t stream);
int gemm_f32_q8_gated_backward(int act, const gemm_f32_q8* gq, const gemm_f32_q8* uq,
                               const float* dH, long long lddh, float* dG, long long lddg,
                               float* dU, long long lddu, const gemm_f32_q8* hq,
                               cudaStream_t stream);

/* ---- 8-bit integer linear layers --------------------------------------- */
/*
 * The layers of a trained model as they are served: weights and activations in
 * 8-bit integers with one fp32 scale a row, a row of activations being a token
 * and a row of weights an output channel.  The pages have no counterpart: these
 * serve the callers that use the product above to train such layers.  A gated
 * block is norm, gated, store, matmul, in this order.
 *
 * The form: rows x cols codes -128 .. 127 and `rows` scales, value =
 * code * scale[row].  Row i's codes are at codes + i * ld (bytes); codes are
 * 16-byte aligned and ld is a multiple of 16, at least cols; bytes beyond a
 * row's last column are neither read for their value nor written.  The scales
 * are contiguous floats.  Both are in device memory and the caller's.
 *
 * What store and norm write for a row z: with a the larger of 2^-100 and z's
 * largest magnitude, code = z * (127 / a) rounded to nearest, ties to even, and
 * scale = a / 127, each operation rounded to fp32.  A row in which z is not
 * finite gets codes 0 and scale NaN, so that its products are NaN.
 *
 * For all four entry points: float and bf16 matrices are row-major with leading
 * dimensions in elements, aligned to their elements, with any leading dimension
 * at least the row; outputs may not share an element with an input or another
 * output, by the rules of the 8-bit checkpoints above; a matrix without rows or
 * columns is a successful no-op; asynchronous on `stream`, with the status
 * codes, workspace and graph-capture rules above.  Results are deterministic.
 */
#define GEMM_F32_TYPE_F32   0
#define GEMM_F32_TYPE_BF16  1
#define GEMM_F32_TYPE_I32   2
typedef struct gemm_f32_i8 {
    signed char* codes;
    float* scales;
    long long ld;
    int rows;
    int cols;
} gemm_f32_i8;

/* gemm_f32_i8_store -- write the rows of X (q->rows x q->cols, floats or bf16
 * by type, row stride ldx) to q. */
int gemm_f32_i8_store(const void* X, int type, long long ldx, const gemm_f32_i8* q,
                      cudaStream_t stream);

/*
 * gemm_f32_i8_norm -- write to q the root-mean-square norm of S = X + R,
 *
 *     S / sqrt(mean(S^2) + eps) * W      (mean over a row, W one value a column)
 *
 * and S itself, the residual stream, to S unless that is NULL.  R NULL: the
 * norm of X, and S must be NULL.  All are floats or all bf16 by type; sums are
 * in fp32, and the norm is that of X + R before it is rounded to the type of S.
 * z above is S * W: the norm's factor is the same for all columns and is
 * multiplied into the scale alone (after a / 127).  eps is finite and at
 * least 1e-30.
 */
#define GEMM_F32_I8_LEAST_EPS 1e-30f
int gemm_f32_i8_norm(const void* X, long long ldx, const void* R, long long ldr, const void* W,
                     float eps, int type, void* S, long long lds, const gemm_f32_i8* q,
                     cudaStream_t stream);

/*
 * gemm_f32_i8_matmul -- Y = a b^T, T x N from T x K tokens a and N x K weights
 * b: the integer sums of code products, exact whatever the sizes, times a's and
 * then b's scale, each product rounded to fp32, as floats or bf16 by type; or
 * with GEMM_F32_TYPE_I32 the sums themselves (the scales then play no part).
 * K is at most GEMM_F32_I8_MAX_COLS, so that no sum overflows 32 bits; K = 0
 * writes zeros.  T and N are at most 2^31 - 1024, and T N at most 10^12.  A
 * token's outputs do not depend on the other tokens of the call, bit for bit.
 * algo: GEMM_F32_ALGO_AUTO, or this entry point's and gated's own: the
 * tensor-core kernel with tiles of CTA pairs (I8_PAIR) or of single CTAs
 * (I8_SINGLE), `splits` being how many ranges of K the latter are split over
 * (at most GEMM_F32_MAX_SPLITS; fewer where K or the workspace's bounds do not
 * allow it; 0: the library chooses), or the kernel for a few tokens (I8_STREAM:
 * a->rows at most GEMM_F32_I8_STREAM_ROWS).
 * Results do not depend on either.
 */
#define GEMM_F32_ALGO_I8_PAIR    6
#define GEMM_F32_ALGO_I8_SINGLE  7
#define GEMM_F32_ALGO_I8_STREAM  8
#define GEMM_F32_I8_STREAM_ROWS  32
#define GEMM_F32_I8_MAX_COLS 131071
int gemm_f32_i8_matmul(const gemm_f32_i8* a, const gemm_f32_i8* b, void* Y, int type,
                       long long ldy, int algo, int splits, cudaStream_t stream);

/*
 * gemm_f32_i8_gated -- both projections of a gated block and their product,
 * H = act(a gate^T) * (a up^T), each as gemm_f32_i8_matmul gives it in fp32;
 * type F32 or BF16.  act: the functions of gemm_f32_q8_gated, but with silu's
 * quotient z / (1 + e^-z) to 2 ulp where that one's is rounded correctly; and
 * where e^-z is beyond 2^126 (z below -87.33) silu is 0, not the up to 1.1e-36
 * that it stands for.
 */
int gemm_f32_i8_gated(int act, const gemm_f32_i8* a, const gemm_f32_i8* gate,
                      const gemm_f32_i8* up, void* H, int type, long long ldh, int algo,
                      int splits, cudaStream_t stream);

/* Release every workspace (synchronises each device that has one). */
int gemm_f32_release(void);

/* Static text for a status code. */
const char* gemm_f32_status_string(int status);

/*
 * gemm_f32_inject_host_fault -- a testing aid that makes one host-side
 * failure happen on purpose, so that a caller's handling of
 * GEMM_F32_ERR_WORKSPACE and GEMM_F32_ERR_DESCRIPTOR can be exercised
 * without any fault on the GPU.  kind = GEMM_F32_INJECT_WORKSPACE: the next
 * workspace (or host-entry buffer) allocation the library attempts reports
 * failure as if cudaMalloc had failed; GEMM_F32_INJECT_DESCRIPTOR: the next
 * TMA descriptor encoding reports failure; GEMM_F32_INJECT_NONE disarms.
 * One-shot and process-wide; off unless called.  The call that meets it
 * returns the status and launches no GEMM kernel (a descriptor failure may
 * follow staging copies already enqueued into the workspace; C is never
 * written); the next call runs normally.  Returns 0, or
 * GEMM_F32_ERR_INVALID_VALUE for an unknown kind.  The pages' counterpart is
 * the error-check macro of "Lecture 5", which exits the process; here the
 * status codes replace the exit.
 */
#define GEMM_F32_INJECT_NONE 0
#define GEMM_F32_INJECT_WORKSPACE 1
#define GEMM_F32_INJECT_DESCRIPTOR 2
int gemm_f32_inject_host_fault(int kind);

/* Library version, major*10000 + minor*100 + patch. */
int gemm_f32_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_F32_H */
