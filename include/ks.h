/*
 * ks.h -- C ABI of libks: Kronecker-sparse (KS) matrix multiplication on
 * AMD MI355X (gfx950).
 *
 * The operation. A KS matrix has a support that is a Kronecker product of
 * identity and all-ones blocks (KS abstract page, taxoreview.com
 * "dblp:303/4794", first paragraph, first sentence). libks handles the
 * support I_a (x) 1_{b x c} (x) I_d: W is (a*b*d) x (a*c*d) and holds
 * a*b*c*d nonzeros, stored densely as a 4-D tensor K of shape (a, d, b, c),
 * gamma fastest, with
 *     W[alpha*b*d + beta*d + delta][alpha*c*d + gamma*d + delta]
 *         = K[alpha][delta][beta][gamma].
 * Every entry point computes Y = X * W^T for a batch of rows:
 *     Y[n][alpha][beta][delta] = sum_gamma K[alpha][delta][beta][gamma]
 *                                        * X[n][alpha][gamma][delta],
 * X is batch x (a*c*d) and Y is batch x (a*b*d), both row-major, batch first.
 * The same page's third paragraph factorises matrices into products of
 * butterfly-support factors, and its first sentence ties KS matrices to
 * Butterfly and Monarch matrices, which are such products: ks_chain_matmul
 * applies a list of factors in order. The page's third sentence describes
 * the kernel principle followed here: one fused pass, output-stationary,
 * with no separate permutation of X or Y through global memory.
 *
 * Conventions for every entry point.
 *  - All tensor pointers (W, X, Y, workspace) are DEVICE pointers owned by
 *    the caller. libks never allocates or frees device memory and keeps no
 *    per-call state; it is safe to call from several host threads.
 *  - Calls are asynchronous on `stream` (0 = the null stream). Argument
 *    errors are detected on the host before any HIP call and returned as a
 *    status; nothing is launched then. Launch failures are returned as
 *    KS_ERR_HIP. Faults during execution surface at the caller's next
 *    synchronisation, as for any HIP kernel.
 *  - batch == 0 is a valid no-op.
 *  - Results are deterministic: the same call on the same inputs gives
 *    bit-identical outputs (no atomics, fixed summation order per kernel).
 *  - No exception crosses the ABI.
 */
#ifndef KS_H_
#define KS_H_

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

/* The KS pattern (a, b, c, d): support I_a (x) 1_{b x c} (x) I_d.
 * Each field must be >= 1 (powers of two are not required). n_in = a*c*d,
 * n_out = a*b*d and nnz = a*b*c*d must each be below 2^31. */
typedef struct ks_pattern_t {
    int32_t a, b, c, d;
} ks_pattern_t;

/* Element types. Accumulation is always fp32 and Y is always fp32.
 *  KS_DTYPE_F32   X fp32,  W fp32.
 *  KS_DTYPE_BF16  X bf16,  W bf16 (products of two bf16 values are exact
 *                 in fp32, so only the fp32 accumulation rounds).
 *  KS_DTYPE_BF16W X fp32,  W bf16 (the later factors of a bf16 chain, whose
 *                 inputs are fp32 intermediates).
 * bf16 is the upper 16 bits of an IEEE fp32 word. */
typedef enum ks_dtype_t {
    KS_DTYPE_F32 = 0,
    KS_DTYPE_BF16 = 1,
    KS_DTYPE_BF16W = 2
} ks_dtype_t;

typedef enum ks_status_t {
    KS_OK = 0,
    KS_ERR_NULL = 1,            /* a required pointer is NULL (batch > 0)      */
    KS_ERR_PATTERN = 2,         /* a field < 1, or n_in/n_out/nnz >= 2^31      */
    KS_ERR_BATCH = 3,           /* batch < 0 or batch >= 2^31                  */
    KS_ERR_DTYPE = 4,           /* unknown dtype                               */
    KS_ERR_CHAIN_MISMATCH = 5,  /* n < 1, or n_out(p[k]) != n_in(p[k+1])       */
    KS_ERR_WORKSPACE = 6,       /* workspace NULL or smaller than required     */
    KS_ERR_ALIGN = 7,           /* pointer not aligned to its element size     */
    KS_ERR_OVERLAP = 8,         /* Y (or workspace) overlaps an input          */
    KS_ERR_HIP = 9,             /* a HIP call failed (launch, device query)    */
    KS_ERR_UNSUPPORTED = 10,    /* a forced kernel cannot run this pattern     */
    KS_ERR_INVALID = 11         /* other invalid argument (flags, options)     */
} ks_status_t;

/* Kernel families, for ks_matmul_ex (tests and benchmarks only). */
typedef enum ks_kernel_t {
    KS_KERNEL_AUTO = 0,     /* the planner's choice (what ks_matmul runs)        */
    KS_KERNEL_GENERIC = 1,  /* one thread per output, any pattern                */
    KS_KERNEL_VALU = 2,     /* weights in registers, fp32 FMA (b, c <= 16)       */
    KS_KERNEL_MFMA = 3,     /* matrix cores (b, c >= 16), LDS-staged tiles       */
    KS_KERNEL_MFMA_LDS = 4, /* same kernels as KS_KERNEL_MFMA (kept for ABI)     */
    KS_KERNEL_COLUMN = 5    /* matrix cores, output computed in place in the
                               staged X tile: b = c in {16, 32}, d a multiple
                               of 32 (b = 16) or 16 (b = 32), fp32 X           */
} ks_kernel_t;

/* Who stores Y in the MFMA kernels, for ks_options_t.store_waves. */
typedef enum ks_store_waves_t {
    KS_STORE_AUTO = 0,      /* the planner's choice                              */
    KS_STORE_COMPUTE = 1,   /* the compute waves, after each step's MFMAs        */
    KS_STORE_DEDICATED = 2  /* a storer wave, overlapped with the next step's
                               MFMAs (needs LDS for two Y tiles)                 */
} ks_store_waves_t;

/* Tile candidates of the matrix-core kernel: k = 1..KS_MFMA_TILES selects
   (B-operand register budget, b split) = (32, 1), (64, 1), (128, 1),
   (128, 2), (64, 2), (128, 4), (64, 4) for the k-th entry. */
#define KS_MFMA_TILES 7

typedef struct ks_options_t {
    int32_t kernel;         /* a ks_kernel_t value                               */
    int32_t rows_per_block; /* 0 = planner default; else rows per workgroup step */
    int32_t store_waves;    /* a ks_store_waves_t value; MFMA family only;
                               KS_ERR_UNSUPPORTED if the tile cannot use it      */
    int32_t mfma_tile;      /* 0 = planner choice; 1..KS_MFMA_TILES forces that
                               tile candidate (MFMA family only);
                               KS_ERR_UNSUPPORTED if it does not fit the pattern */
    int32_t mfma_loaders;   /* 0 = planner choice; 1 or 2 waves streaming X into
                               LDS (MFMA family only; 2 needs c >= 64, else
                               KS_ERR_UNSUPPORTED)                               */
    int32_t reserved[3];    /* must be zero                                      */
} ks_options_t;

/* Chain flags. */
#define KS_CHAIN_AUTO 0u      /* fuse consecutive factors where the planner can */
#define KS_CHAIN_NO_FUSE 1u   /* one launch per factor, through the workspace   */

/* Human-readable name of a status; never NULL. */
const char* ks_status_string(ks_status_t status);

/* Library version string, e.g. "libks 0.1.0 gfx950". */
const char* ks_version(void);

/*
 * ks_matmul: Y = X * W^T for one KS factor p.
 *   W      device, K tensor of shape (p.a, p.d, p.b, p.c), contiguous,
 *          element type per dt.
 *   X      device, batch x (a*c*d) row-major, element type per dt.
 *   Y      device, batch x (a*b*d) row-major fp32; fully overwritten.
 *   batch  number of rows, 0 <= batch < 2^31.
 *   dt     KS_DTYPE_F32, KS_DTYPE_BF16 or KS_DTYPE_BF16W.
 *   stream HIP stream for the launch.
 * Pointers must be aligned to their element size (4 bytes fp32, 2 bytes
 * bf16); 16-byte alignment enables wider loads but is not required.
 * Y must not overlap X or W (KS_ERR_OVERLAP).
 */
ks_status_t ks_matmul(ks_pattern_t p, const void* W, const void* X, void* Y,
                      int64_t batch, ks_dtype_t dt, hipStream_t stream);

/*
 * ks_matmul_ex: ks_matmul with options; opt may be NULL (same as ks_matmul).
 * opt->kernel forces a kernel family; KS_ERR_UNSUPPORTED if that family
 * cannot run p with dt. For tests and benchmarks that compare kernels on
 * the same input; results of every family agree within fp32 rounding.
 */
ks_status_t ks_matmul_ex(ks_pattern_t p, const void* W, const void* X, void* Y,
                         int64_t batch, ks_dtype_t dt, hipStream_t stream,
                         const ks_options_t* opt);

/*
 * Gradients of ks_matmul, for a layer's backward pass. The pages give the
 * layer (a KS linear layer usable from PyTorch: KS abstract page,
 * taxoreview.com "dblp:303/4794", first paragraph, last sentence); its
 * derivatives are the chain rule on Y = X * W^T. With dY = dL/dY
 * (batch x a*b*d):
 *   dX = dY * W     dX[n][alpha][gamma][delta]
 *                     = sum_beta K[alpha][delta][beta][gamma] dY[n][alpha][beta][delta]
 *   dK              dK[alpha][delta][beta][gamma]
 *                     = sum_n dY[n][alpha][beta][delta] X[n][alpha][gamma][delta]
 *
 * ks_matmul_dx_workspace_size: bytes of workspace ks_matmul_dx needs (W's
 *   blocks transposed: nnz elements of W's type, rounded up to 256), to
 *   *bytes. KS_ERR_NULL if bytes is NULL; pattern and dtype statuses as for
 *   ks_matmul.
 * ks_matmul_dx: dX = dY * W.
 *   W      device K tensor (a, d, b, c) as in ks_matmul.
 *   dY     device, batch x (a*b*d): fp32 for KS_DTYPE_F32 and KS_DTYPE_BF16W,
 *          bf16 for KS_DTYPE_BF16; W is bf16 for KS_DTYPE_BF16 and BF16W.
 *   dX     device fp32, batch x (a*c*d); fully overwritten.
 *   ws     device workspace, >= ks_matmul_dx_workspace_size bytes, 16-byte
 *          aligned (KS_ERR_WORKSPACE if NULL or smaller, KS_ERR_ALIGN).
 *   Runs as the forward product of pattern (a, c, b, d) with every block of
 *   W transposed (two launches on `stream`). dX must not overlap dY, W or
 *   ws, nor ws dY or W (KS_ERR_OVERLAP). batch = 0: nothing is launched.
 */
ks_status_t ks_matmul_dx_workspace_size(ks_pattern_t p, ks_dtype_t dt, size_t* bytes);
ks_status_t ks_matmul_dx(ks_pattern_t p, const void* W, const void* dY, void* dX, int64_t batch,
                         ks_dtype_t dt, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * ks_matmul_dw_workspace_size: bytes of workspace ks_matmul_dw needs for
 *   this batch (0 if none; partial sums over ranges of rows), to *bytes.
 * ks_matmul_dw: dK (the gradient with respect to the K tensor).
 *   dY     device fp32, batch x (a*b*d).
 *   X      device, batch x (a*c*d): fp32 for KS_DTYPE_F32 and KS_DTYPE_BF16W,
 *          bf16 for KS_DTYPE_BF16 (the forward input).
 *   dW     device fp32, shape (a, d, b, c); fully overwritten (zeros when
 *          batch = 0).
 *   ws     device workspace of the queried size (may be NULL when 0),
 *          16-byte aligned.
 *   Partial sums over row ranges are added in a fixed order, so repeated
 *   calls give identical bits. dW must not overlap dY, X or ws, nor ws dY
 *   or X (KS_ERR_OVERLAP).
 */
ks_status_t ks_matmul_dw_workspace_size(ks_pattern_t p, int64_t batch, ks_dtype_t dt, size_t* bytes);
ks_status_t ks_matmul_dw(ks_pattern_t p, const void* dY, const void* X, void* dW, int64_t batch,
                         ks_dtype_t dt, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * ks_matmul_dw_noalloc: ks_matmul_dw for callers that cannot allocate device
 * memory -- code under HIP graph capture, tight training loops, harnesses
 * that forbid hipMalloc. It allocates nothing and takes no workspace: the
 * partial sums go to a scratch array of KS_DW_SCRATCH_BYTES that libks
 * keeps on every GPU it runs on until the process ends. Same arguments,
 * results (bit for bit: the same kernels and summation order) and statuses
 * as ks_matmul_dw without ws / ws_bytes; KS_ERR_WORKSPACE if the call would
 * need more scratch than KS_DW_SCRATCH_BYTES (the planner keeps every dK
 * call's partial sums within it, so this does not happen for valid
 * arguments). All calls on one GPU share its scratch: calls that overlap in
 * time on one GPU (several streams or host threads) race and give wrong
 * results; calls in sequence on one stream are safe.
 */
#define KS_DW_SCRATCH_BYTES (64u << 20)
ks_status_t ks_matmul_dw_noalloc(ks_pattern_t p, const void* dY, const void* X, void* dW, int64_t batch,
                                 ks_dtype_t dt, hipStream_t stream);

/*
 * ks_chain_workspace_size: bytes of device workspace ks_chain_matmul needs
 * for these arguments (0 if none), written to *bytes.
 *   p, n   the factors in application order (p[0] is applied to X first).
 *   dt     KS_DTYPE_F32, KS_DTYPE_BF16 or KS_DTYPE_BF16W (chain dtype: the
 *          types of X and of every W; intermediates are always fp32).
 *   flags  KS_CHAIN_AUTO or KS_CHAIN_NO_FUSE.
 * Returns the same validation statuses as ks_chain_matmul for p, n, batch,
 * dt and flags; KS_ERR_NULL if bytes is NULL.
 */
ks_status_t ks_chain_workspace_size(const ks_pattern_t* p, int n, int64_t batch,
                                    ks_dtype_t dt, unsigned flags, size_t* bytes);

/*
 * ks_chain_matmul: Y = X * (W_{n-1} ... W_1 W_0)^T, factor 0 applied first.
 *   p      host array of n patterns; n_out(p[k]) must equal n_in(p[k+1]).
 *   W      host array of n device pointers; W[k] holds factor k's K tensor
 *          (p[k].a, p[k].d, p[k].b, p[k].c).
 *   X      device, batch x n_in(p[0]); Y device fp32, batch x n_out(p[n-1]).
 *   dt     KS_DTYPE_F32: everything fp32. KS_DTYPE_BF16: X and every W are
 *          bf16; intermediates and Y are fp32, so factors after the first
 *          read fp32 inputs with bf16 weights. KS_DTYPE_BF16W: X fp32 and
 *          every W bf16 (the tail of a bf16 chain run on its own).
 *   ws     device workspace of ws_bytes >= ks_chain_workspace_size(...);
 *          may be NULL when that size is 0. 16-byte aligned. Must not
 *          overlap X, Y or any W.
 *   flags  KS_CHAIN_AUTO: consecutive factors whose joint tile fits on chip
 *          run as one fused launch with the intermediates kept in LDS.
 *          Scanning the chain from factor 0, at each factor the planner
 *          takes the first that applies of: the pair (1, b0, 16, 64) ->
 *          (b0, 8, 8, 8) with b0 % 8 == 0 (a group of beta0 needs whole
 *          rows of X and yields a slab of Y's row); the pair (a, 16, 16, 16)
 *          -> (16a, 16, 16, 1) (the second factor works inside the first
 *          one's per-alpha output slabs; the last two factors of the 16-ary
 *          butterfly); the longest run of at least two factors with blocks
 *          of b * c <= 16, at most 64 KB of weights each and rows of at most
 *          4096 elements, applied to whole rows held in LDS (radix-2 and
 *          radix-4 butterflies, Walsh-Hadamard products); else the factor
 *          alone. KS_CHAIN_NO_FUSE: one launch per factor. Results of the
 *          two modes agree to rounding.
 * All launches go to `stream` in order; there is no host synchronisation.
 */
ks_status_t ks_chain_matmul(const ks_pattern_t* p, int n, const void* const* W,
                            const void* X, void* Y, int64_t batch, ks_dtype_t dt,
                            void* ws, size_t ws_bytes, unsigned flags,
                            hipStream_t stream);

/*
 * ks_chain_plan: the launch groups ks_chain_matmul uses for these arguments.
 * Writes the number of groups to *groups and, for each group in order, the
 * number of consecutive factors it runs (1, or more for a fused group) to
 * group_len[0 .. min(*groups, cap) - 1]. Pure host code; no HIP call. Same
 * validation statuses as ks_chain_workspace_size; KS_ERR_NULL if groups is
 * NULL (group_len may be NULL when cap is 0).
 */
ks_status_t ks_chain_plan(const ks_pattern_t* p, int n, int64_t batch, ks_dtype_t dt,
                          unsigned flags, int* group_len, int cap, int* groups);

/*
 * ks_plan_describe: write a one-line description of the kernel and tile the
 * planner picks for (p, batch, dt) into buf (NUL-terminated, truncated to
 * len). Pure host code; no HIP call. For tests and benchmark labels.
 */
ks_status_t ks_plan_describe(ks_pattern_t p, int64_t batch, ks_dtype_t dt,
                             char* buf, size_t len);

/*
 * ks_pair_closure: the closure rule for running factor f and then factor g
 * in one pass, which the chain planner applies (KS abstract page, first
 * paragraph, first sentence: Butterfly and Monarch matrices are chains of
 * such factors). f's output groups (fixed alpha, delta of f; all beta) and
 * g's input groups (fixed alpha, delta of g; all gamma) link the
 * intermediate's n_out(f) values into closed components: a component's
 * outputs depend only on its own inputs, f blocks and g blocks. Reports the
 * component count, the largest component's sizes and the tile of components
 * whose X reads come in runs of 16 bytes (4 fp32 values). A pair can run
 * fused only if such a tile's intermediates fit in LDS and its weights near
 * the compute units; the planner also needs a kernel family for the shape.
 * Pure host code, no HIP call. KS_ERR_NULL (out), KS_ERR_PATTERN,
 * KS_ERR_CHAIN_MISMATCH (n_out(f) != n_in(g)), KS_ERR_UNSUPPORTED (an
 * intermediate of more than 2^22 values is not analysed).
 */
typedef struct ks_closure_t {
    int64_t components;       /* closed components of the intermediate */
    int64_t mid;              /* intermediate values of the largest component */
    int64_t inputs;           /* values of X it reads */
    int64_t outputs;          /* values of Y it writes */
    int64_t weights;          /* weights it needs: its blocks of f and of g */
    int64_t in_run;           /* shortest run of consecutive X indices it reads */
    int64_t out_run;          /* shortest run of consecutive Y indices it writes */
    int64_t tile_components;  /* components per tile with 16-byte X runs */
    int64_t tile_weights;     /* weights of such a tile */
    int32_t uniform;          /* 1: all components have the same size */
    int32_t reserved;         /* 0 */
} ks_closure_t;

ks_status_t ks_pair_closure(ks_pattern_t f, ks_pattern_t g, ks_closure_t* out);

/*
 * ks_chain_describe: one description per launch group of the chain
 * ks_chain_matmul would run for these arguments, "[first..last] kernel",
 * separated by "; ", into buf (NUL-terminated, truncated to len). Same
 * validation as ks_chain_plan; pure host code, no HIP call. Describes the
 * path for 16-byte-aligned X and Y (a group that needs them runs another
 * kernel otherwise). For tests and benchmark labels.
 */
ks_status_t ks_chain_describe(const ks_pattern_t* p, int n, int64_t batch, ks_dtype_t dt,
                              unsigned flags, char* buf, size_t len);

/*
 * Operators around the product, for serving and fine-tuning a layer of KS
 * factors: low-rank adapters beside a frozen projection, a preference loss on
 * token logits, and the optimizer step. The conventions above hold for all of
 * them: device pointers of the caller, asynchronous on `stream`, argument
 * errors found on the host before any HIP call, no allocation, no atomics and
 * a fixed summation order.
 */

/* Element types of single tensors (the types that ks_dtype_t combines). */
typedef enum ks_elem_t {
    KS_ELEM_F32 = 0,
    KS_ELEM_BF16 = 1
} ks_elem_t;

/*
 * Low-rank adapters of many requests. Adapter g of `count` has
 *   A[g]      rank x n_in,   row-major, the weights' type of the ks_dtype_t
 *   B[g]      n_out x rank,  row-major, the same type
 *   scale[g]  fp32
 * with the adapters one after another. Row n of a batch belongs to adapter
 * g = ids[n]; an id outside [0, count) means none, so such a row gets the
 * shared projection alone. 1 <= rank <= KS_ADAPTER_MAX_RANK and
 * 1 <= count <= KS_ADAPTER_MAX_COUNT; batch * rank and each tensor's element
 * count have to stay below 2^31, else KS_ERR_INVALID.
 */
#define KS_ADAPTER_MAX_RANK 256
#define KS_ADAPTER_MAX_COUNT 65535

typedef struct ks_adapters_t {
    const void* A;        /* device */
    const void* B;        /* device */
    const float* scale;   /* device */
    int64_t n_in, n_out;
    int32_t rank, count;
} ks_adapters_t;

/*
 * ks_adapter_matmul: Y += H B^T with H = scale X A^T, each row with its own
 * adapter:
 *   H[n][r] = scale[g] sum_k X[n][k] A[g][r][k],  Y[n][o] += sum_r H[n][r] B[g][o][r]
 *   ids    device int32, batch values.
 *   X      device, batch x n_in, X's type of dt (as for ks_matmul).
 *   Y      device fp32, batch x n_out; added to.
 *   H      device fp32, batch x rank: fully overwritten, zeros for rows
 *          without an adapter. ks_adapter_backward reads it.
 *   ws     device workspace of ks_adapter_workspace_size bytes, 16-byte
 *          aligned (may be NULL when that is 0).
 * The intermediate H is fp32 in every case. Pointers need the alignment of
 * their element; 16 bytes select wider loads. Y and H must not overlap any
 * input or each other (KS_ERR_OVERLAP).
 */
ks_status_t ks_adapter_workspace_size(const ks_adapters_t* ad, int64_t batch, size_t* bytes);
ks_status_t ks_adapter_matmul(const ks_adapters_t* ad, const int32_t* ids, const void* X, float* Y, float* H,
                              int64_t batch, ks_dtype_t dt, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * ks_adapter_backward: gradients of ks_adapter_matmul. With
 * E[n][r] = scale[g] sum_o dY[n][o] B[g][o][r]:
 *   dX[n][k]    += sum_r E[n][r] A[g][r][k]      (NULL: not computed)
 *   dA[g][r][k]  = sum_{n of g} E[n][r] X[n][k]  fp32, count x rank x n_in
 *   dB[g][o][r]  = sum_{n of g} dY[n][o] H[n][r] fp32, count x n_out x rank
 *   dY     device fp32, batch x n_out.   X, H: as ks_adapter_matmul had and wrote them.
 *   dX     device fp32, batch x n_in; added to (the projection's own dX).
 *   dA, dB fully overwritten, zeros for adapters without rows; both NULL: not
 *          computed (then X and H may be NULL).
 *   ws     device workspace of ks_adapter_backward_workspace_size bytes, 16-byte
 *          aligned (may be NULL when that is 0).
 * Partial sums over ranges of an adapter's rows are added in a fixed order.
 * batch = 0 writes the zeros of dA and dB.
 * The size query and the call give KS_ERR_UNSUPPORTED where a grid could not hold
 * the work, e.g. 65535 adapters of more than 16320 values and over 64 rows.
 */
ks_status_t ks_adapter_backward_workspace_size(const ks_adapters_t* ad, int64_t batch, size_t* bytes);
ks_status_t ks_adapter_backward(const ks_adapters_t* ad, const int32_t* ids, const float* dY, const void* X,
                                const float* H, float* dX, float* dA, float* dB, int64_t batch, ks_dtype_t dt,
                                void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * ks_chain_adapter_matmul: the chain of ks_chain_matmul (KS_CHAIN_AUTO) and
 * the adapters beside it, Y = X (W_{n-1} ... W_0)^T + H B^T. H may be NULL (not
 * kept). Above 1024 rows, a chain that ends in a fused pair of a GPT-2-medium
 * MLP's kind, (1, b, 16, 64) then (b, 8, 8, 8) with b a multiple of 32, adds
 * bf16 adapters of a rank that is a multiple of 4 and at most 32 in that launch
 * to every four rows, counted from the first, that share one or change it once;
 * the sums are then taken in another order, so a row without an adapter has the
 * chain's value up to rounding, and an infinite value of B may give NaN (H enters
 * as three parts, and a part may be 0). Y is fully overwritten; ad->n_in and ad->n_out
 * have to be the chain's (KS_ERR_CHAIN_MISMATCH). Workspace as for
 * ks_chain_matmul, of the size that ks_chain_adapter_workspace_size gives.
 */
ks_status_t ks_chain_adapter_workspace_size(const ks_pattern_t* p, int n, const ks_adapters_t* ad, int64_t batch,
                                            ks_dtype_t dt, size_t* bytes);
ks_status_t ks_chain_adapter_matmul(const ks_pattern_t* p, int n, const void* const* W, const ks_adapters_t* ad,
                                    const int32_t* ids, const void* X, float* Y, float* H, int64_t batch,
                                    ks_dtype_t dt, void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * ks_chain_adapter_backward: dX of the chain (dY W_{n-1} ... W_0, W frozen)
 * plus the adapters', and dA and dB (both NULL: not computed). The chain's part
 * is the chain of the factors in reverse with every block transposed, planned as
 * ks_chain_matmul plans it.
 *   Wt     NULL: W's blocks are transposed in the workspace by each call. Else
 *          device, what ks_chain_transpose wrote for the same p, n and weights
 *          (ks_chain_transpose_size bytes, 16-byte aligned): a layer whose W does
 *          not change makes it once; W may then be NULL. Where both are given
 *          either is read: the pair (1, b, 16, 64), (b, 8, 8, 8) with bf16 weights,
 *          b up to 64 and a multiple of 16 runs as one launch on W itself (W and
 *          dY 16-byte aligned).
 *   ws     of ks_chain_adapter_backward_workspace_size bytes, which has to be
 *          told whether Wt will be given (may be NULL when that is 0).
 */
ks_status_t ks_chain_transpose_size(const ks_pattern_t* p, int n, ks_dtype_t dt, size_t* bytes);
ks_status_t ks_chain_transpose(const ks_pattern_t* p, int n, const void* const* W, void* Wt, ks_dtype_t dt,
                               hipStream_t stream);
ks_status_t ks_chain_adapter_backward_workspace_size(const ks_pattern_t* p, int n, const ks_adapters_t* ad,
                                                     int64_t batch, ks_dtype_t dt, int have_transposed,
                                                     size_t* bytes);
ks_status_t ks_chain_adapter_backward(const ks_pattern_t* p, int n, const void* const* W, const void* Wt,
                                      const ks_adapters_t* ad, const int32_t* ids, const float* dY, const void* X,
                                      const float* H, float* dX, float* dA, float* dB, int64_t batch, ks_dtype_t dt,
                                      void* ws, size_t ws_bytes, hipStream_t stream);

/*
 * Token logits. x[s][t][v] of `sequences` x `tokens` x `vocab` values lies at
 * data[s * seq_stride + t * row_stride + v] (strides in elements, row_stride
 * >= vocab, seq_stride >= (tokens - 1) * row_stride + vocab), so a batch with
 * its last position cut off needs no copy. labels[s * label_stride + t] is the
 * token that position t should give; a negative label masks the position: its
 * logits are not read (they may hold anything), its log probability is 0 and
 * its gradient is 0. A label >= vocab gives NaN.
 */
typedef struct ks_logits_t {
    const void* data;       /* device */
    const int64_t* labels;  /* device */
    int64_t seq_stride, row_stride, label_stride;
    int64_t sequences, tokens, vocab;
    int32_t elem;           /* a ks_elem_t value */
    int32_t reserved;       /* must be zero */
} ks_logits_t;

/*
 * ks_sequence_logp: tokens[s][t] = x[s][t][label] - log sum_v exp x[s][t][v]
 * (0 where masked) and total[s] = sum_t tokens[s][t]; both device fp32,
 * contiguous.
 *   stats  device fp32, sequences x tokens x 2, or NULL: each row's maximum and
 *          its sum of exp(x - maximum), which ks_preference_backward reads.
 */
ks_status_t ks_sequence_logp(const ks_logits_t* x, float* tokens, float* total, float* stats, hipStream_t stream);

/*
 * ks_preference_loss: the paired preference loss of a policy against a
 * reference. Sequences 0 .. P-1 are the chosen answers, P .. 2P-1 the rejected
 * ones (sequences must be even: KS_ERR_INVALID).
 *   rewards[s] = beta sum_t (tokens[s][t] - ref[s][t]) over unmasked t
 *   z_i = rewards[i] - rewards[P + i]
 *   loss = 1/P sum_i (1 - smoothing) log(1 + exp(-z_i)) + smoothing log(1 + exp(z_i))
 *   (a term of weight 0 is 0, whatever its logarithm)
 *   ref     device fp32, ref[s * ref_stride + t]: the reference's tokens of
 *           ks_sequence_logp; of no effect where masked.
 *   loss    device fp32, one value (0 if there is no pair).
 *   rewards device fp32, 2P.   tokens device fp32, 2P x T.
 *   grad    device fp32, 2P: d loss / d total[s], for ks_preference_backward.
 *   stats   device fp32, 2P x T x 2: as ks_sequence_logp writes them.
 *   dlogits NULL: the loss alone. Else the gradient of the loss, of x's element
 *           type, at dlogits[s * d_seq_stride + t * d_row_stride + v]; it may
 *           be x's own memory with x's strides.
 * beta > 0 and 0 <= smoothing <= 1, else KS_ERR_INVALID.
 *
 * ks_preference_backward: that gradient from stats and grad of an earlier
 * call, times upstream[0] (device fp32; NULL means 1).
 */
ks_status_t ks_preference_loss(const ks_logits_t* x, const float* ref, int64_t ref_stride, float beta, float smoothing,
                               float* loss, float* rewards, float* tokens, float* grad, float* stats, void* dlogits,
                               int64_t d_seq_stride, int64_t d_row_stride, hipStream_t stream);
ks_status_t ks_preference_backward(const ks_logits_t* x, const float* stats, const float* grad, const float* upstream,
                                   void* dlogits, int64_t d_seq_stride, int64_t d_row_stride, hipStream_t stream);

/*
 * One optimizer step over many tensors. For each element
 *   m = beta1 m + (1 - beta1) g,   v = beta2 v + (1 - beta2) g^2
 *   p = (1 - lr weight_decay) p - lr / (1 - beta1^step) m / (sqrt(v / (1 - beta2^step)) + eps)
 * in fp32, p rounded to the nearest value of its type at the end.
 * state_bits 32: m and v are fp32. state_bits 8: one byte each, and
 * scales[2 j], scales[2 j + 1] hold the scales of m and of v of the values
 * 256 j .. 256 j + 255 of the tensor:
 *   m = scale k |k| / 127^2  (k signed),   v = scale k^4 / 255^4  (k unsigned)
 * A value between two codes takes the upper one with the probability that
 * keeps its mean, so that the slow average v still moves by less than a code a
 * step; v > 0 never becomes code 0. The random number of value i of a tensor
 * is a hash of options->seed and 256 * (blocks of the tensors before it) + i,
 * so a step is a function of its arguments. A block with a value that is not
 * finite gets a scale that is not finite.
 * The tensors' memory must not overlap between tensors; within one tensor that
 * is checked (KS_ERR_OVERLAP). n = 0 and tensors with n = 0 are no-ops.
 */
typedef struct ks_adamw_tensor_t {
    void* p;          /* device */
    const void* g;    /* device */
    void* m;          /* device: fp32, or int8  */
    void* v;          /* device: fp32, or uint8 */
    float* scales;    /* device: 2 ceil(n / 256) values; unused for 32 bits */
    int64_t n;        /* elements, below 2^31 */
    int32_t p_elem, g_elem;  /* ks_elem_t values */
} ks_adamw_tensor_t;

typedef struct ks_adamw_options_t {
    double lr, beta1, beta2, eps, weight_decay;
    double max_norm;      /* > 0: gradients are scaled by min(1, max_norm / (norm + 1e-6)) */
    int64_t step;         /* >= 1 */
    uint32_t seed;
    int32_t state_bits;   /* 8 or 32 */
} ks_adamw_options_t;

/*
 * ks_grad_norm: norm[0] = sqrt(sum of g^2 over all tensors), device fp32.
 * Only g, g_elem and n of the tensors are read. ws of
 * ks_grad_norm_workspace_size bytes, 16-byte aligned.
 * ks_adamw_step: the step; norm (device fp32) is read if max_norm > 0. If that
 * norm is not finite the step changes nothing.
 * ks_adamw_state_values: m_out[i] and v_out[i] (host arrays of device fp32
 * pointers) get the values that tensor i's 8-bit states stand for.
 */
ks_status_t ks_grad_norm_workspace_size(const ks_adamw_tensor_t* t, int n, size_t* bytes);
ks_status_t ks_grad_norm(const ks_adamw_tensor_t* t, int n, float* norm, void* ws, size_t ws_bytes,
                         hipStream_t stream);
ks_status_t ks_adamw_step(const ks_adamw_tensor_t* t, int n, const ks_adamw_options_t* options, const float* norm,
                          hipStream_t stream);
ks_status_t ks_adamw_state_values(const ks_adamw_tensor_t* t, int n, float* const* m_out, float* const* v_out,
                                  hipStream_t stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* KS_H_ */
