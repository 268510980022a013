/*
 * kron_linear.h -- C ABI of libkronlinear.so, the B200 (sm_100a) implementation of
 * the sum-of-Kronecker-products linear layer
 *
 *     y = x W + bias,   W = sum_{i<r} kron(C_i, B_i),   C_i = S (.) A_i,
 *
 * as defined on the page "kronecker-layer-benchmark" (section "1. Build W, then
 * multiply", KronLinear.weight/forward; rectangular B_i as in section "2. The vec
 * trick").  W is never formed: each row x_n is viewed as X_n (p x m1) and
 * Y_n = sum_i C_i^T X_n B_i (section "2. The vec trick" and "3. The vec trick
 * without the loop"), with both contractions fused on chip.
 *
 * Layouts (all row-major, contiguous, no padding):
 *   x, dX   [N][p*m1]      X_n[a][j]  = x[n][a*m1 + j]
 *   y, dY   [N][q*m2]      Y_n[c][k]  = y[n][c*m2 + k]
 *   S, dS   [p][q]
 *   A, dA   [r][p][q]
 *   B, dB   [r][m1][m2]
 *   bias, dbias [q*m2]
 *
 * Element types by path (kron_dtype_t):
 *   KRON_F32   every tensor is float32; exact FP32 arithmetic on the CUDA cores.
 *   KRON_TF32  every tensor is float32; both contractions run on the tcgen05 tensor
 *              cores with TF32 operands and FP32 accumulation.
 *   KRON_BF16  x, y, dY, dX, S, A, B and bias are bfloat16; dS, dA, dB and dbias are
 *              float32.  tcgen05 tensor cores with BF16 operands, FP32 accumulation.
 *   KRON_TF32 and KRON_BF16 run only where a tensor-core kernel exists for the shape;
 *   a call of any other shape returns KRON_ERR_UNSUPPORTED and launches nothing (it is
 *   never run on another path).  KRON_F32 takes any shape whose FP32 tile fits shared
 *   memory.  kron_linear_workspace_size returns 0 for a shape the requested path does
 *   not take, so it also answers whether a backward is supported.
 *
 * Ownership and synchronisation: every pointer except `stream` is a DEVICE pointer
 * owned by the caller.  The library allocates no memory and never synchronises; all
 * work is enqueued on `stream` (a cudaStream_t passed as void*, NULL = legacy default
 * stream).  No result depends on an earlier call.  The only device memory of its own
 * is compiled in: the error word of kron_linear_device_error and the scratch array of
 * kron_linear_backward_noalloc.
 *
 * Errors: arguments, shapes, alignment and workspace size are checked on the host
 * before anything is launched; a failing check returns its status and launches
 * nothing.  Shapes the requested path has no kernel for return KRON_ERR_UNSUPPORTED;
 * nothing ever falls back to another path or to the CPU.  A failed launch returns KRON_ERR_CUDA;
 * faults during execution surface at the caller's next synchronisation.
 * kron_last_error() gives a one-line description of the last failure on the
 * calling host thread.
 */
#ifndef KRON_LINEAR_H
#define KRON_LINEAR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KRON_LINEAR_ABI_VERSION 2

#if defined(__GNUC__)
#define KRON_API __attribute__((visibility("default")))
#else
#define KRON_API
#endif

typedef enum {
    KRON_F32 = 0,   /* exact FP32 (FFMA)                          */
    KRON_TF32 = 1,  /* FP32 I/O, TF32 tensor cores, FP32 accumulate */
    KRON_BF16 = 2   /* BF16 I/O, BF16 tensor cores, FP32 accumulate */
} kron_dtype_t;

typedef enum {
    KRON_OK = 0,
    KRON_ERR_INVALID_ARG = 1,  /* null pointer, non-positive size, bad dtype or flag   */
    KRON_ERR_UNSUPPORTED = 2,  /* valid shape that this path does not implement          */
    KRON_ERR_ALIGNMENT = 3,    /* a pointer is not 16-byte aligned                       */
    KRON_ERR_WORKSPACE = 4,    /* workspace NULL or smaller than kron_linear_workspace_size */
    KRON_ERR_CUDA = 5,         /* a CUDA runtime call or kernel launch failed            */
    KRON_ERR_TIMEOUT = 6       /* a bounded device-side wait gave up (kron_linear_device_error) */
} kron_status_t;

/* Skip the work of (a, c) blocks where S is zero (the m1 x m2 block of W is zero,
 * page "kronecker-layer-benchmark", introduction).  Only provably-zero products are
 * skipped: dS stays exact at zero entries of S.  Results equal the unflagged call
 * up to rounding. */
#define KRON_FLAG_SKIP_ZERO_BLOCKS 1u

/*
 * Forward: y = x W + bias.
 *   x     [N][p*m1]  input rows
 *   S, A, B          factors as above
 *   bias  [q*m2]     may be NULL (no bias)
 *   y     [N][q*m2]  output, overwritten
 *   N >= 0 rows (N == 0 is a no-op and x, y may then be NULL); p, q, m1, m2, r >= 1.
 * Requirements: x, y, S, A, B, bias 16-byte aligned (KRON_ERR_ALIGNMENT);
 * m1 and m2 multiples of 4 (F32/TF32) or 8 (BF16), else KRON_ERR_UNSUPPORTED.
 */
KRON_API kron_status_t kron_linear_forward(const void *x, const void *S, const void *A, const void *B,
                                  const void *bias, void *y,
                                  int64_t N, int p, int q, int m1, int m2, int r,
                                  kron_dtype_t dtype, unsigned flags, void *stream);

/*
 * Backward: gradients of L = <dY, y> (dY = dL/dy).
 *   dX    [N][p*m1]   = dY W^T                                   (may be NULL: skipped)
 *   dS    [p][q]      = sum_i dC_i (.) A_i
 *   dA    [r][p][q]   = dC_i (.) S,   dC_i = sum_n (X_n B_i) dY_n^T
 *   dB    [r][m1][m2] = sum_n X_n^T C_i dY_n
 *   dbias [q*m2]      = sum_n dY_n                                (may be NULL: skipped)
 * With N == 0, x, dY and dX may be NULL and the factor gradients are set to zero.
 * Gradients OVERWRITE their outputs.  T = X_n B_i is recomputed, nothing is kept
 * from the forward call.  The sums over rows are split into a fixed number of
 * contiguous row ranges whose partials are added in a fixed order, so results are
 * bitwise identical across calls with the same inputs on the same GPU model.
 * `workspace` is device scratch of at least kron_linear_workspace_size(...) bytes,
 * 256-byte aligned, owned by the caller; its contents on entry are ignored.
 * On the tensor-core paths of the tutorial layer's shape (p = q = m1 = m2 = 32, r = 4)
 * the parameter-gradient kernel sums the row ranges itself after a grid-wide barrier:
 * it is a cooperative launch of one CTA per row range (at most 148), all of which must
 * be resident at once.  On a device or partition that cannot hold them (fewer SMs, or
 * SMs taken by other work under MPS) the launch fails and the call returns
 * KRON_ERR_CUDA; the other paths add the ranges with a separate reduction kernel.
 */
KRON_API kron_status_t kron_linear_backward(const void *x, const void *S, const void *A, const void *B,
                                   const void *dY, void *dX, void *dS, void *dA, void *dB,
                                   void *dbias,
                                   int64_t N, int p, int q, int m1, int m2, int r,
                                   kron_dtype_t dtype, unsigned flags,
                                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * Backward with the l1 penalty on S fused into the dS epilogue.
 *
 * The layer is trained with the loss plus l1 * sum_{a,c} |S[a][c]| (page
 * "kronecker-layer-benchmark", introduction: an l1 penalty on S makes S sparse and with it
 * W block-sparse; section "Setup": the step's loss is the cross-entropy plus the model's
 * penalty).  The gradient of that term, l1 * sign(S), is added to dS inside the kernel that
 * writes dS, so the caller launches nothing for it:
 *   dS [p][q] = sum_i dC_i (.) A_i + l1 * sign(S)
 * sign(0) = 0: at S[a][c] = 0 the term is 0, the subgradient that autograd takes for |.|.
 * The sum is formed in double and rounded once to float32.
 *   l1   the penalty's weight, 0 <= l1 <= 1e30 (else KRON_ERR_INVALID_ARG); with l1 == 0
 *        the results are bit for bit those of kron_linear_backward.
 * With N == 0 the factor gradients are zero except dS = l1 * sign(S).
 * Every other argument, output and rule is kron_linear_backward's.  (The penalty's value is
 * not computed: the caller adds l1 * sum|S| to the loss it reports if it wants it.)
 */
KRON_API kron_status_t kron_linear_backward_l1(const void *x, const void *S, const void *A,
                                               const void *B, const void *dY, void *dX,
                                               void *dS, void *dA, void *dB, void *dbias,
                                               int64_t N, int p, int q, int m1, int m2, int r,
                                               kron_dtype_t dtype, unsigned flags, double l1,
                                               void *workspace, size_t workspace_bytes,
                                               void *stream);

/*
 * Backward without a caller-provided workspace.  (An addition of this library: the
 * paper has no counterpart.)
 *
 * Some callers cannot allocate device memory at the moment they run the backward: a
 * real-time loop in which cudaMalloc's device-wide synchronisation is not acceptable,
 * a host whose device memory is entirely owned by another allocator, or plain C code
 * with no allocator of its own.  This entry point takes the same arguments as
 * kron_linear_backward without the workspace and uses instead a fixed scratch array
 * of KRON_NOALLOC_SCRATCH_BYTES compiled into the library; it allocates nothing.
 *   - Every GPU that loads the library holds that array until the process exits.
 *   - Problems whose kron_linear_workspace_size exceeds KRON_NOALLOC_SCRATCH_BYTES are
 *     rejected with KRON_ERR_WORKSPACE before anything is launched.
 *   - All calls share the one array per device: calls that overlap on the GPU (for
 *     example on two streams) race on it and must be serialised by the caller.
 *   - The first call on a device looks up the array's device address (with that device
 *     current); make that first call before any stream capture.  The address belongs to
 *     the current CUDA context: it is looked up again after the context changes (after
 *     cudaDeviceReset, or under a context made current through the driver API), so the
 *     first call under a new context must also come before any capture.
 * Results are the same as kron_linear_backward's.
 */
#define KRON_NOALLOC_SCRATCH_BYTES (8u << 20)
KRON_API kron_status_t kron_linear_backward_noalloc(const void *x, const void *S, const void *A,
                                                    const void *B, const void *dY, void *dX,
                                                    void *dS, void *dA, void *dB, void *dbias,
                                                    int64_t N, int p, int q, int m1, int m2, int r,
                                                    kron_dtype_t dtype, unsigned flags,
                                                    void *stream);

/*
 * Triple Kronecker layer (page "LLM Compression via Kronecker Product Decomposition",
 * section "Triple Kronecker -- AxBxC (Extreme Compression)"), with r terms:
 *
 *     y = x W + bias,   W = sum_i kron(A_i, kron(B_i, C_i)),
 *     A [r][p][q], B [r][m1][m2], C [r][s1][s2], x [N][p*m1*s1], y [N][q*m2*s2],
 *     W[(a*m1 + j)*s1 + u][(c*m2 + k)*s2 + v] = sum_i A_i[a][c] B_i[j][k] C_i[u][v].
 *
 * It runs as the two-factor layer above with S = ones and the block factor
 * kron(B_i, C_i) ((m1*s1) x (m2*s2)), formed in the workspace by each call, so the shapes,
 * paths, dtypes (KRON_BF16: x, y, dY, dX, A, B, C, bias bf16; gradients fp32) and errors
 * are those of kron_linear_forward / kron_linear_backward for (p, q, m1*s1, m2*s2, r); in
 * BF16 the block factor is rounded once to bf16.  The backward returns dA = dC' and chains
 * the block factor's gradient to dB and dC (fixed-order double sums); dX and dbias may be
 * NULL.  `workspace` is kron3_linear_workspace_size(..., backward) bytes (forward: 0, backward:
 * 1), 256-byte aligned, owned by the caller; 0 means the arguments are invalid or the
 * backward has no kernel for the block shape on this path.
 */
KRON_API size_t kron3_linear_workspace_size(int64_t N, int p, int q, int m1, int m2, int s1,
                                            int s2, int r, kron_dtype_t dtype, int backward);
KRON_API kron_status_t kron3_linear_forward(const void *x, const void *A, const void *B,
                                            const void *C, const void *bias, void *y, int64_t N,
                                            int p, int q, int m1, int m2, int s1, int s2, int r,
                                            kron_dtype_t dtype, unsigned flags, void *workspace,
                                            size_t workspace_bytes, void *stream);
KRON_API kron_status_t kron3_linear_backward(const void *x, const void *A, const void *B,
                                             const void *C, const void *dY, void *dX, void *dA,
                                             void *dB, void *dC, void *dbias, int64_t N, int p,
                                             int q, int m1, int m2, int s1, int s2, int r,
                                             kron_dtype_t dtype, unsigned flags, void *workspace,
                                             size_t workspace_bytes, void *stream);

/*
 * Rank-r Kronecker fit of a dense matrix, to initialise the layer's factors from a dense
 * layer (page "LLM Compression via Kronecker Product Decomposition", sections "Van Loan
 * Rearrangement (1993)", "Rank-K" and "Adaptive Normalization"):
 *
 *   Wt[a*q + c][j*m2 + k] = W[a*m1 + j][c*m2 + k]            ((p*q) x (m1*m2))
 *   Wt ~ sum_{i<r} sigma_i u_i v_i^T                           (r leading singular pairs)
 *   A_i = sqrt(sigma_i) reshape(u_i, p, q),  B_i = sqrt(sigma_i) reshape(v_i, m1, m2)
 *   alpha = |W|_F / |sum_i kron(A_i, B_i)|_F; with normalize != 0, A_i and B_i are both
 *   scaled by sqrt(alpha) (the fit then has the Frobenius norm of W).
 *
 * With S = ones, (S, A, B) are factors of this layer: sum_i kron(S (.) A_i, B_i) is the
 * best Kronecker sum of r terms to W in the Frobenius norm (times alpha when normalized).
 * The singular pairs come from randomized subspace iteration (Halko, Martinsson and Tropp,
 * 2011): Q = orth(Wt Omega), then power_iters times Q = orth(Wt orth(Wt^T Q)), and the
 * eigenpairs of (Q^T Wt)(Q^T Wt)^T.  The fit is exact (to rounding) when W has Kronecker
 * rank <= k; otherwise more power iterations and a larger k bring it closer to the exact
 * truncated SVD.  Sums run in double in a fixed order: results are bitwise reproducible.
 *   W       [p*m1][q*m2] float32, device
 *   omega   [k][m1*m2]  float32, device: the random test matrix (e.g. standard normal),
 *           drawn by the caller; 1 <= r <= k <= 64, k <= p*q, k <= m1*m2
 *   power_iters  0..16
 *   A [r][p][q], B [r][m1][m2], sigma [k] (estimated singular values of Wt, largest
 *   first), alpha [1]: float32 outputs, device, overwritten
 *   workspace of kron_vanloan_workspace_size(p, q, m1, m2, k) bytes, 256-byte aligned
 * Every pointer is 16-byte aligned (KRON_ERR_ALIGNMENT).  Bad sizes or pointers return
 * KRON_ERR_INVALID_ARG before anything is launched; all work is enqueued on `stream`.
 */
KRON_API size_t kron_vanloan_workspace_size(int p, int q, int m1, int m2, int k);
KRON_API kron_status_t kron_vanloan_fit(const void *W, int p, int q, int m1, int m2, int r,
                                        const void *omega, int k, int power_iters,
                                        int normalize, void *A, void *B, void *sigma,
                                        void *alpha, void *workspace, size_t workspace_bytes,
                                        void *stream);

/*
 * The gated half of a feed-forward block over two projections of this layer's form:
 *
 *     h = act(x Wg + bg) * (x Wu + bu),   W* = sum_i kron(S* (.) A*_i, B*_i)
 *
 * The projections are stacked, gate first:
 *   S, dS [2][p][q];  A, dA [2][r][p][q];  B, dB [2][r][m1][m2];  bias, dbias [2][q*m2]
 *   x, dX [N][p*m1];  h, dH [N][q*m2]
 * `activation` is a kron_activation_t.  flags must be 0.
 *   KRON_F32   every tensor float32, exact FP32 arithmetic on the CUDA cores; m1 and m2
 *              multiples of 4, and a row's tile has to fit shared memory, else
 *              KRON_ERR_UNSUPPORTED
 *   KRON_BF16  every tensor bfloat16, the gradients too (each rounded once from float32);
 *              tcgen05 tensor cores: both projections, the activation and the product in one
 *              kernel.  Sizes are run-time values; m1 and m2 multiples of 8 up to 256, p and q
 *              at most 1024, and the factors of some slice of the layer have to fit shared
 *              memory, else KRON_ERR_UNSUPPORTED.  With |p| = p rounded up to a multiple of 16 and
 *              |m| = m rounded up to 16, 32 or a multiple of 64, they do for
 *                  ceil(r / 4) (|p| + |m1|) + 2 |m1| <= 646,
 *              and for the backward, which forms dX with the roles swapped, where also
 *                  2 ceil(r / 8) (|q| + |m2|) + 2 |m2| <= 646,
 *              and for some larger ones
 *   KRON_TF32  KRON_ERR_UNSUPPORTED
 * Backward: gradients of <dH, h>; the pre-activations are formed again, nothing is kept from
 * the forward call.  bias may be NULL (none); dX and dbias may be NULL (skipped).  On KRON_BF16
 * T = X B and the pre-activations' gradients are rounded to bfloat16 between the products.
 * With N == 0 the forward is a no-op and the factor gradients are zero.
 * h is not x, dX is not x, and no gradient is the tensor that it belongs to (the inputs are read
 * until the last kernel): KRON_ERR_INVALID_ARG for the same pointer, and no other overlap of
 * inputs and outputs either.  dX may be dH.
 * `workspace`: kron_glu_workspace_size(..., backward) bytes, 256-byte aligned, owned by the
 * caller; two calls that may run at the same time need one each.  The forward needs 0 bytes
 * (workspace may then be NULL), but for some shapes and many rows in KRON_F32.  0 also means
 * arguments that the call refuses, and for the backward with N > 0 only that; whether the forward
 * has a kernel for a shape, a call with N = 0 tells without launching anything.  A backward that is
 * refused does not keep the forward from running.  For the KRON_BF16 backward of more than eight
 * rows it holds x^T dg and x^T du in float32 (8 p m1 q m2 bytes, and as much again for each range
 * that many rows are split into) beside dg and du.  N <= 2^30.
 * Results are bitwise reproducible on one GPU model.  Everything else as for the layer.
 */
typedef enum {
    KRON_ACT_SILU = 0,      /* g sigmoid(g)                                        */
    KRON_ACT_GELU = 1,      /* g (1 + erf(g / sqrt 2)) / 2                         */
    KRON_ACT_GELU_TANH = 2, /* g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2     */
    KRON_ACT_SIGMOID = 3    /* sigmoid(g)                                          */
} kron_activation_t;
KRON_API size_t kron_glu_workspace_size(int64_t N, int p, int q, int m1, int m2, int r,
                                        kron_dtype_t dtype, int backward);
KRON_API kron_status_t kron_glu_forward(const void *x, const void *S, const void *A, const void *B,
                                        const void *bias, void *h, int64_t N, int p, int q,
                                        int m1, int m2, int r, int activation, kron_dtype_t dtype,
                                        unsigned flags, void *workspace, size_t workspace_bytes,
                                        void *stream);
KRON_API kron_status_t kron_glu_backward(const void *x, const void *S, const void *A,
                                         const void *B, const void *bias, const void *dH, void *dX,
                                         void *dS, void *dA, void *dB, void *dbias, int64_t N,
                                         int p, int q, int m1, int m2, int r, int activation,
                                         kron_dtype_t dtype, unsigned flags, void *workspace,
                                         size_t workspace_bytes, void *stream);

/*
 * Distillation loss against a teacher's top logits: what trains a compressed model to answer
 * as the dense one that it came from.  Row n holds the student's logits x [V] and up to K of
 * the teacher's logits t_j with their columns i_j:
 *
 *   p    = softmax_j(t_j / tau) over the row's entries,   q = softmax(x / tau)
 *   loss[n] = w_n ( (1 - lam) tau^2 sum_j p_j (log p_j - log q_{i_j})
 *                   + lam (log sum exp(x) - x_label) )
 *   dlogits[n][v] = w_n dloss_n ( (1 - lam) tau (q_v - sum_{j: i_j = v} p_j)
 *                                 + lam (softmax(x)_v - [v = label]) )
 *
 *   logits  [N] rows of V elements, `ld` elements apart (ld >= V); float32 (KRON_F32) or
 *           bfloat16 (KRON_BF16); KRON_TF32 returns KRON_ERR_UNSUPPORTED
 *   values  [N][K] float32; indices [N][K], index_bytes = 4 (int32) or 8 (int64).  An index
 *           outside [0, V) is no entry, and its value is not looked at; neither has an entry
 *           of value -inf any weight.  A column may be listed more than once: its
 *           probabilities add up.  A row without entries has no teacher term.  1 <= K <= 1024.
 *   labels  [N] int64; a label outside [0, V) (such as -100) is none: the row's second term
 *           is zero.  May be NULL when lam = label_weight is 0.
 *   weights [N] float32, NULL = ones.  A row of weight 0 gives loss 0 and gradient 0 whatever
 *           its logits and dloss hold, and so does one without any term (no entries or lam = 1,
 *           and no label or lam = 0).
 *   loss    [N] float32, not reduced
 *   lse     [N][2] float32: the log-sum-exp of the row at the temperature and at one, which
 *           kron_distill_backward takes (one that the gradient does not need repeats the
 *           other); forward: may be NULL.  The backward forms the sums of a row again
 *           where one is above 1024 in size, whose rounding would be 1e-4 of a probability
 *   dloss   [N] float32, the gradient of `loss`, NULL = ones
 *   dlogits rows ld_out elements apart, of the logits' type; may be the logits themselves
 *           (the same pointer and stride), and does not overlap them otherwise
 *   0.05 <= temperature <= 1e3, 0 <= label_weight <= 1
 * kron_distill_step gives `loss` and the `dlogits` of the sum of `loss` in one call.  It reads
 * every row twice, the second time from L2 where the rows at work at a time (up to 740) fit
 * there.  Sums are formed in float32 in a fixed order: results are bitwise
 * reproducible.  No workspace.  Tensors need the alignment of their elements; rows that are
 * also 16-byte aligned alike in logits and dlogits are stored 16 bytes at a time.  Everything
 * else as for the layer above.
 */
KRON_API kron_status_t kron_distill_forward(const void *logits, int64_t ld, const float *values,
                                            const void *indices, int index_bytes,
                                            const int64_t *labels, const float *weights,
                                            float *loss, float *lse, int64_t N, int64_t V, int K,
                                            double temperature, double label_weight,
                                            kron_dtype_t dtype, void *stream);
KRON_API kron_status_t kron_distill_backward(const void *logits, int64_t ld, const float *values,
                                             const void *indices, int index_bytes,
                                             const int64_t *labels, const float *weights,
                                             const float *lse, const float *dloss, void *dlogits,
                                             int64_t ld_out, int64_t N, int64_t V, int K,
                                             double temperature, double label_weight,
                                             kron_dtype_t dtype, void *stream);
KRON_API kron_status_t kron_distill_step(const void *logits, int64_t ld, const float *values,
                                         const void *indices, int index_bytes,
                                         const int64_t *labels, const float *weights, float *loss,
                                         void *dlogits, int64_t ld_out, int64_t N, int64_t V,
                                         int K, double temperature, double label_weight,
                                         kron_dtype_t dtype, void *stream);

/* Bytes of device workspace kron_linear_backward needs for this problem (0 if the
 * arguments are invalid).  Depends only on the arguments, not on the device. */
KRON_API size_t kron_linear_workspace_size(int64_t N, int p, int q, int m1, int m2, int r,
                                  kron_dtype_t dtype);

/* Static description of a status code. */
KRON_API const char *kron_status_string(kron_status_t status);

/* One-line description of the last failure on this host thread ("" if none). */
KRON_API const char *kron_last_error(void);

/* Device-side error state of the tensor-core kernels.  Every wait inside those
 * kernels is bounded: if one makes no progress for 2 s the kernel raises an error
 * word in device memory and returns instead of hanging.  This call synchronises the
 * current device, reads that word and returns KRON_ERR_TIMEOUT if it is set
 * (KRON_OK otherwise); clear != 0 resets it. */
KRON_API kron_status_t kron_linear_device_error(int clear);

/* KRON_LINEAR_ABI_VERSION of the loaded library. */
KRON_API int kron_linear_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KRON_LINEAR_H */
