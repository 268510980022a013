// glu.h -- declarations shared by the translation units of the gated Kronecker feed-forward
// half (glu.cu, glu_tc.cu, glu_wgrad.cu): h = act(x Wg + bg) * (x Wu + bu).
#pragma once

#include "../../include/kron_linear.h"
#include "internal.h"
#include "packed.cuh"

namespace kron {
namespace glu {

// What one run of the two-stage tensor-core kernel computes.
enum Mode {
    kForward,  // h from x
    kPre,      // dg = dH u act'(g) and du = dH act(g), both pre-activations formed again
    kInput     // dX = dg Wg^T + du Wu^T
};

// The kernel's tiles for one shape and mode.  In its own terms the kernel contracts P groups
// of M1 values into Q groups of M2 values (kInput: the layer's q, m2, p, m1).
struct Plan {
    int P, M1, Q, M2, r;
    int nsrc, ranks;          // sources, and ranks that contract each of them
    int MP, NT, RB;           // k columns per slice, rows per tile, ranks per block: NT = RB
    int rbl;                  // ranks of the fullest block
    int nac, AC;              // chunks of the a index, and their width
    int nblk, nblk_src;       // rank blocks in all and per source
    int sw, kch, kb;          // x rows: swizzle width, chunks of it per row, bytes per row
    int nqs, qc, qcp, nks;    // c slices, columns per slice (and padded to 16), k slices
    int ybufs, stages, tbufs, dbufs;   // buffers of Y, x, T and D1
    int g1;                            // groups of epilogue-1 warps at work
    int exact;                         // no padding anywhere
    int tm_y;                          // first TMEM column of Y
    int off_c, off_t, off_x, smem;     // shared memory: B^T at 0, C', T, x ring
    int t_bytes, x_bytes, c_chunk;
    int ntiles, groups;       // row tiles, and CTAs per slice
};

// ---- exact FP32 (glu_f32.cu, simt_f32.cu) ----
// Rows from which on the layer's kernels for its compiled shape (p = q = m1 = m2 = 32, r = 4) are
// the faster ones.
constexpr int64_t kCompiledRows = 15 * kRowParts;
// Whether both projections, the activation and the product of this shape run as one kernel.
bool f32_pre_supported(const Shape &s);
// h (grad = false), or dg and du from dH (grad = true); factors stacked gate, up.
cudaError_t f32_pre(const void *x, const void *S, const void *A, const void *B, const void *bias,
                    const void *dH, void *out0, void *out1, const Shape &s, int activation,
                    bool grad, cudaStream_t st);
// simt_backward of both projections: gradients G0, G1 into dX0, dX1 (may be null) and the
// partials of gate and up, parts x partial_stride floats each, into ws.
cudaError_t simt_backward_pair(const void *x, const void *S, const void *A, const void *B,
                               const void *G0, const void *G1, void *dX0, void *dX1, float *ws,
                               int parts, const Shape &s, cudaStream_t st);
// The same by a kernel of its own where its tiles fit; the partials of `parts` <= max_parts ranges.
cudaError_t f32_backward_pair(const void *x, const void *S, const void *A, const void *B,
                              const void *G0, const void *G1, void *dX0, void *dX1, float *ws,
                              int max_parts, int *parts, const Shape &s, cudaStream_t st);
// reduce_partials of both projections; gradients stacked as the factors are (reduce.cu).
cudaError_t reduce_partials_pair(const float *ws, int parts, const void *S, const void *A,
                                 float *dS, float *dA, float *dB, float *dbias, const Shape &s,
                                 cudaStream_t st);

bool tc_plan(Plan *pl, const Shape &s, Mode mode, int sms);

struct TcArgs {
    const void *src0, *src1;      // x, or dg and du
    const void *S, *A, *B, *bias; // stacked gate and up
    const void *dH;
    void *out0, *out1;            // h or dX; dg and du
    int64_t N;
    int activation;
};
cudaError_t tc_run(const Plan &pl, const TcArgs &a, Mode mode, cudaStream_t st);

// Dense weight gradients of the two projections, x^T [dg | du], in split row ranges, then
// the factors' gradients from them.
struct WgradPlan {
    int direct;               // few rows: without dW
    int splits, tm;           // row ranges; rows of dW per tile
    int64_t rows_per_split;
    size_t part_floats;       // one split: [2][din][dout] and the column sums [2][dout]
    size_t ws_bytes;
};
WgradPlan wgrad_plan(const Shape &s, int sms);
cudaError_t wgrad_run(const WgradPlan &pl, const void *x, const void *dg, const void *du,
                      const void *S, const void *A, const void *B, void *dS, void *dA, void *dB,
                      void *dbias, void *ws, const Shape &s, cudaStream_t st);

// act(g) and act'(g) with the accurate functions (exact-FP32 path).
__device__ __forceinline__ float act_f32(int act, float g, float *d) {
    if (act == KRON_ACT_GELU) {
        const float c = 0.5f * erfcf(-g * 0.70710678118654752f);
        const float e = expf(-0.5f * g * g);
        *d = c + (e == 0.f ? 0.f : g * e * 0.39894228040143268f);
        return g * c;
    }
    if (act == KRON_ACT_GELU_TANH) {
        const float g2 = g * g;
        const float v = 1.5957691216057308f * g * (1.f + 0.044715f * g2);
        const float s = 1.f / (1.f + expf(-v)), w = s * (1.f / (1.f + expf(v)));
        *d = s + (w == 0.f ? 0.f : g * w * 1.5957691216057308f * (1.f + 0.134145f * g2));
        return g * s;
    }
    const float s = 1.f / (1.f + expf(-g)), c = 1.f / (1.f + expf(g));   // c = 1 - s
    if (act == KRON_ACT_SIGMOID) {
        *d = s * c;
        return s;
    }
    const float f = g * s;
    *d = s + f * c;
    return f;
}

// Activation, and with GRAD its derivative, of two values, from hardware exponentials and
// reciprocals: about 2^-21 of the value (gelu 2^-17) and, of the terms that a derivative is the sum
// of, of each, far below the bfloat16 rounding of what is stored.  In the tails an argument of size
// v is rounded, 2^-23 v of an exponential, and one that overflows gives 0.
__device__ __forceinline__ f2 sigmoid2(f2 g) {
    // an exponential that overflows gives 0
    return rcp_2(add2(ex2_2(mul2(g, dup2(-1.4426950408889634f))), dup2(1.f)));
}

// (1 + erf(g / sqrt 2)) / 2, e = exp(-g^2 / 2): the lower tail as e times a polynomial in 1 / (1 +
// 0.31 |g|), a minimax fit of degree 6 without constant term, 2^-17.6 of the tail for |g| <= 14,
// where e vanishes; the upper one is 1 less that, and neither cancels.  (Scalar: in packed
// arithmetic gelu took 48 us instead of 49 for 20000 x 1024, r = 4, but silu, in the same kernel,
// 45.7 instead of 43.6.  erff: 55, and nothing left of the value below g = -5.)
__device__ __forceinline__ float normal_cdf(float g, float e) {
    const float t = rcp(fmaf(fabsf(g), 0.31f, 1.f));
    float c = fmaf(t, -0.0739276037f, 0.1804459095f);
    c = fmaf(t, c, 0.0157496296f);
    c = fmaf(t, c, 0.1334271729f);
    c = fmaf(t, c, 0.120441936f);
    c = fmaf(t, c, 0.1238606423f);
    c *= t * e;
    return g < 0.f ? c : 1.f - c;
}

template <int ACT, bool GRAD>
__device__ __forceinline__ f2 act2(f2 g, f2 &d) {
    if constexpr (ACT == KRON_ACT_SILU) {
        const f2 s = sigmoid2(g), f = mul2(g, s);
        if (GRAD) d = fma2(f, fma2(s, dup2(-1.f), dup2(1.f)), s);
        return f;
    } else if constexpr (ACT == KRON_ACT_SIGMOID) {
        const f2 s = sigmoid2(g);
        if (GRAD) {
            // 1 - s as exp(-g) s, which keeps its bits where s is next to 1; s is 0 where exp(-g)
            // is infinite
            float t0, t1;
            unpack2(ex2_2(mul2(g, dup2(-1.4426950408889634f))), t0, t1);
            d = mul2(s, mul2(s, pack2(fminf(t0, 3.4e38f), fminf(t1, 3.4e38f))));
        }
        return s;
    } else if constexpr (ACT == KRON_ACT_GELU) {
        float lo, hi, e0, e1;
        unpack2(g, lo, hi);
        const f2 e = ex2_2(mul2(mul2(g, g), dup2(-0.72134752f)));     // exp(-g^2 / 2)
        unpack2(e, e0, e1);
        const f2 c = pack2(normal_cdf(lo, e0), normal_cdf(hi, e1));
        if (GRAD) {
            // g exp(-g^2 / 2) / sqrt(2 pi); nothing where the exponential vanishes
            const f2 gz = pack2(e0 == 0.f ? 0.f : lo, e1 == 0.f ? 0.f : hi);
            d = fma2(mul2(gz, e), dup2(0.39894228f), c);
        }
        return mul2(g, c);
    } else {
        // (1 + tanh(v)) / 2 = sigmoid(2 v) with v = sqrt(2/pi) (g + 0.044715 g^3)
        const f2 g2 = mul2(g, g);
        const f2 s = sigmoid2(mul2(mul2(g, dup2(1.5957691f)), fma2(g2, dup2(0.044715f), dup2(1.f))));
        if (GRAD) {
            const f2 w = mul2(s, fma2(s, dup2(-1.f), dup2(1.f)));
            float w0, w1, a, b;
            unpack2(w, w0, w1);
            unpack2(mul2(mul2(g, dup2(1.5957691f)), fma2(g2, dup2(0.134145f), dup2(1.f))), a, b);
            d = fma2(w, pack2(w0 == 0.f ? 0.f : a, w1 == 0.f ? 0.f : b), s);
        }
        return mul2(g, s);
    }
}

}  // namespace glu
}  // namespace kron
