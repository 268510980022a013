// glu.cu -- entry points of the gated Kronecker feed-forward half (kron_glu_forward,
// kron_glu_backward): checks, workspace, and the order of the launches.
//
//   h = act(g) * u,  g = x Wg + bg,  u = x Wu + bu,  W* = sum_i kron(S* (.) A*_i, B*_i)
//   du = dH act(g),  dg = dH u act'(g);  each projection's gradients as the layer's
//
// BF16: one tensor-core kernel forward; backward: the pre-activations' gradients, dX, the dense
// weight gradients and their contraction (glu_tc.cu, glu_wgrad.cu).  F32: one CUDA-core kernel
// for both projections and the activation (glu_f32.cu), or the layer's kernels for each with the
// elementwise kernels below; backward by the layer's kernels over both projections at once; FFMA
// bound.
#include "glu.h"

#include <math.h>
#include <stdarg.h>
#include <stdio.h>

namespace kron {
kron_status_t report_failure(kron_status_t st, const char *msg);

namespace {

using glu::Mode;
using glu::Plan;

kron_status_t bad(kron_status_t st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
kron_status_t bad(kron_status_t st, const char *fmt, ...) {
    char msg[240];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof(msg), fmt, ap);
    va_end(ap);
    return report_failure(st, msg);
}

kron_status_t cuda_bad(cudaError_t e, const char *what) {
    return bad(KRON_ERR_CUDA, "%s (%s): %s", what, launch_step(), cudaGetErrorString(e));
}

// h = act(g) * u, in place of u.
__global__ void gate_f32_kernel(const float4 *g, float4 *u, int64_t n4, int act) {
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n4;
         i += (int64_t)gridDim.x * blockDim.x) {
        const float4 a = g[i];
        float4 b = u[i];
        float d;
        b.x *= glu::act_f32(act, a.x, &d);
        b.y *= glu::act_f32(act, a.y, &d);
        b.z *= glu::act_f32(act, a.z, &d);
        b.w *= glu::act_f32(act, a.w, &d);
        u[i] = b;
    }
}

// (g, u) -> (dg, du), in place.
__global__ void gate_grad_f32_kernel(float4 *g, float4 *u, const float4 *dh, int64_t n4, int act) {
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n4;
         i += (int64_t)gridDim.x * blockDim.x) {
        float4 a = g[i], b = u[i];
        const float4 h = dh[i];
        float *pa = &a.x, *pb = &b.x;
        const float *ph = &h.x;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            float d;
            const float f = glu::act_f32(act, pa[t], &d);
            pa[t] = ph[t] * pb[t] * d;
            pb[t] = ph[t] * f;
        }
        g[i] = a;
        u[i] = b;
    }
}

__global__ void add_f32_kernel(float4 *y, const float4 *x, int64_t n4) {
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n4;
         i += (int64_t)gridDim.x * blockDim.x) {
        float4 a = y[i];
        const float4 b = x[i];
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
        y[i] = a;
    }
}

unsigned grid_for(int64_t n4) {
    const int64_t b = (n4 + 255) / 256;
    return (unsigned)(b < 148 * 16 ? (b > 0 ? b : 1) : 148 * 16);
}

size_t pad256(size_t n) { return (n + 255) & ~(size_t)255; }

kron_status_t check_sizes(int64_t N, int p, int q, int m1, int m2, int r, int activation,
                          kron_dtype_t dtype, unsigned flags, bool backward) {
    report_failure(KRON_OK, "");
    if (dtype != KRON_F32 && dtype != KRON_TF32 && dtype != KRON_BF16)
        return bad(KRON_ERR_INVALID_ARG, "unknown dtype %d", (int)dtype);
    if (activation < KRON_ACT_SILU || activation > KRON_ACT_SIGMOID)
        return bad(KRON_ERR_INVALID_ARG, "unknown activation %d", activation);
    if (flags) return bad(KRON_ERR_INVALID_ARG, "unknown flag bits 0x%x", flags);
    if (N < 0 || p < 1 || q < 1 || m1 < 1 || m2 < 1 || r < 1)
        return bad(KRON_ERR_INVALID_ARG,
                   "sizes must be N >= 0 and p, q, m1, m2, r >= 1 (got N=%lld p=%d q=%d m1=%d "
                   "m2=%d r=%d)", (long long)N, p, q, m1, m2, r);
    if (dtype == KRON_TF32)
        return bad(KRON_ERR_UNSUPPORTED, "the gated half runs on KRON_F32 and KRON_BF16");
    if ((int64_t)p * m1 > (1 << 20) || (int64_t)q * m2 > (1 << 20) || r > 1024 ||
        N > ((int64_t)1 << 30))
        return bad(KRON_ERR_INVALID_ARG, "sizes out of range");
    const int mult = dtype == KRON_BF16 ? 8 : 4;
    if (m1 % mult || m2 % mult)
        return bad(KRON_ERR_UNSUPPORTED, "m1 and m2 must be multiples of %d for this dtype", mult);
    const Shape s{N > 0 ? N : 1, p, q, m1, m2, r};
    Plan pl;
    if (dtype == KRON_BF16) {
        if (p > 1024 || q > 1024 || m1 > 256 || m2 > 256)
            return bad(KRON_ERR_UNSUPPORTED,
                       "KRON_BF16 takes p and q up to 1024 and m1 and m2 up to 256 (got p=%d q=%d "
                       "m1=%d m2=%d)", p, q, m1, m2);
        if (!glu::tc_plan(&pl, s, glu::kForward, kRowParts))
            return bad(KRON_ERR_UNSUPPORTED,
                       "no tensor-core kernel for p=%d q=%d m1=%d m2=%d r=%d: too large r (p + m1) "
                       "for shared memory", p, q, m1, m2, r);
        if (backward && !glu::tc_plan(&pl, s, glu::kInput, kRowParts))
            return bad(KRON_ERR_UNSUPPORTED,
                       "no tensor-core kernel for the gradients of p=%d q=%d m1=%d m2=%d r=%d: too "
                       "large r (q + m2) for shared memory", p, q, m1, m2, r);
    } else if (simt_forward_rows(s) <= 0 || (backward && simt_backward_rows(s) <= 0)) {
        return bad(KRON_ERR_UNSUPPORTED,
                   "no %s kernel for p=%d q=%d m1=%d m2=%d r=%d: the FP32 tile does not fit shared "
                   "memory", backward ? "backward" : "forward", p, q, m1, m2, r);
    }
    return KRON_OK;
}

// F32: whether both projections run in one kernel with the activation.  The compiled shape's own
// kernels are faster than that one where they have rows to fill the SMs with: forward of 2000 rows
// 90 us in one kernel and 101 in two and an elementwise pass, 2368 rows 117 and 103, 20000 rows
// 766 and 616.
bool fused_f32(const Shape &s) {
    const bool compiled = s.p == 32 && s.q == 32 && s.m1 == 32 && s.m2 == 32 && s.r == 4;
    return glu::f32_pre_supported(s) && !(compiled && s.N >= glu::kCompiledRows);
}

// Workspace: forward F32 [g] unless fused; backward F32 [g][u][dX of up][partials of both];
// backward BF16 [dg][du][weight gradients].
size_t need_bytes(const Shape &s, kron_dtype_t dtype, bool backward) {
    const size_t h = (size_t)s.N * s.d_out(), x = (size_t)s.N * s.d_in();
    if (dtype == KRON_BF16)
        return backward ? 2 * pad256(2 * h) + glu::wgrad_plan(s, kRowParts).ws_bytes : 0;
    if (!backward) return fused_f32(s) ? 0 : pad256(4 * h);
    return 2 * pad256(4 * h) + pad256(4 * x) +
           2 * kron_linear_workspace_size(s.N, s.p, s.q, s.m1, s.m2, s.r, KRON_F32);
}

bool a16(const void *p) { return ((uintptr_t)p & 15u) == 0; }

kron_status_t check_workspace(const void *ws, size_t bytes, size_t need) {
    if (need == 0) return KRON_OK;
    if (!ws || bytes < need)
        return bad(KRON_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need,
                   ws ? bytes : (size_t)0);
    if ((uintptr_t)ws & 255u)
        return bad(KRON_ERR_ALIGNMENT, "workspace must be 256-byte aligned");
    return KRON_OK;
}

// The factors of one projection of a stacked fp32 tensor.
struct Half {
    const float *S, *A, *B, *bias;
};
Half half_of(const void *S, const void *A, const void *B, const void *bias, const Shape &s, int k) {
    const size_t pq = (size_t)s.p * s.q, mm = (size_t)s.m1 * s.m2;
    return Half{(const float *)S + k * pq, (const float *)A + k * s.r * pq,
                (const float *)B + k * s.r * mm,
                bias ? (const float *)bias + (size_t)k * s.d_out() : nullptr};
}

// Both pre-activations of the F32 path.
cudaError_t pre_f32(const void *x, const void *S, const void *A, const void *B, const void *bias,
                    float *g, float *u, const Shape &s, cudaStream_t st) {
    const Half a = half_of(S, A, B, bias, s, 0), b = half_of(S, A, B, bias, s, 1);
    const cudaError_t e = simt_forward(x, a.S, a.A, a.B, a.bias, g, s, false, st);
    return e != cudaSuccess ? e : simt_forward(x, b.S, b.A, b.B, b.bias, u, s, false, st);
}

}  // namespace
}  // namespace kron

using namespace kron;

extern "C" {

size_t kron_glu_workspace_size(int64_t N, int p, int q, int m1, int m2, int r, kron_dtype_t dtype,
                               int backward) {
    const bool back = backward != 0;
    if (check_sizes(N, p, q, m1, m2, r, KRON_ACT_SILU, dtype, 0, back) != KRON_OK || N == 0)
        return 0;
    return need_bytes(Shape{N, p, q, m1, m2, r}, dtype, backward != 0);
}

kron_status_t kron_glu_forward(const void *x, const void *S, const void *A, const void *B,
                               const void *bias, void *h, int64_t N, int p, int q, int m1, int m2,
                               int r, int activation, kron_dtype_t dtype, unsigned flags,
                               void *workspace, size_t workspace_bytes, void *stream) {
    kron_status_t st = check_sizes(N, p, q, m1, m2, r, activation, dtype, flags, false);
    if (st != KRON_OK) return st;
    if (!S || !A || !B || (N > 0 && (!x || !h)))
        return bad(KRON_ERR_INVALID_ARG, "S, A, B (and x, h when N > 0) must be non-null");
    if (!a16(x) || !a16(S) || !a16(A) || !a16(B) || !a16(bias) || !a16(h))
        return bad(KRON_ERR_ALIGNMENT, "all tensors must be 16-byte aligned");
    if (N == 0) return KRON_OK;
    if (h == x) return bad(KRON_ERR_INVALID_ARG, "h must not be x: not an in-place operation");
    const Shape s{N, p, q, m1, m2, r};
    st = check_workspace(workspace, workspace_bytes, need_bytes(s, dtype, false));
    if (st != KRON_OK) return st;
    cudaStream_t cs = (cudaStream_t)stream;
    cudaError_t e;
    if (dtype == KRON_BF16) {
        Plan pl;
        glu::tc_plan(&pl, s, glu::kForward, tc::num_sms());
        glu::TcArgs a{};
        a.src0 = x;
        a.S = S;
        a.A = A;
        a.B = B;
        a.bias = bias;
        a.out0 = h;
        a.N = N;
        a.activation = activation;
        e = glu::tc_run(pl, a, glu::kForward, cs);
    } else {
        if (fused_f32(s)) {
            e = glu::f32_pre(x, S, A, B, bias, nullptr, h, nullptr, s, activation, false, cs);
        } else {
            e = pre_f32(x, S, A, B, bias, (float *)workspace, (float *)h, s, cs);
            if (e == cudaSuccess) {
                const int64_t n4 = N * s.d_out() / 4;
                launch_step() = "gate launch";
                gate_f32_kernel<<<grid_for(n4), 256, 0, cs>>>(
                    (const float4 *)workspace, (float4 *)h, n4, activation);
                e = cudaGetLastError();
            }
        }
    }
    return e == cudaSuccess ? KRON_OK : cuda_bad(e, "gated forward");
}

kron_status_t kron_glu_backward(const void *x, const void *S, const void *A, const void *B,
                                const void *bias, const void *dH, void *dX, void *dS, void *dA,
                                void *dB, void *dbias, int64_t N, int p, int q, int m1, int m2,
                                int r, int activation, kron_dtype_t dtype, unsigned flags,
                                void *workspace, size_t workspace_bytes, void *stream) {
    kron_status_t st = check_sizes(N, p, q, m1, m2, r, activation, dtype, flags, true);
    if (st != KRON_OK) return st;
    if (!S || !A || !B || !dS || !dA || !dB || (N > 0 && (!x || !dH)))
        return bad(KRON_ERR_INVALID_ARG,
                   "S, A, B, dS, dA, dB (and x, dH when N > 0) must be non-null");
    if (!a16(x) || !a16(S) || !a16(A) || !a16(B) || !a16(bias) || !a16(dH) || !a16(dX) ||
        !a16(dS) || !a16(dA) || !a16(dB) || !a16(dbias))
        return bad(KRON_ERR_ALIGNMENT, "all tensors must be 16-byte aligned");
    if ((N > 0 && dX == x && dX) || dS == S || dA == A || dB == B || (dbias && dbias == bias))
        return bad(KRON_ERR_INVALID_ARG, "a gradient must not be the tensor that it belongs to");
    const Shape s{N, p, q, m1, m2, r};
    cudaStream_t cs = (cudaStream_t)stream;
    const size_t E = dtype == KRON_BF16 ? 2 : 4, pq = (size_t)p * q, mm = (size_t)m1 * m2;
    const size_t din = (size_t)s.d_in(), dout = (size_t)s.d_out();
    cudaError_t e = cudaSuccess;
    if (N == 0) {
        launch_step() = "zero gradients";
        e = cudaMemsetAsync(dS, 0, 2 * pq * E, cs);
        if (e == cudaSuccess) e = cudaMemsetAsync(dA, 0, 2 * r * pq * E, cs);
        if (e == cudaSuccess) e = cudaMemsetAsync(dB, 0, 2 * r * mm * E, cs);
        if (e == cudaSuccess && dbias) e = cudaMemsetAsync(dbias, 0, 2 * dout * E, cs);
        return e == cudaSuccess ? KRON_OK : cuda_bad(e, "gated backward");
    }
    st = check_workspace(workspace, workspace_bytes, need_bytes(s, dtype, true));
    if (st != KRON_OK) return st;
    char *ws = (char *)workspace;
    const size_t hb = pad256((size_t)N * dout * E);
    if (dtype == KRON_BF16) {
        const int sms = tc::num_sms();
        void *dg = ws, *du = ws + hb;
        Plan pl;
        glu::tc_plan(&pl, s, glu::kPre, sms);
        glu::TcArgs a{};
        a.src0 = x;
        a.S = S;
        a.A = A;
        a.B = B;
        a.bias = bias;
        a.dH = dH;
        a.out0 = dg;
        a.out1 = du;
        a.N = N;
        a.activation = activation;
        e = glu::tc_run(pl, a, glu::kPre, cs);
        if (e == cudaSuccess && dX) {
            glu::tc_plan(&pl, s, glu::kInput, sms);
            a.src0 = dg;
            a.src1 = du;
            a.bias = a.dH = nullptr;
            a.out0 = dX;
            a.out1 = nullptr;
            e = glu::tc_run(pl, a, glu::kInput, cs);
        }
        if (e == cudaSuccess)
            e = glu::wgrad_run(glu::wgrad_plan(s, kRowParts), x, dg, du, S, A, B, dS, dA, dB,
                               dbias, ws + 2 * hb, s, cs);
        return e == cudaSuccess ? KRON_OK : cuda_bad(e, "gated backward");
    }
    float *g = (float *)ws, *u = (float *)(ws + hb), *dx2 = (float *)(ws + 2 * hb);
    float *part = (float *)(ws + 2 * hb + pad256((size_t)N * din * 4));
    const int max_parts = (int)(kron_linear_workspace_size(N, p, q, m1, m2, r, KRON_F32) /
                                (partial_stride(s) * sizeof(float)));
    int parts = max_parts;
    if (fused_f32(s)) {
        e = glu::f32_pre(x, S, A, B, bias, dH, g, u, s, activation, true, cs);
    } else {
        e = pre_f32(x, S, A, B, bias, g, u, s, cs);
        if (e == cudaSuccess) {
            const int64_t n4 = N * s.d_out() / 4;
            launch_step() = "gate launch";
            gate_grad_f32_kernel<<<grid_for(n4), 256, 0, cs>>>((float4 *)g, (float4 *)u,
                                                              (const float4 *)dH, n4, activation);
            e = cudaGetLastError();
        }
    }
    if (e == cudaSuccess)
        e = glu::f32_backward_pair(x, S, A, B, g, u, dX, dX ? dx2 : nullptr, part, max_parts,
                                   &parts, s, cs);
    if (e == cudaSuccess)
        e = glu::reduce_partials_pair(part, parts, S, A, (float *)dS, (float *)dA, (float *)dB,
                                      (float *)dbias, s, cs);
    if (e == cudaSuccess && dX) {
        const int64_t n4 = N * s.d_in() / 4;
        launch_step() = "dX launch";
        add_f32_kernel<<<grid_for(n4), 256, 0, cs>>>((float4 *)dX, (const float4 *)dx2, n4);
        e = cudaGetLastError();
    }
    return e == cudaSuccess ? KRON_OK : cuda_bad(e, "gated backward");
}

}  // extern "C"
