// distill.cu -- distillation loss against a teacher's top logits (kron_distill_forward,
// kron_distill_backward, kron_distill_step; include/kron_linear.h).
//
// Row n of the student's logits x [V], the teacher's K logits t_j at the columns i_j:
//   p_j  = softmax_j(t_j / tau) over the row's entries,   q = softmax(x / tau)
//   loss = w [ (1 - lam) tau^2 sum_j p_j (log p_j - log q_{i_j}) + lam (lse(x) - x_label) ]
//   dx_v = w dl [ (1 - lam) tau (q_v - sum_{j: i_j = v} p_j) + lam (softmax(x)_v - [v = label]) ]
//
// One CTA of 256 threads per row, five to eight per SM (more threads where there are few rows).
// Pass 1 reads the row with a running maximum m per thread and the sums of exp((x - m)/tau) and
// exp(x - m); pass 2 (gradient) reads it again, from L2 where the rows at work fit there, and
// writes the dense part c_t q + c_1 softmax(x); the K + 1 columns that the teacher and the label
// touch are then overwritten by the thread that owns the first entry of the column, in fp32, from
// logits fetched before anything is written (so dlogits may be the logits).  Exponents are
// differences from a value next to the row's maximum, however far from zero the logits are.
// Bound: HBM moves the logits once in and once out (126 us for 4096 x 50257 bf16); per element
// and pass one ex2 (two for a tau other than 1, 2 and 4), 92 us on the special-function units,
// and with the packed FP32 instructions some 11 issue slots.  Measured 184 to 188 us
// (earlier forms of it: 181; with scalar FP32 instructions 191; 512 threads, three CTAs per SM:
// 212; rows split over clusters of four CTAs and held in registers, one read: 301, the barriers
// of the shorter pieces not covered).  740 rows at work exceed L2 where a row has more than 170
// KB: 1024 x 50257 fp32 read 333 MB for 206, 1024 x 131072 bf16 462 for 268.
#include "../../include/kron_linear.h"
#include "internal.h"
#include "packed.cuh"

#include <cuda_bf16.h>
#include <math.h>
#include <stdio.h>

namespace kron {
kron_status_t report_failure(kron_status_t st, const char *msg);

namespace {

constexpr int kMaxK = 1024;      // teacher entries per row
constexpr float kLog2e = 1.4426950408889634f;

struct Args {
    const void *logits;
    int64_t ld;
    const float *values;
    const void *indices;
    const int64_t *labels;
    const float *weights;
    const float *dloss;
    float *loss;
    float *lse;
    const float *lse_in;
    void *dlogits;
    int64_t ld_out;
    int V, K;
    float tau, lam;
    bool idx64;
};

// How the two exponentials of one logit are formed.
enum Exps {
    kOne,     // one temperature only (tau = 1, or one of the two terms has weight zero)
    kSquare,  // tau = 2: exp(x) = exp(x/2)^2
    kFourth,  // tau = 4
    kTwo      // any other tau
};

template <typename T> struct Vec;
template <> struct Vec<float> {
    static constexpr int n = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, f2 (&f)[2]) {
        f[0] = pack2(__uint_as_float(u.x), __uint_as_float(u.y));
        f[1] = pack2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint4 pack(const f2 (&f)[2]) {
        float a, b, c, d;
        unpack2(f[0], a, b);
        unpack2(f[1], c, d);
        return make_uint4(__float_as_uint(a), __float_as_uint(b), __float_as_uint(c),
                          __float_as_uint(d));
    }
    // the largest of the vector's values (a NaN only where all are)
    static __device__ __forceinline__ float max(const uint4 &u) {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)),
                     fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float v) { *p = v; }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int n = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, f2 (&f)[4]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            f[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint4 pack(const f2 (&f)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            unpack2(f[i], lo, hi);
            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
    static __device__ __forceinline__ float max(const uint4 &u) {
        const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&u);
        const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(m), __high2float(m));
    }
    static __device__ __forceinline__ float get(const __nv_bfloat16 *p) {
        return __bfloat162float(*p);
    }
    static __device__ __forceinline__ void put(__nv_bfloat16 *p, float v) {
        *p = __float2bfloat16_rn(v);
    }
};

// Running maximum of the logits and the sums of exp((x - m) a / log2 e) for the two scales.
struct Stat {
    float m, s, s1;
};

template <int E> __device__ __forceinline__ float second(float e, float d) {
    if constexpr (E == kSquare) return e * e;
    if constexpr (E == kFourth) return (e * e) * (e * e);
    if constexpr (E == kTwo) return ex2(d * kLog2e);
    return 0.f;
}

// Moves the sums of `st` to the maximum m (>= st.m).  A maximum of -inf means nothing but
// -inf has been seen, and the sums are then zero.
template <int E> __device__ __forceinline__ void rebase(Stat &st, float m, float a) {
    if (m > st.m) {
        const float d = st.m - m;      // -inf at the first finite value: factors 0
        const float e = ex2(d * a);
        st.s *= e;
        if constexpr (E != kOne) st.s1 *= second<E>(e, d);
        st.m = m;
    }
}

template <int E> __device__ __forceinline__ void merge(Stat &st, const Stat &o, float a) {
    Stat t = o;
    const float m = fmaxf(st.m, t.m);
    rebase<E>(st, m, a);
    rebase<E>(t, m, a);
    st.s += t.s;
    if constexpr (E != kOne) st.s1 += t.s1;
}

template <int E> __device__ __forceinline__ void add_one(Stat &st, float x, float a) {
    rebase<E>(st, x, a);
    // -inf contributes nothing (also while every value so far is -inf); a NaN or +inf makes
    // the sum NaN, as the definition does
    const float d = x == -INFINITY ? -INFINITY : x - st.m;
    const float e = ex2(d * a);
    st.s += e;
    if constexpr (E != kOne) st.s1 += second<E>(e, d);
}

template <int E> __device__ __forceinline__ Stat shuffle_xor(const Stat &st, int o) {
    Stat t;
    t.m = __shfl_xor_sync(0xffffffffu, st.m, o);
    t.s = __shfl_xor_sync(0xffffffffu, st.s, o);
    t.s1 = E == kOne ? 0.f : __shfl_xor_sync(0xffffffffu, st.s1, o);
    return t;
}

// What the columns that are written last need: what is subtracted from their logits first, the
// coefficients of the teacher's and the label's share, the label's logit and the label.
struct Last {
    float at, share, hard, xlab;
    int label;
};

// What a row needs of the teacher, in shared memory: columns (-1: no entry), probabilities,
// student logits at the columns.
struct RowSmem {
    alignas(16) int col[kMaxK + 4];
    float prob[kMaxK];
    float x[kMaxK];
    Stat warp[32];
    float red[32];
    float redm[32];
    Last last;
};

// Sum over the CTA in a fixed order; every thread gets it.
template <int kThreads>
__device__ __forceinline__ float block_sum(float v, float *red) {
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = 0.f;
    for (int i = 0; i < kThreads / 32; ++i) t += red[i];
    return t;
}
template <int kThreads>
__device__ __forceinline__ float block_max(float v, float *red) {
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float t = -INFINITY;
    for (int i = 0; i < kThreads / 32; ++i) t = fmaxf(t, red[i]);
    return t;
}

// Where a row's probabilities are read off: q = exp((x - at)/tau) exp(t), softmax(x) =
// exp(x - at) exp(one), with `at` next to the row's maximum: the exponents are small however far
// from zero the logits are.
struct Origin {
    float at, t, one;
};
// From pass 1: the maximum and the logarithms of the two sums.
__device__ __forceinline__ Origin origin_of(float m, float lsum_t, float lsum_1) {
    return {m, -lsum_t, -lsum_1};
}
// From the log-sum-exps, in 64 bits: no error but theirs.  With one exponential only the one at
// its temperature is known.
template <int E>
__device__ __forceinline__ Origin origin_of(const float *lse, float tau, bool hard) {
    const float lse_t = hard ? lse[1] : lse[0];
    const float at = E == kOne ? (float)((double)lse_t * tau) : lse[1];
    const float t = (float)((double)at / tau - lse_t);
    return {at, t, E == kOne ? t : 0.f};
}
// Rounding a log-sum-exp moves every probability by 2^-24 of its size (its products with 1/tau by
// half as much): beyond this size, 1e-4 of a probability, a gradient forms the sums again.
constexpr float kLseMax = 1024.f;
__device__ __forceinline__ bool lse_is_near(const float *lse) {
    return fabsf(lse[0]) <= kLseMax && fabsf(lse[1]) <= kLseMax;
}

// The threads' statistics merged in a fixed order; every thread gets the row's.
template <int E, int kThreads>
__device__ __forceinline__ Stat block_stat(Stat st, float a, Stat *warp) {
    for (int o = 16; o; o >>= 1) {
        const Stat t = shuffle_xor<E>(st, o);
        merge<E>(st, t, a);
    }
    if ((threadIdx.x & 31) == 0) warp[threadIdx.x >> 5] = st;
    __syncthreads();
    Stat r = warp[0];
    for (int i = 1; i < kThreads / 32; ++i) merge<E>(r, warp[i], a);
    return r;
}

// The dense part of a row's gradient, soft q + hard softmax(x), of one or two logits.
template <int E> struct Dense {
    f2 a, b, ct, c1, b1;
    // Whether (x - at) a is formed as one multiply-add x a + b whose rounded constant the
    // coefficients make up for; else the caller subtracts `at` first (a fourth instruction in
    // packed arithmetic: 197 us instead of 188 for 4096 x 50257 bf16, tau = 2, with the loss).
    static __device__ __forceinline__ bool is_near(const Origin &o, float scale) {
        return fabsf(o.at * scale) <= 0x1p24f && (E != kTwo || fabsf(o.at * kLog2e) <= 0x1p24f);
    }
    // scale: log2(e) / tau (or log2(e), where only the label's term is there)
    __device__ __forceinline__ Dense(float soft, float hard, const Origin &o, float scale) {
        const bool near = is_near(o, scale);
        const float bt = near ? -o.at * scale : 0.f, bo = near ? -o.at * kLog2e : 0.f;
        // what is left of at a + b, at most 1
        const float rt = near ? fmaf(o.at, scale, bt) : 0.f;
        const float ro = near ? fmaf(o.at, kLog2e, bo) : 0.f;
        const float r1 = E == kSquare ? 2.f * rt : E == kFourth ? 4.f * rt : E == kTwo ? ro : rt;
        const float ft = soft * ex2(fmaf(o.t, kLog2e, -rt));
        const float f1 = hard * ex2(fmaf(o.one, kLog2e, -r1));
        a = dup2(scale);
        b = dup2(bt);
        b1 = dup2(bo);
        ct = dup2(E == kOne ? ft + f1 : ft);
        c1 = dup2(f1);
    }
    __device__ __forceinline__ f2 two(f2 v) const {
        const f2 e = ex2_2(fma2(v, a, b));
        if constexpr (E == kOne) return mul2(ct, e);
        if constexpr (E == kSquare) return mul2(e, fma2(c1, e, ct));
        if constexpr (E == kFourth) return mul2(e, fma2(mul2(c1, e), mul2(e, e), ct));
        return fma2(c1, ex2_2(fma2(v, dup2(kLog2e), b1)), mul2(ct, e));
    }
    __device__ __forceinline__ float one(float v) const {
        float lo, hi;
        unpack2(two(dup2(v)), lo, hi);
        return lo;
    }
};

// Short rows (a classifier's logits): a warp per row, the teacher's entries in its own part of
// shared memory.  20000 x 10 with its gradient takes 20 us; with a CTA per row it took
// 121 us, nearly all of it starting and ending CTAs.
constexpr int kShortV = 1024, kShortK = 64, kShortWarps = 8;

template <typename T, int E, bool STATS, bool GRAD>
__global__ void __launch_bounds__(32 * kShortWarps) distill_short_kernel(const Args g, int64_t N) {
    __shared__ int s_col[kShortWarps][kShortK];
    __shared__ float s_prob[kShortWarps][kShortK], s_x[kShortWarps][kShortK];
    using Vc = Vec<T>;
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, V = g.V, K = g.K;
    const int64_t row = (int64_t)blockIdx.x * kShortWarps + wp;
    if (row >= N) return;
    const T *x = static_cast<const T *>(g.logits) + row * g.ld;
    T *out = GRAD ? static_cast<T *>(g.dlogits) + row * g.ld_out : nullptr;
    const float w = g.weights ? g.weights[row] : 1.f;
    // weight 0 wins over an infinite or NaN dloss
    const float coef = GRAD && g.dloss && w != 0.f ? w * g.dloss[row] : w;
    if (coef == 0.f) {
        if (STATS && lane == 0) {
            g.loss[row] = 0.f;
            if (g.lse) g.lse[2 * row] = g.lse[2 * row + 1] = 0.f;
        }
        if (GRAD)
            for (int v = lane; v < V; v += 32) Vc::put(out + v, 0.f);
        return;
    }
    const bool hard_only = g.lam == 1.f;
    const float inv_tau = hard_only ? 1.f : 1.f / g.tau, a = kLog2e * inv_tau;
    int *col = s_col[wp];
    float *prob = s_prob[wp], *xs = s_x[wp];
    float tm = -INFINITY;
    for (int j = lane; j < K; j += 32) {
        const int64_t i = g.idx64 ? static_cast<const int64_t *>(g.indices)[row * K + j]
                                  : static_cast<const int *>(g.indices)[row * K + j];
        const bool there = i >= 0 && i < V;
        col[j] = there ? (int)i : -1;
        prob[j] = there ? g.values[row * K + j] : -INFINITY;
        xs[j] = there ? Vc::get(x + i) : 0.f;
        tm = fmaxf(tm, prob[j]);
    }
    const int64_t lab64 = g.labels ? g.labels[row] : -1;
    const int label = lab64 >= 0 && lab64 < V ? (int)lab64 : -1;
    const float xlab = label >= 0 ? Vc::get(x + label) : 0.f;
    for (int o = 16; o; o >>= 1) tm = fmaxf(tm, __shfl_xor_sync(0xffffffffu, tm, o));
    float ts = 0.f;
    for (int j = lane; j < K; j += 32) {
        const float e = prob[j] == -INFINITY ? 0.f : ex2((prob[j] - tm) * (kLog2e / g.tau));
        prob[j] = e;
        ts += e;
    }
    for (int o = 16; o; o >>= 1) ts += __shfl_xor_sync(0xffffffffu, ts, o);
    const bool any = ts != 0.f;
    const float its = any ? 1.f / ts : 0.f;
    Origin origin;
    Stat st{-INFINITY, 0.f, 0.f};
    float lsum = 0.f, lsum1 = 0.f;
    if (STATS || !lse_is_near(g.lse_in + 2 * row)) {
        for (int v = lane; v < V; v += 32) add_one<E>(st, Vc::get(x + v), a);
        for (int o = 16; o; o >>= 1) {
            const Stat t = shuffle_xor<E>(st, o);
            merge<E>(st, t, a);
        }
        // (with one exponential and both terms, tau is 1 and the two agree)
        lsum = logf(st.s), lsum1 = E == kOne ? lsum : logf(st.s1);
        origin = origin_of(st.m, lsum, lsum1);
    } else {
        origin = origin_of<E>(g.lse_in + 2 * row, hard_only ? 1.f : g.tau, hard_only);
    }
    if constexpr (STATS) {
        const float llse = logf(ts);
        float kl = 0.f;
        if (!hard_only)
            for (int j = lane; j < K; j += 32)
                if (col[j] >= 0 && prob[j] != 0.f)
                    kl += prob[j] * its * ((g.values[row * K + j] - tm) * inv_tau - llse -
                                           ((xs[j] - st.m) * inv_tau - lsum));
        for (int o = 16; o; o >>= 1) kl += __shfl_xor_sync(0xffffffffu, kl, o);
        if (lane == 0) {
            float l = (1.f - g.lam) * g.tau * g.tau * kl;
            if (g.lam != 0.f && label >= 0) l += g.lam * (st.m - xlab + lsum1);
            g.loss[row] = w * l;
            if (g.lse) {
                g.lse[2 * row] = st.m * inv_tau + lsum;
                g.lse[2 * row + 1] = E == kOne ? st.m * inv_tau + lsum : st.m + lsum1;
            }
        }
    }
    if constexpr (GRAD) {
        const float soft = hard_only || !any ? 0.f : coef * (1.f - g.lam) * g.tau;
        const float hard = g.lam != 0.f && label >= 0 ? coef * g.lam : 0.f;
        __syncwarp();           // the row's gathers and entries are complete
        if (soft == 0.f && hard == 0.f) {   // no term: zero, whatever the logits hold
            for (int v = lane; v < V; v += 32) Vc::put(out + v, 0.f);
            return;
        }
        const Dense<E> dense(soft, hard, origin, a);
        const float at = Dense<E>::is_near(origin, a) ? 0.f : origin.at;
        const float share = soft == 0.f ? 0.f : soft * its;
        for (int v = lane; v < V; v += 32) Vc::put(out + v, dense.one(Vc::get(x + v) - at));
        __syncwarp();
        bool listed = false;
        for (int j = lane; j < K; j += 32) {
            const int c = col[j];
            if (c < 0) continue;
            listed = listed || c == label;
            float p = 0.f;
            bool first = true;  // a column listed more than once: its first entry writes it
            for (int k = 0; k < K; ++k)
                if (col[k] == c) {
                    if (k < j) first = false;
                    p += prob[k];
                }
            if (first)
                Vc::put(out + c, dense.one(xs[j] - at) - (share == 0.f ? 0.f : share * p) -
                                     (c == label ? hard : 0.f));
        }
        listed = __any_sync(0xffffffffu, listed);
        if (lane == 0 && label >= 0 && !listed) Vc::put(out + label, dense.one(xlab - at) - hard);
    }
}

// A row's sums formed again by a gradient, for log-sum-exps that are too far from zero.  A call,
// whose registers are not the gradient's (inlined: 157 -> 168 us for 4096 x 50257 bf16).
template <typename T, int E, int kThreads>
__device__ __noinline__ Origin far_origin(const T *x, int V, float a, Stat *warp) {
    Stat st{-INFINITY, 0.f, 0.f};
    for (int v = threadIdx.x; v < V; v += kThreads) add_one<E>(st, Vec<T>::get(x + v), a);
    const Stat r = block_stat<E, kThreads>(st, a, warp);
    const float lsum = logf(r.s);
    return origin_of(r.m, lsum, E == kOne ? lsum : logf(r.s1));
}

// Threads per SM for which registers are set aside.  Loss and gradient in one kernel take five
// CTAs of 256 threads (48 registers) rather than six (40): 4096 x 50257 bf16 at tau = 1, 2 and 4
// took 183, 188 and 195 us and 192, 188 and 191; 1023 x 32000 38, 39 and 41 and 42, 41 and 43.
constexpr int threads_per_sm(bool stats, bool grad, int threads) {
    return !stats ? 2048 : grad && threads == 256 ? 1280 : 1536;
}

template <typename T, int E, bool STATS, bool GRAD, int kThreads>
__global__ void __launch_bounds__(kThreads, threads_per_sm(STATS, GRAD, kThreads) / kThreads)
distill_kernel(const Args g) {
    __shared__ RowSmem sm;
    using Vc = Vec<T>;
    constexpr int n = Vc::n;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x;
    const T *x = static_cast<const T *>(g.logits) + row * g.ld;
    T *out = GRAD ? static_cast<T *>(g.dlogits) + row * g.ld_out : nullptr;
    const float w = g.weights ? g.weights[row] : 1.f;
    // weight 0 wins over an infinite or NaN dloss
    const float coef = GRAD && g.dloss && w != 0.f ? w * g.dloss[row] : w;
    const int V = g.V, K = g.K;

    // 16-byte body of the row, aligned for the logits; the gradient's vector stores also
    // need the output row at the same offset from a 16-byte boundary
    const int head = min(V, (int)(((16 - ((uintptr_t)x & 15)) & 15) / sizeof(T)));
    const int nv = (V - head) / n;
    const uint4 *xv = reinterpret_cast<const uint4 *>(x + head);
    const bool same = GRAD && (((uintptr_t)x ^ (uintptr_t)out) & 15) == 0;

    if (coef == 0.f) {   // a row without weight: zero, whatever its logits hold
        if (STATS && tid == 0) {
            g.loss[row] = 0.f;
            if (g.lse) g.lse[2 * row] = g.lse[2 * row + 1] = 0.f;
        }
        if (GRAD)
            for (int v = tid; v < V; v += kThreads) Vc::put(out + v, 0.f);
        return;
    }

    // the temperature of the (only, or first) exponential
    const bool hard_only = g.lam == 1.f;
    const float inv_tau = hard_only ? 1.f : 1.f / g.tau;
    const float a = kLog2e * inv_tau;

    // ---- the teacher's distribution over the row's entries
    float tm = -INFINITY;
    const int Kp = (K + 3) & ~3;
    for (int j = tid; j < Kp; j += kThreads) {
        int64_t i = -1;
        if (j < K)
            i = g.idx64 ? static_cast<const int64_t *>(g.indices)[row * K + j]
                        : static_cast<const int *>(g.indices)[row * K + j];
        const bool there = i >= 0 && i < V;
        const float t = there ? g.values[row * K + j] : -INFINITY;
        sm.col[j] = there ? (int)i : -1;
        if (j < K) {
            sm.prob[j] = t;
            sm.x[j] = there ? Vc::get(x + i) : 0.f;
        }
        tm = fmaxf(tm, t);
    }
    const int64_t lab64 = g.labels ? g.labels[row] : -1;
    const int label = lab64 >= 0 && lab64 < V ? (int)lab64 : -1;
    const float xlab = label >= 0 ? Vc::get(x + label) : 0.f;

    tm = block_max<kThreads>(tm, sm.redm);
    float ts = 0.f;
    bool twice = false, listed = false;   // a column listed twice; the label's column listed
    for (int j = tid; j < K; j += kThreads) {
        const float t = sm.prob[j];
        const float e = t == -INFINITY ? 0.f : ex2((t - tm) * (kLog2e / g.tau));
        sm.prob[j] = e;
        ts += e;
        listed = listed || (label >= 0 && sm.col[j] == label);
    }
    if constexpr (GRAD) {
        // all threads share the pairs: thread tid has entry j = tid % step and every G-th four
        // of the entries before it
        for (int j0 = 0; j0 < K; j0 += kThreads) {
            const int step = min(K - j0, kThreads), G = kThreads / step;
            const int j = j0 + tid % step, part = tid / step, c = sm.col[j];
            if (part < G && c >= 0)
                for (int k = 4 * part; k < j; k += 4 * G) {
                    const int4 o = *reinterpret_cast<const int4 *>(sm.col + k);
                    twice = twice || o.x == c || (o.y == c && k + 1 < j) ||
                            (o.z == c && k + 2 < j) || (o.w == c && k + 3 < j);
                }
        }
    }
    ts = block_sum<kThreads>(ts, sm.red);
    const bool any = ts != 0.f;   // NaN counts: it has to show
    const float its = any ? 1.f / ts : 0.f;

    // ---- the student's log-sum-exp at both temperatures
    Origin origin;
    if constexpr (STATS) {
        Stat st{-INFINITY, 0.f, 0.f};
        // sums of the thread's even and odd elements, relative to st.m
        f2 sum = pack2(0.f, 0.f), sum1 = sum;
        const f2 a2 = pack2(a, a), l2 = pack2(kLog2e, kLog2e);
        auto add_vec = [&](const uint4 &u) {
            const float m = Vc::max(u);
            if (m > st.m) {
                const float d = st.m - m, e = ex2(d * a);
                sum = mul2(sum, pack2(e, e));
                if constexpr (E != kOne) {
                    const float e1 = second<E>(e, d);
                    sum1 = mul2(sum1, pack2(e1, e1));
                }
                st.m = m;
            }
            const float base = st.m == -INFINITY ? 0.f : -st.m;
            const f2 b2 = pack2(base, base);
            f2 f[n / 2];
            Vc::unpack(u, f);
#pragma unroll
            for (int i = 0; i < n / 2; ++i) {
                const f2 d = add2(f[i], b2);      // exact next to the maximum, however large
                const f2 e = ex2_2(mul2(d, a2));
                sum = add2(sum, e);
                if constexpr (E == kSquare) sum1 = fma2(e, e, sum1);
                if constexpr (E == kFourth) {
                    const f2 q = mul2(e, e);
                    sum1 = fma2(q, q, sum1);
                }
                if constexpr (E == kTwo) sum1 = add2(sum1, ex2_2(mul2(d, l2)));
            }
        };
        int v = tid;
        for (; v + 3 * kThreads < nv; v += 4 * kThreads) {
            uint4 u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = xv[v + i * kThreads];
#pragma unroll
            for (int i = 0; i < 4; ++i) add_vec(u[i]);
        }
        for (; v < nv; v += kThreads) add_vec(xv[v]);
        {
            float lo, hi;
            unpack2(sum, lo, hi);
            st.s = lo + hi;
            unpack2(sum1, lo, hi);
            st.s1 = lo + hi;
        }
        if (tid < head) add_one<E>(st, Vc::get(x + tid), a);
        const int tail = head + nv * n + tid;
        if (tail < V) add_one<E>(st, Vc::get(x + tail), a);
        const Stat r = block_stat<E, kThreads>(st, a, sm.warp);
        // (with one exponential and both terms, tau is 1 and the two agree)
        const float lsum = logf(r.s), lsum1 = E == kOne ? lsum : logf(r.s1);
        origin = origin_of(r.m, lsum, lsum1);

        // ---- the loss
        const float llse = logf(ts);
        float kl = 0.f;
        if (!hard_only)
            for (int j = tid; j < K; j += kThreads) {
                const float e = sm.prob[j];
                if (sm.col[j] >= 0 && e != 0.f) {
                    const float lp = (g.values[row * K + j] - tm) * inv_tau - llse;
                    const float lq = (sm.x[j] - r.m) * inv_tau - lsum;
                    kl += e * its * (lp - lq);
                }
            }
        kl = block_sum<kThreads>(kl, sm.red);
        if (tid == 0) {
            float l = (1.f - g.lam) * g.tau * g.tau * kl;
            if (g.lam != 0.f && label >= 0) l += g.lam * (r.m - xlab + lsum1);
            g.loss[row] = w * l;
            if (g.lse) {
                g.lse[2 * row] = r.m * inv_tau + lsum;
                g.lse[2 * row + 1] = E == kOne ? r.m * inv_tau + lsum : r.m + lsum1;
            }
        }
    } else if (lse_is_near(g.lse_in + 2 * row)) {
        origin = origin_of<E>(g.lse_in + 2 * row, hard_only ? 1.f : g.tau, hard_only);
    } else {
        origin = far_origin<T, E, kThreads>(x, V, a, sm.warp);
    }
    if constexpr (!GRAD) return;

    // ---- the gradient: c_t q + c_1 softmax(x), less the teacher's and the label's share
    const float soft = hard_only || !any ? 0.f : coef * (1.f - g.lam) * g.tau;
    const float hard = g.lam != 0.f && label >= 0 ? coef * g.lam : 0.f;
    const Dense<E> dense(soft, hard, origin, a);
    const bool near = Dense<E>::is_near(origin, a);
    Last last{near ? 0.f : origin.at, soft == 0.f ? 0.f : soft * its, hard, xlab, label};
    if (STATS && tid == 0) sm.last = last;
    if (soft == 0.f && hard == 0.f) {   // no term: zero, whatever the logits hold
        __syncthreads();                // in place, every thread has read them
        for (int v = tid; v < V; v += kThreads) Vc::put(out + v, 0.f);
        return;
    }
    // every gather of the row is done before it may be overwritten
    const bool dup = __syncthreads_or(twice), has_label = __syncthreads_or(listed);
    auto grad_vec = [&](const uint4 &u, int v) {
        f2 f[n / 2];
        Vc::unpack(u, f);
#pragma unroll
        for (int i = 0; i < n / 2; ++i) f[i] = dense.two(f[i]);
        T *o = out + head + v * n;
        if (same) {
            __stcs(reinterpret_cast<uint4 *>(o), Vc::pack(f));
        } else {
#pragma unroll
            for (int i = 0; i < n / 2; ++i) {
                float lo, hi;
                unpack2(f[i], lo, hi);
                Vc::put(o + 2 * i, lo);
                Vc::put(o + 2 * i + 1, hi);
            }
        }
    };
    if (near) {
        int v = tid;
        for (; v + 3 * kThreads < nv; v += 4 * kThreads) {
            uint4 u[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = __ldcs(xv + v + i * kThreads);
#pragma unroll
            for (int i = 0; i < 4; ++i) grad_vec(u[i], v + i * kThreads);
        }
        for (; v < nv; v += kThreads) grad_vec(__ldcs(xv + v), v);
        if (tid < head) Vc::put(out + tid, dense.one(Vc::get(x + tid)));
        const int tail = head + nv * n + tid;
        if (tail < V) Vc::put(out + tail, dense.one(Vc::get(x + tail)));
    } else {
        for (int v = tid; v < V; v += kThreads)
            Vc::put(out + v, dense.one(Vc::get(x + v) - last.at));
    }
    __syncthreads();
    // with the loss in the same kernel there are no registers to keep these over the dense pass
    if constexpr (STATS) last = sm.last;
    for (int j = tid; j < K; j += kThreads) {
        const int c = sm.col[j];
        if (c < 0) continue;
        float p = sm.prob[j];
        bool first = true;      // a column listed more than once: its first entry writes it
        if (dup) {
            p = 0.f;
            for (int k = 0; k < K; ++k)
                if (sm.col[k] == c) {
                    if (k < j) first = false;
                    p += sm.prob[k];
                }
        }
        if (first)
            Vc::put(out + c, dense.one(sm.x[j] - last.at) -
                                 (last.share == 0.f ? 0.f : last.share * p) -
                                 (c == last.label ? last.hard : 0.f));
    }
    if (tid == 0 && last.label >= 0 && !has_label)
        Vc::put(out + last.label, dense.one(last.xlab - last.at) - last.hard);
}

kron_status_t bad(kron_status_t st, const char *fmt, double a = 0, double b = 0) {
    char msg[224];
    snprintf(msg, sizeof(msg), fmt, a, b);
    return report_failure(st, msg);
}

// Threads per row: with more than four rows per SM 256, with fewer as many as let all rows run at
// once (515 x 50257 fp32 with its gradient: 58 us with 256 threads, 53 with 384).
template <typename T, int E, bool STATS, bool GRAD>
cudaError_t launch(int64_t N, const Args &g, cudaStream_t st) {
    if (g.V <= kShortV && g.K <= kShortK)
        distill_short_kernel<T, E, STATS, GRAD>
            <<<(unsigned)((N + kShortWarps - 1) / kShortWarps), 32 * kShortWarps, 0, st>>>(g, N);
    else if (N > 4 * kRowParts)
        distill_kernel<T, E, STATS, GRAD, 256><<<(unsigned)N, 256, 0, st>>>(g);
    else if (N > 2 * kRowParts)
        distill_kernel<T, E, STATS, GRAD, 384><<<(unsigned)N, 384, 0, st>>>(g);
    else
        distill_kernel<T, E, STATS, GRAD, 768><<<(unsigned)N, 768, 0, st>>>(g);
    return cudaGetLastError();
}

template <typename T, bool STATS, bool GRAD>
cudaError_t launch_exps(int exps, int64_t N, const Args &g, cudaStream_t st) {
    switch (exps) {
        case kOne: return launch<T, kOne, STATS, GRAD>(N, g, st);
        case kSquare: return launch<T, kSquare, STATS, GRAD>(N, g, st);
        case kFourth: return launch<T, kFourth, STATS, GRAD>(N, g, st);
        default: return launch<T, kTwo, STATS, GRAD>(N, g, st);
    }
}

template <bool STATS, bool GRAD>
kron_status_t run(const Args &g, int64_t N, kron_dtype_t dtype, void *stream) {
    const bool one = g.tau == 1.f || g.lam == 0.f || g.lam == 1.f;
    const int exps = one ? kOne : g.tau == 2.f ? kSquare : g.tau == 4.f ? kFourth : kTwo;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dtype == KRON_BF16
                              ? launch_exps<__nv_bfloat16, STATS, GRAD>(exps, N, g, st)
                              : launch_exps<float, STATS, GRAD>(exps, N, g, st);
    if (e != cudaSuccess) {
        char msg[200];
        snprintf(msg, sizeof(msg), "distillation launch: %s", cudaGetErrorString(e));
        return report_failure(KRON_ERR_CUDA, msg);
    }
    return KRON_OK;
}

// The checks that every entry point shares.
kron_status_t check(const void *logits, int64_t ld, const void *values, const void *indices,
                    int index_bytes, const void *labels, const void *weights, int64_t N, int64_t V,
                    int K, double tau, double lam, kron_dtype_t dtype) {
    report_failure(KRON_OK, "");
    if (dtype != KRON_F32 && dtype != KRON_BF16)
        return bad(KRON_ERR_UNSUPPORTED, "the loss takes KRON_F32 or KRON_BF16 logits (dtype %g)",
                   (double)dtype);
    if (N < 0 || N > 0x7fffffff || V < 1 || V > (1 << 30) || K < 1)
        return bad(KRON_ERR_INVALID_ARG,
                   "sizes must be 0 <= N < 2^31, 1 <= V <= 2^30, K >= 1 (N = %g, V = %g)",
                   (double)N, (double)V);
    if (K > kMaxK)
        return bad(KRON_ERR_UNSUPPORTED, "at most %g teacher logits per row (K = %g)",
                   (double)kMaxK, (double)K);
    if (ld < V) return bad(KRON_ERR_INVALID_ARG, "row stride %g below V = %g", (double)ld, (double)V);
    if (index_bytes != 4 && index_bytes != 8)
        return bad(KRON_ERR_INVALID_ARG, "indices have 4 or 8 bytes (got %g)", index_bytes);
    if (!(tau >= 0.05 && tau <= 1e3))
        return bad(KRON_ERR_INVALID_ARG, "the temperature must be in [0.05, 1e3] (got %g)", tau);
    if (!(lam >= 0.0 && lam <= 1.0))
        return bad(KRON_ERR_INVALID_ARG, "the label weight must be in [0, 1] (got %g)", lam);
    if (lam > 0.0 && !labels && N > 0)
        return bad(KRON_ERR_INVALID_ARG, "labels are needed when their weight is above 0 (%g)", lam);
    if (N > 0 && (!logits || !values || !indices))
        return bad(KRON_ERR_INVALID_ARG, "logits, values and indices must be non-null");
    const uintptr_t e = dtype == KRON_BF16 ? 1 : 3;
    if (((uintptr_t)logits & e) || ((uintptr_t)values & 3) ||
        ((uintptr_t)indices & (uintptr_t)(index_bytes - 1)) || ((uintptr_t)labels & 7) ||
        ((uintptr_t)weights & 3))
        return bad(KRON_ERR_ALIGNMENT, "tensors must be aligned to their element size");
    return KRON_OK;
}

Args args(const void *logits, int64_t ld, const float *values, const void *indices,
          int index_bytes, const int64_t *labels, const float *weights, int64_t V, int K,
          double tau, double lam) {
    Args g{};
    g.logits = logits;
    g.ld = ld;
    g.values = values;
    g.indices = indices;
    g.labels = lam > 0.0 ? labels : nullptr;
    g.weights = weights;
    g.V = (int)V;
    g.K = K;
    g.tau = (float)tau;
    g.lam = (float)lam;
    g.idx64 = index_bytes == 8;
    return g;
}

}  // namespace
}  // namespace kron

using namespace kron;

extern "C" {

kron_status_t kron_distill_forward(const void *logits, int64_t ld, const float *values,
                                   const void *indices, int index_bytes, const int64_t *labels,
                                   const float *weights, float *loss, float *lse, int64_t N,
                                   int64_t V, int K, double temperature, double label_weight,
                                   kron_dtype_t dtype, void *stream) {
    const kron_status_t st = check(logits, ld, values, indices, index_bytes, labels, weights, N, V,
                                   K, temperature, label_weight, dtype);
    if (st != KRON_OK) return st;
    if (N > 0 && !loss) return bad(KRON_ERR_INVALID_ARG, "loss must be non-null");
    if (((uintptr_t)loss | (uintptr_t)lse) & 3)
        return bad(KRON_ERR_ALIGNMENT, "loss and lse must be 4-byte aligned");
    if (N == 0) return KRON_OK;
    Args g = args(logits, ld, values, indices, index_bytes, labels, weights, V, K, temperature,
                  label_weight);
    g.loss = loss;
    g.lse = lse;
    return run<true, false>(g, N, dtype, stream);
}

kron_status_t kron_distill_backward(const void *logits, int64_t ld, const float *values,
                                    const void *indices, int index_bytes, const int64_t *labels,
                                    const float *weights, const float *lse, const float *dloss,
                                    void *dlogits, int64_t ld_out, int64_t N, int64_t V, int K,
                                    double temperature, double label_weight, kron_dtype_t dtype,
                                    void *stream) {
    const kron_status_t st = check(logits, ld, values, indices, index_bytes, labels, weights, N, V,
                                   K, temperature, label_weight, dtype);
    if (st != KRON_OK) return st;
    if (N > 0 && (!lse || !dlogits))
        return bad(KRON_ERR_INVALID_ARG, "lse and dlogits must be non-null");
    if (logits && dlogits == logits && ld_out != ld)
        return bad(KRON_ERR_INVALID_ARG, "in place, both row strides are the same (%g, %g)",
                   (double)ld, (double)ld_out);
    if (ld_out < V)
        return bad(KRON_ERR_INVALID_ARG, "row stride %g of dlogits below V = %g", (double)ld_out,
                   (double)V);
    if ((((uintptr_t)lse | (uintptr_t)dloss) & 3) ||
        ((uintptr_t)dlogits & (dtype == KRON_BF16 ? 1 : 3)))
        return bad(KRON_ERR_ALIGNMENT, "tensors must be aligned to their element size");
    if (N == 0) return KRON_OK;
    Args g = args(logits, ld, values, indices, index_bytes, labels, weights, V, K, temperature,
                  label_weight);
    g.lse_in = lse;
    g.dloss = dloss;
    g.dlogits = dlogits;
    g.ld_out = ld_out;
    return run<false, true>(g, N, dtype, stream);
}

kron_status_t kron_distill_step(const void *logits, int64_t ld, const float *values,
                                const void *indices, int index_bytes, const int64_t *labels,
                                const float *weights, float *loss, void *dlogits, int64_t ld_out,
                                int64_t N, int64_t V, int K, double temperature,
                                double label_weight, kron_dtype_t dtype, void *stream) {
    const kron_status_t st = check(logits, ld, values, indices, index_bytes, labels, weights, N, V,
                                   K, temperature, label_weight, dtype);
    if (st != KRON_OK) return st;
    if (N > 0 && (!loss || !dlogits))
        return bad(KRON_ERR_INVALID_ARG, "loss and dlogits must be non-null");
    if (logits && dlogits == logits && ld_out != ld)
        return bad(KRON_ERR_INVALID_ARG, "in place, both row strides are the same (%g, %g)",
                   (double)ld, (double)ld_out);
    if (ld_out < V)
        return bad(KRON_ERR_INVALID_ARG, "row stride %g of dlogits below V = %g", (double)ld_out,
                   (double)V);
    if (((uintptr_t)loss & 3) || ((uintptr_t)dlogits & (dtype == KRON_BF16 ? 1 : 3)))
        return bad(KRON_ERR_ALIGNMENT, "tensors must be aligned to their element size");
    if (N == 0) return KRON_OK;
    Args g = args(logits, ld, values, indices, index_bytes, labels, weights, V, K, temperature,
                  label_weight);
    g.loss = loss;
    g.dlogits = dlogits;
    g.ld_out = ld_out;
    return run<true, true>(g, N, dtype, stream);
}

}  // extern "C"
