// glu_f32.cu -- the gated Kronecker feed-forward half in exact FP32 (glu.h): both projections, the
// activation and the product in one kernel; for GRAD dg = dH u act'(g) and du = dH act(g).
//
// A CTA takes R rows and KS of the m2 columns k of every block, which need no other columns:
//   stage 1  T[n][(t,k)][a] = sum_j X[(n,a),j] B_t[j,k]       t the 2 G terms of a pass: the same
//   stage 2  Y[n][c,k]     += sum_(i,a) C_i[a,c] T[n][(i,k)][a]   ranks of gate and up
// Every operand lies with the summed index innermost, so that a 16-byte load brings four of its
// values.  Both stages have 8 x 8 outputs per thread: 16 loads (four cycles of shared memory each,
// whatever neighbouring threads share) for 256 multiply-adds.  In stage 2 half a warp takes the
// gate's and half the up projection's; the sums meet in shared memory, for the whole CTA to apply
// the activation to.  Row strides are 4 mod 8 words: neighbouring threads read neighbouring rows,
// on distinct banks.
// 1000 x 1024, r = 2: 28 us (4 x 4 outputs, one word per load, two CTAs of 4 rows per SM: 45;
// packed multiply-adds over pairs of the summed index, 4 x 8 outputs: 28, but 1.6 times the time
// at 20000 rows: one takes 2.3 cycles, two plain ones the same).  FFMA bounds it from below: a
// stage takes 15,500 cycles, 8,200 of FFMA and 7,200 of shared memory, one after the other, as
// the warps load in step; loads one step ahead need more registers than there are (26,000).
#include "glu.h"
#include "internal.h"

namespace kron {
namespace glu {
namespace {

constexpr int kThreads = 512;
constexpr int kMaxSmem = 227 * 1024;
constexpr int kHalf = kThreads / 2;    // stage-2 items

struct FPlan {
    int R, KS, G;              // rows, columns k, and ranks of each projection per pass
    int nks, grid;             // k slices, CTAs per slice
    int Pp, ldx, lda;          // p padded to 4; strides of rows along j and along a
    int64_t tiles;
    int offB, offC, offT, smem;    // words, words, words, bytes
    uint32_t d_x4, d_pp, d_p4, d_m1, d_k4, d_q, d_nt;   // reciprocals of M1/4, Pp, Pp/4, M1, KS/4,
                                                        // Q, NT
};

// e / d by the reciprocal ceil(2^32 / d): exact while e d < 2^32 (e < 2^16 here, as d is, or the
// factors would not fit shared memory); 0 stands for d = 1.
inline uint32_t recip(uint32_t d) { return d == 1 ? 0 : (uint32_t)(((1ull << 32) + d - 1) / d); }
__device__ __forceinline__ int over(int e, uint32_t rc) {
    return rc ? (int)__umulhi((uint32_t)e, rc) : e;
}

inline int up4i(int v) { return (v + 3) & ~3; }
// the next stride that is 4 mod 8
inline int odd4(int v) { return (up4i(v) & 4) ? up4i(v) : up4i(v) + 4; }

__device__ __forceinline__ float4 four(const float *p) {
    return *reinterpret_cast<const float4 *>(p);
}
__device__ __forceinline__ float dot4(const float4 &a, const float4 &b, float c) {
    return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, c))));
}

__device__ __forceinline__ void copy16(float *dst, const float *src, bool live) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src),
                 "r"(live ? 16 : 0) : "memory");       // zeros where nothing is read
}

// MULTI: several passes over the ranks, with the sums of stage 2 kept in between.
template <bool GRAD, bool MULTI>
__global__ void __launch_bounds__(kThreads, 1)
glu_f32_kernel(const float *__restrict__ x, const float *__restrict__ S,
               const float *__restrict__ A, const float *__restrict__ B,
               const float *__restrict__ bias, const float *__restrict__ dH,
               float *__restrict__ out0, float *__restrict__ out1, const Shape s, const FPlan pl,
               const int act) {
    extern __shared__ __align__(16) float smem[];
    float *const Xs = smem, *const Bs = smem + pl.offB, *const Cs = smem + pl.offC;
    float *const Ts = smem + pl.offT;
    const int P = s.p, Q = s.q, M1 = s.m1, M2 = s.m2, R = pl.R, KS = pl.KS, G = pl.G;
    const int Pp = pl.Pp, ldx = pl.ldx, lda = pl.lda;
    const int k0 = blockIdx.y * KS, k4s = KS >> 2, live4 = min(KS, M2 - k0) >> 2;
    const int NC = 2 * G * KS, NT = NC >> 3, MT = (R * Pp + 7) >> 3;   // stage 1: columns, items
    const int CT = (Q + 7) >> 3, K8 = (k4s + 1) >> 1;

    // this thread's stage-2 item: projection h, row n, columns c = tc + u CT, and k in the quads
    // tk and tk + K8 of the slice
    const int h = (threadIdx.x >> 4) & 1, item = (threadIdx.x >> 5) * 16 + (threadIdx.x & 15);
    const int n = item / (CT * K8), tc = item / K8 % CT, tk = item % K8;
    const int tk1 = min(tk + K8, k4s - 1);

    // rows of x, row i = (n, a) at i / 8 + (i mod 8) MT: the eight rows of a stage-1 item are
    // neighbours in T
    auto load_x = [&](int64_t tile) {
        const int64_t n0 = tile * R;
        for (int e = threadIdx.x; e < 8 * MT * (M1 >> 2); e += kThreads) {
            const int row = over(e, pl.d_x4), j = (e - row * (M1 >> 2)) << 2;
            const int rn = over(row, pl.d_pp), a = row - rn * Pp;
            const bool live = a < P && rn < R && n0 + rn < s.N;
            copy16(Xs + ((row >> 3) + (row & 7) * MT) * ldx + j,
                   live ? x + ((n0 + rn) * P + a) * M1 + j : x, live);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    // B and C = S (.) A of gl ranks from i0 on
    auto load_factors = [&](int i0, int gl) {
        // column (proj, i, k) of B at (proj G + i) KS + (k >> 2) + (k & 3) KS/4: stage 2 reads
        // k = 4 tk + v of neighbouring tk
#pragma unroll 4
        for (int e = threadIdx.x; e < 2 * gl * k4s * M1; e += kThreads) {
            const int t = over(e, pl.d_m1), j = e - t * M1, f = over(t, pl.d_k4), kq = t - f * k4s;
            const int pr = f >= gl, i = f - pr * gl;
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            if (kq < live4)
                v = *reinterpret_cast<const float4 *>(
                    B + ((size_t)(pr * s.r + i0 + i) * M1 + j) * M2 + k0 + 4 * kq);
            float *d = Bs + ((pr * G + i) * KS + kq) * ldx + j;
            d[0] = v.x;
            d[k4s * ldx] = v.y;
            d[2 * k4s * ldx] = v.z;
            d[3 * k4s * ldx] = v.w;
        }
        // four a of one c at [proj][i][c][a]
#pragma unroll 2
        for (int e = threadIdx.x; e < 2 * gl * (Pp >> 2) * Q; e += kThreads) {
            const int t = over(e, pl.d_q), c = e - t * Q, f = over(t, pl.d_p4);
            const int a = (t - f * (Pp >> 2)) << 2, pr = f >= gl, i = f - pr * gl;
            const float *ps = S + ((size_t)pr * P + a) * Q + c;
            const float *pa = A + ((size_t)(pr * s.r + i0 + i) * P + a) * Q + c;
            float v[4];
#pragma unroll
            for (int w = 0; w < 4; ++w) v[w] = a + w < P ? ps[w * Q] * pa[w * Q] : 0.f;
            *reinterpret_cast<float4 *>(Cs + ((pr * G + i) * Q + c) * lda + a) =
                make_float4(v[0], v[1], v[2], v[3]);
        }
    };

    load_x(blockIdx.x);
    if (!MULTI) load_factors(0, s.r);
    for (int64_t tile = blockIdx.x; tile < pl.tiles; tile += gridDim.x) {
        const int64_t n0 = tile * R;
        float y[8][8];
        for (int i0 = 0; i0 < s.r; i0 += G) {
            const int gl = MULTI ? min(G, s.r - i0) : s.r;
            if (MULTI) {
                if (i0 || tile != blockIdx.x) __syncthreads();   // the pass before has read its own
                load_factors(i0, gl);
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncthreads();
            for (int t = threadIdx.x; t < MT * NT; t += kThreads) {
                const int tm = over(t, pl.d_nt), tn = t - tm * NT;
                const float *px = Xs + tm * ldx, *pb = Bs + tn * ldx;
                float acc[8][8];
#pragma unroll
                for (int u = 0; u < 8; ++u)
#pragma unroll
                    for (int v = 0; v < 8; ++v) acc[u][v] = 0.f;
#pragma unroll 1
                for (int j = 0; j < M1; j += 4) {
                    float4 xv[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) xv[u] = four(px + u * MT * ldx + j);
#pragma unroll
                    for (int v = 0; v < 8; ++v) {
                        const float4 b = four(pb + v * NT * ldx + j);
#pragma unroll
                        for (int u = 0; u < 8; ++u) acc[u][v] = dot4(xv[u], b, acc[u][v]);
                    }
                }
#pragma unroll
                for (int g = 0; g < 2; ++g) {
                    const int rn = over(tm * 8 + 4 * g, pl.d_pp), a = tm * 8 + 4 * g - rn * Pp;
                    if (rn >= R) break;
                    float *d = Ts + (rn * NC + tn) * lda + a;
                    // zero behind the last a, also where a factor is infinite
                    const bool v1 = a + 1 < P, v2 = a + 2 < P, v3 = a + 3 < P;
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        *reinterpret_cast<float4 *>(d + v * NT * lda) = make_float4(
                            acc[4 * g][v], v1 ? acc[4 * g + 1][v] : 0.f,
                            v2 ? acc[4 * g + 2][v] : 0.f, v3 ? acc[4 * g + 3][v] : 0.f);
                }
            }
            __syncthreads();
            // x has been read: the next tile's comes while stage 2 runs
            if (i0 + G >= s.r && tile + gridDim.x < pl.tiles) load_x(tile + gridDim.x);
            if (!MULTI || i0 == 0)
#pragma unroll
                for (int u = 0; u < 8; ++u)
#pragma unroll
                    for (int v = 0; v < 8; ++v) y[u][v] = 0.f;
            if (n < R) {
                for (int i = 0; i < gl; ++i) {
                    const float *pt = Ts + (n * NC + (h * G + i) * KS + tk) * lda;
                    const float *pc = Cs + ((h * G + i) * Q + tc) * lda;
                    const int second = (tk1 - tk) * lda;
#pragma unroll 1
                    for (int a = 0; a < Pp; a += 4) {
                        float4 tv[8];
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            tv[v] = four(pt + v * k4s * lda + a);
                            tv[v + 4] = four(pt + v * k4s * lda + a + second);
                        }
#pragma unroll
                        for (int u = 0; u < 8; ++u) {
                            // columns behind the last c read what is there, for nothing
                            const float4 c = four(pc + u * CT * lda + a);
#pragma unroll
                            for (int v = 0; v < 8; ++v) y[u][v] = dot4(tv[v], c, y[u][v]);
                        }
                    }
                }
            }
        }
        // Y as [proj][n][c][k], over T
        __syncthreads();
        if (n < R) {
            float *py = Ts + ((h * R + n) * Q + tc) * KS + 4 * tk;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                if (tc + u * CT >= Q) break;
                float *d = py + u * CT * KS;
                *reinterpret_cast<float4 *>(d) = make_float4(y[u][0], y[u][1], y[u][2], y[u][3]);
                *reinterpret_cast<float4 *>(d + 4 * (tk1 - tk)) =
                    make_float4(y[u][4], y[u][5], y[u][6], y[u][7]);
            }
        }
        __syncthreads();
        for (int e = threadIdx.x; e < R * Q * k4s; e += kThreads) {
            const int t = over(e, pl.d_k4), kq = e - t * k4s, rn = over(t, pl.d_q), c = t - rn * Q;
            if (n0 + rn >= s.N || kq >= live4) continue;
            const float4 g4 = four(Ts + 4 * e), u4 = four(Ts + 4 * (R * Q * k4s + e));
            float gs[4] = {g4.x, g4.y, g4.z, g4.w}, us[4] = {u4.x, u4.y, u4.z, u4.w};
            const int col = c * M2 + k0 + 4 * kq;
            const size_t o = (size_t)(n0 + rn) * Q * M2 + col;
            if (bias) {
                const float4 b0 = four(bias + col), b1 = four(bias + (size_t)Q * M2 + col);
                gs[0] += b0.x; gs[1] += b0.y; gs[2] += b0.z; gs[3] += b0.w;
                us[0] += b1.x; us[1] += b1.y; us[2] += b1.z; us[3] += b1.w;
            }
            float d, f;
            if constexpr (GRAD) {
                const float4 dh = four(dH + o);
                const float hv[4] = {dh.x, dh.y, dh.z, dh.w};
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    f = act_f32(act, gs[v], &d);
                    gs[v] = hv[v] * us[v] * d;
                    us[v] = hv[v] * f;
                }
                *reinterpret_cast<float4 *>(out0 + o) = make_float4(gs[0], gs[1], gs[2], gs[3]);
                *reinterpret_cast<float4 *>(out1 + o) = make_float4(us[0], us[1], us[2], us[3]);
            } else {
#pragma unroll
                for (int v = 0; v < 4; ++v) us[v] *= act_f32(act, gs[v], &d);
                *reinterpret_cast<float4 *>(out0 + o) = make_float4(us[0], us[1], us[2], us[3]);
            }
        }
    }
}

int cdiv(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

// The tile by an estimate of the kernel's cycles: a warp's step of either stage is 256 multiply-
// adds and 16 loads on one of the SM's four schedulers, 310 cycles; a pass loads its factors, which
// takes about 700 cycles per four elements and thread, a tile waits for its rows.
bool find_plan(FPlan *best, const Shape &s) {
    double best_cost = 0;
    bool found = false;
    FPlan p{};
    p.Pp = up4i(s.p);
    p.ldx = odd4(s.m1);
    p.lda = odd4(p.Pp);
    for (int parts = 1; parts <= 64 && parts <= s.m2 / 4; ++parts) {
        p.KS = up4i(cdiv(s.m2, parts));
        p.nks = cdiv(s.m2, p.KS);
        if (p.nks != parts || p.nks > 65535) continue;
        const int items_row = (s.q + 7) / 8 * ((p.KS + 7) / 8);
        if (items_row > kHalf) continue;
        for (int R = 1; R <= 16 && R * items_row <= kHalf && R <= s.N; ++R) {
            // as many ranks per pass as fit, in passes of equal length
            const int64_t x = ((int64_t)R * p.Pp + 7) / 8 * 8 * p.ldx;
            const int64_t rank = 2 * ((int64_t)p.KS * p.ldx + (int64_t)s.q * p.lda +
                                      (int64_t)R * p.KS * p.lda);
            const int64_t fit = (kMaxSmem / 4 - x) / rank;
            if (x + rank > kMaxSmem / 4) break;
            const int passes = cdiv(s.r, fit);
            p.R = R;
            p.G = cdiv(s.r, passes);
            const int64_t nc = 2 * (int64_t)p.G * p.KS;
            const int64_t b = nc * p.ldx, c = 2 * (int64_t)p.G * s.q * p.lda;
            const int64_t t = R * nc * p.lda, y = 2 * (int64_t)R * s.q * p.KS;   // Y over T
            if ((x + b + c + (t > y ? t : y)) * 4 > kMaxSmem) continue;
            p.offB = (int)x;
            p.offC = (int)(x + b);
            p.offT = (int)(x + b + c);
            p.smem = (int)((x + b + c + (t > y ? t : y)) * 4);
            p.tiles = (s.N + R - 1) / R;
            const int per = kRowParts / p.nks > 0 ? kRowParts / p.nks : 1;
            p.grid = (int)(p.tiles < per ? p.tiles : per);
            const double waves = (double)cdiv(p.tiles, p.grid) *
                                 cdiv((int64_t)p.nks * p.grid, kRowParts);
            const int w1 = cdiv(((int64_t)R * p.Pp + 7) / 8 * (nc / 8), 128);
            const int w2 = cdiv((int64_t)R * items_row * 2, 128);
            const double s1 = passes * (w1 * s.m1 / 4 * 310.0 + 300);
            const double s2 = s.r * (p.Pp / 4) * w2 * 310.0;
            const double load_f = 1500 + (nc * s.m1 / 4 + p.G * p.Pp * s.q / 2.0) / kThreads * 700;
            const double load_x = 1200;
            const double tile = s1 + s2 + load_x + 600;
            // several passes: the sums of stage 2 leave the registers for stage 1 (2368 x 1024,
            // r = 4: 172 us in two passes over 14 rows, 122 in one over 7)
            const double cost = passes == 1 ? load_f + waves * tile
                                            : waves * (passes * load_f + tile) * 1.4;
            if (!found || cost < best_cost) {
                best_cost = cost;
                p.d_x4 = recip((uint32_t)s.m1 / 4);
                p.d_pp = recip((uint32_t)p.Pp);
                p.d_p4 = recip((uint32_t)p.Pp / 4);
                p.d_m1 = recip((uint32_t)s.m1);
                p.d_k4 = recip((uint32_t)p.KS / 4);
                p.d_q = recip((uint32_t)s.q);
                p.d_nt = recip((uint32_t)(nc / 8));
                *best = p;
                found = true;
            }
        }
    }
    return found;
}

}  // namespace

// A call needs the plan twice: the last one is kept.
static bool f32_plan(FPlan *p, const Shape &s) {
    static thread_local struct { Shape s; FPlan pl; bool known, ok; } kept = {};
    if (!kept.known || kept.s.N != s.N || kept.s.p != s.p || kept.s.q != s.q ||
        kept.s.m1 != s.m1 || kept.s.m2 != s.m2 || kept.s.r != s.r) {
        kept.ok = find_plan(&kept.pl, s);
        kept.s = s;
        kept.known = true;
    }
    *p = kept.pl;
    return kept.ok;
}

bool f32_pre_supported(const Shape &s) {
    FPlan p;
    return f32_plan(&p, s);
}

cudaError_t f32_pre(const void *x, const void *S, const void *A, const void *B, const void *bias,
                    const void *dH, void *out0, void *out1, const Shape &s, int activation,
                    bool grad, cudaStream_t st) {
    FPlan p;
    launch_step() = "gated plan";
    if (!f32_plan(&p, s)) return cudaErrorInvalidConfiguration;
    auto *f = p.G < s.r ? (grad ? glu_f32_kernel<true, true> : glu_f32_kernel<false, true>)
                        : (grad ? glu_f32_kernel<true, false> : glu_f32_kernel<false, false>);
    launch_step() = "shared memory size";
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, p.smem);
    if (e != cudaSuccess) return e;
    launch_step() = "gated launch";
    f<<<dim3((unsigned)p.grid, (unsigned)p.nks), kThreads, p.smem, st>>>(
        (const float *)x, (const float *)S, (const float *)A, (const float *)B,
        (const float *)bias, (const float *)dH, (float *)out0, (float *)out1, s, p, activation);
    return cudaGetLastError();
}

}  // namespace glu
}  // namespace kron
