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
// FFMA bounds it from below, 8,200 cycles per stage for 1000 x 1024, r = 2, and then the loads,
// 7,200: a warp's step takes both in turn unless the next step's loads run while it computes,
// which takes the registers of 256 threads.  That size takes 28 us, with the loads of the factors
// and the packing of rows into tiles (4 x 4 outputs, one word per load, two CTAs of 4 rows per SM:
// 45); 20000 rows 357 us, 30 TFLOP/s (512 threads, no loads ahead: 416).  Packed multiply-adds
// over pairs of the summed index were no faster: one takes 2.3 cycles, two plain ones the same.
#include "glu.h"
#include "internal.h"

namespace kron {
namespace glu {
namespace {

constexpr int kThreads = 256, kBackThreads = 384;
// Also every kernel's limit, whatever the size of a call's tiles: the limit is shared by the host
// threads that call it.
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
struct Operand {
    const float *p;
    int s, t;       // summed index innermost: four rows s apart, the second four t behind them;
};                  // else: s between summed indices, the second four outputs t behind the first

__device__ __forceinline__ float part(const float4 &v, int w) {
    return w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w;
}
__device__ __forceinline__ void rows8(float4 (&v)[8], const Operand &a, int k) {
#pragma unroll
    for (int u = 0; u < 8; ++u) v[u] = four(a.p + (u & 3) * a.s + (u >> 2) * a.t + k);
}

// acc += a b over K values, a multiple of 4; AI, BI: whether the summed index lies innermost;
// AHEAD: whether a step's rows of a are loaded while the one before computes (forward: 3000 rows,
// r = 3, 115 us instead of 141; backward, which lacks the registers: 368 instead of 357).
template <bool AI, bool BI, bool AHEAD>
__device__ __forceinline__ void mm8(float (&acc)[8][8], const Operand &a, const Operand &b, int K) {
    static_assert(AI || !BI, "not needed");
    float4 av[8];
    if constexpr (AI && AHEAD) rows8(av, a, 0);
#pragma unroll 1
    for (int k = 0; k < K; k += 4) {
        float4 next[8];
        if constexpr (AI && !AHEAD) rows8(av, a, k);
        if constexpr (AI && AHEAD) rows8(next, a, min(k + 4, K - 4));
        if constexpr (BI) {
            float4 bv[8];
            rows8(bv, b, k);
#pragma unroll
            for (int v = 0; v < 8; ++v)
#pragma unroll
                for (int w = 0; w < 4; ++w)
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        acc[u][v] = fmaf(part(av[u], w), part(bv[v], w), acc[u][v]);
        } else {
#pragma unroll
            for (int w = 0; w < 4; ++w) {
                const float4 b0 = four(b.p + (k + w) * b.s), b1 = four(b.p + (k + w) * b.s + b.t);
                float4 a0, a1;
                if constexpr (!AI) {
                    a0 = four(a.p + (k + w) * a.s);
                    a1 = four(a.p + (k + w) * a.s + a.t);
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    float f;
                    if constexpr (AI) f = part(av[u], w);
                    else f = u < 4 ? part(a0, u) : part(a1, u - 4);
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        acc[u][v] = fmaf(f, part(b0, v), acc[u][v]);
                        acc[u][v + 4] = fmaf(f, part(b1, v), acc[u][v + 4]);
                    }
                }
            }
        }
        if constexpr (AI && AHEAD) {
#pragma unroll
            for (int u = 0; u < 8; ++u) av[u] = next[u];
        }
    }
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
                mm8<true, true, true>(acc, Operand{px, MT * ldx, 4 * MT * ldx},
                                Operand{pb, NT * ldx, 4 * NT * ldx}, M1);
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
                    // columns behind the last c read what is there, for nothing
                    mm8<true, true, true>(y, Operand{pc, CT * lda, 4 * CT * lda},
                                    Operand{pt, k4s * lda, (tk1 - tk) * lda}, Pp);
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

// ---- backward of both projections ----
//
// A CTA takes a range of rows of one projection, in tiles of R rows, all ranks at once (G = dg or
// du):
//   U[(n,a),(i,k)] = sum_c C_i[a,c] G[(n,c),k]        T[(n,a),(i,k)] = sum_j X[(n,a),j] B_i[j,k]
//   dX[(n,a),j] = sum_(i,k) U B_i[j,k]   dB_i[j,k] += sum_(n,a) X U   dC_i[a,c] += sum_(n,k) T G
// Each tensor lies once in shared memory; 8 x 8 outputs per thread take a step of four summed
// indices by 16 loads of four words whichever way an operand lies.  dB and dC have few outputs and
// a long sum, so `slots` sets of them are summed side by side, each over its rows of the tile, and
// added in order at the end: bitwise reproducible.  777 rows, 512 -> 768, r = 2: 38 us (the
// layer's own kernel, 4 x 4 outputs and one rank at a time: 75); whole backward calls of 1 to 20000
// rows and blocks of 8 to 100 take 0.55 to 1.0 of the time that they took with that kernel.  384
// threads: 3000 rows, r = 3 take 357 us, with 512 370.
struct BPlan {
    int R, slots, parts;
    int64_t rows;                  // per range
    int Pp, Qp, ldx, ldg, ldc, ldt;
    int offG, offB, offC, offU, offT, offS, offD, smem;    // words; smem in bytes
};

// Four sums of a slot: set by the first tile, added to by the others.
__device__ __forceinline__ void add4(float *d, const float *acc, bool first) {
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (!first) v = four(d);
    v.x += acc[0];
    v.y += acc[1];
    v.z += acc[2];
    v.w += acc[3];
    *reinterpret_cast<float4 *>(d) = v;
}

__device__ __forceinline__ int eighth(int n) { return (n + 7) >> 3; }
__device__ __forceinline__ int warps_of(int n) { return (n + 31) & ~31; }

__global__ void __launch_bounds__(kBackThreads, 1)
glu_f32_backward_kernel(const float *__restrict__ x, const float *__restrict__ S,
                        const float *__restrict__ A, const float *__restrict__ B,
                        const float *__restrict__ g0, const float *__restrict__ g1,
                        float *__restrict__ dx0, float *__restrict__ dx1, float *__restrict__ ws,
                        const size_t ws_stride, const Shape s, const BPlan pl) {
    extern __shared__ __align__(16) float smem[];
    float *const Xs = smem, *const Gs = smem + pl.offG, *const Bs = smem + pl.offB;
    float *const Cs = smem + pl.offC, *const Us = smem + pl.offU, *const Ts = smem + pl.offT;
    // slots of [dB][dC as [i][a][Qp]], and dbias
    float *const Ss = smem + pl.offS, *const Ds = smem + pl.offD;
    const int P = s.p, Q = s.q, M1 = s.m1, M2 = s.m2, r = s.r, R = pl.R, rk = r * M2;
    const int Pp = pl.Pp, Qp = pl.Qp, ldx = pl.ldx, ldg = pl.ldg, ldc = pl.ldc, ldt = pl.ldt;
    const int proj = blockIdx.y, n_dc = r * P * Q, n_db = r * M1 * M2;
    const int n_slot = n_db + r * P * Qp;
    S += (size_t)proj * P * Q;
    A += (size_t)proj * n_dc;
    B += (size_t)proj * n_db;
    const float *const G = proj ? g1 : g0;
    float *const dX = proj ? dx1 : dx0;
    float *const out = ws + ((size_t)proj * gridDim.x + blockIdx.x) * ws_stride;
    const int64_t lo = blockIdx.x * pl.rows, hi = lo + pl.rows < s.N ? lo + pl.rows : s.N;

    for (int e = threadIdx.x; e < r * M1 * (M2 >> 2); e += kBackThreads) {    // B as [j][(i,k)]
        const int row = e / (M2 >> 2), k = (e - row * (M2 >> 2)) << 2, i = row / M1;
        copy16(Bs + (row - i * M1) * ldt + i * M2 + k, B + (size_t)row * M2 + k, true);
    }
    for (int e = threadIdx.x; e < r * Pp * Qp; e += kBackThreads) {           // C as [i][a][c]
        const int row = e / Qp, c = e - row * Qp, i = row / Pp, a = row - i * Pp;
        float v = 0.f;
        if (a < P && c < Q) v = S[(size_t)a * Q + c] * A[((size_t)i * P + a) * Q + c];
        Cs[row * ldc + c] = v;
    }
    const int MT = eighth(P), NT = eighth(M2), CT = eighth(Q), JT = eighth(M1);
    const int MR = eighth(R * Pp), nq = M2 >> 2, jq = M1 >> 2;
    const int n_ut = R * r * MT * NT;
    const int n_x = dX ? warps_of(MR * JT) : 0, n_c = warps_of(pl.slots * r * MT * CT);
    const int n_b = warps_of(pl.slots * r * JT * NT);
    for (int64_t n0 = lo; n0 < hi; n0 += R) {
        const bool first = n0 == lo;
        for (int e = threadIdx.x; e < R * Pp * jq; e += kBackThreads) {
            const int row = e / jq, j = (e - row * jq) << 2, n = row / Pp, a = row - n * Pp;
            const bool live = a < P && n0 + n < hi;
            copy16(Xs + row * ldx + j, live ? x + ((n0 + n) * P + a) * M1 + j : x, live);
        }
        for (int e = threadIdx.x; e < R * Qp * nq; e += kBackThreads) {
            const int row = e / nq, k = (e - row * nq) << 2, n = row / Qp, c = row - n * Qp;
            const bool live = c < Q && n0 + n < hi;
            copy16(Gs + row * ldg + k, live ? G + ((n0 + n) * Q + c) * M2 + k : G, live);
        }
        asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
        __syncthreads();
        for (int t = threadIdx.x; t < 2 * n_ut; t += kBackThreads) {
            const bool second = t >= n_ut;           // T
            int e = second ? t - n_ut : t;
            const int tk = e % NT;
            e /= NT;
            const int ta = e % MT;
            e /= MT;
            const int i = e % r, n = e / r;
            Operand oa, ob;
            if (second) {
                oa = Operand{Xs + (n * Pp + ta) * ldx, MT * ldx, 4 * MT * ldx};
                ob = Operand{Bs + i * M2 + 4 * tk, ldt, 4 * NT};
            } else {
                oa = Operand{Cs + (i * Pp + ta) * ldc, MT * ldc, 4 * MT * ldc};
                ob = Operand{Gs + n * Qp * ldg + 4 * tk, ldg, 4 * NT};
            }
            float acc[8][8] = {};
            mm8<true, false, false>(acc, oa, ob, second ? M1 : Qp);
            float *d = (second ? Ts : Us) + n * Pp * ldt + i * M2 + 4 * tk;
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int a = ta + u * MT;
                if (a >= Pp) break;
                const bool live = a < P;       // zero behind the last a, also for infinite factors
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    if (tk + h * NT < nq)
                        *reinterpret_cast<float4 *>(d + a * ldt + 4 * h * NT) =
                            live ? make_float4(acc[u][4 * h], acc[u][4 * h + 1], acc[u][4 * h + 2],
                                               acc[u][4 * h + 3])
                                 : make_float4(0.f, 0.f, 0.f, 0.f);
            }
        }
        __syncthreads();
        for (int t = threadIdx.x; t < n_x + n_c + n_b; t += kBackThreads) {
            float acc[8][8] = {};
            if (t < n_x + n_c) {
                const bool is_x = t < n_x;
                int e = is_x ? t : t - n_x;
                int n = 0, step = R, K = rk, i = 0, ta, tb;
                Operand oa, ob;
                if (is_x) {
                    tb = e % JT;
                    ta = e / JT;
                    if (ta >= MR) continue;
                    oa = Operand{Us + ta * ldt, MR * ldt, 4 * MR * ldt};
                    ob = Operand{Bs + 4 * tb * ldt, ldt, 4 * JT * ldt};
                } else {
                    tb = e % CT;
                    e /= CT;
                    ta = e % MT;
                    e /= MT;
                    i = e % r;
                    n = e / r;
                    if (n >= pl.slots) continue;
                    step = pl.slots;
                    K = M2;
                    oa = Operand{Ts + (n * Pp + ta) * ldt + i * M2, MT * ldt, 4 * MT * ldt};
                    ob = Operand{Gs + (n * Qp + 4 * tb) * ldg, ldg, 4 * CT * ldg};
                }
                const int slot = n;
                for (; n < R; n += step) {
                    mm8<true, true, false>(acc, oa, ob, K);
                    oa.p += step * Pp * ldt;
                    ob.p += step * Qp * ldg;
                }
                if (is_x) {
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int row = ta + u * MR, rn = row / Pp, a = row - rn * Pp;
                        if (rn >= R || a >= P || n0 + rn >= hi) continue;
                        float *d = dX + ((n0 + rn) * P + a) * M1 + 4 * tb;
                        *reinterpret_cast<float4 *>(d) =
                            make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
                        if (tb + JT < jq)
                            *reinterpret_cast<float4 *>(d + 4 * JT) =
                                make_float4(acc[u][4], acc[u][5], acc[u][6], acc[u][7]);
                    }
                } else {
                    float *d = Ss + slot * n_slot + n_db + (i * P + ta) * Qp + 4 * tb;
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        if (ta + u * MT >= P) break;
                        add4(d + u * MT * Qp, &acc[u][0], first);
                        if (4 * (tb + CT) < Qp) add4(d + u * MT * Qp + 4 * CT, &acc[u][4], first);
                    }
                }
            } else {
                int e = t - n_x - n_c;
                const int tk = e % NT;
                e /= NT;
                const int tj = e % JT;
                e /= JT;
                const int i = e % r, slot = e / r;
                if (slot >= pl.slots) continue;
                for (int n = slot; n < R; n += pl.slots)
                    mm8<false, false, false>(
                        acc, Operand{Xs + n * Pp * ldx + 4 * tj, ldx, 4 * JT},
                        Operand{Us + n * Pp * ldt + i * M2 + 4 * tk, ldt, 4 * NT}, Pp);
                float *d = Ss + slot * n_slot + (i * M1 + 4 * tj) * M2 + 4 * tk;
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    if (tj + (u >> 2) * JT >= jq) break;
                    float *du = d + (4 * (u >> 2) * JT + (u & 3)) * M2;
                    add4(du, &acc[u][0], first);
                    if (tk + NT < nq) add4(du + 4 * NT, &acc[u][4], first);
                }
            }
        }
        for (int e = threadIdx.x; e < Q * M2; e += kBackThreads) {
            const int c = e / M2, k = e - c * M2;
            float v = 0.f;
            for (int n = 0; n < R; ++n) v += Gs[(n * Qp + c) * ldg + k];
            Ds[e] = first ? v : Ds[e] + v;
        }
        __syncthreads();
    }
    for (int e = threadIdx.x; e < n_slot; e += kBackThreads) {
        float v = 0.f;
        for (int k = 0; k < pl.slots; ++k) v += Ss[k * n_slot + e];
        const int row = (e - n_db) / Qp, c = e - n_db - row * Qp;
        if (e < n_db) out[n_dc + e] = v;
        else if (c < Q) out[row * Q + c] = v;
    }
    for (int e = threadIdx.x; e < Q * M2; e += kBackThreads) out[n_dc + n_db + e] = Ds[e];
}

// Ranges for one CTA per SM; the largest tile that fits shared memory, then as many slots.  At
// least two rows per tile, or all of the range.
bool backward_plan(BPlan *b, const Shape &s, int max_parts) {
    BPlan p{};
    int parts = kRowParts / 2 < max_parts ? kRowParts / 2 : max_parts;
    p.rows = (s.N + parts - 1) / parts;
    p.parts = cdiv(s.N, p.rows);
    p.Pp = up4i(s.p);
    p.Qp = up4i(s.q);
    p.ldx = odd4(s.m1);
    p.ldg = odd4(s.m2);
    p.ldc = odd4(p.Qp);
    const int64_t rk = (int64_t)s.r * s.m2;
    if (rk > 4096 || s.d_out() > 16384 || s.p > 1024 || (int64_t)s.r * s.p * s.q > 16384 ||
        rk * s.m1 > 16384)
        return false;
    p.ldt = odd4((int)rk);
    const int sums = (int)((int64_t)s.r * s.p * p.Qp + rk * s.m1);
    // the last rows of a tensor are read up to seven rows further
    const int ld = p.ldt > p.ldc ? p.ldt : p.ldc, ld2 = p.ldx > p.ldg ? p.ldx : p.ldg;
    const int tail = 8 * (ld > ld2 ? ld : ld2);
    const int most = (int)(p.rows < 16 ? p.rows : 16);
    for (int R = most; R >= 1 && (R > 1 || p.rows == 1); --R) {
        const int tiles = cdiv(p.rows, R);
        if (cdiv(p.rows, tiles) != R && R != most) continue;       // tiles of equal height
        p.R = R;
        p.offG = R * p.Pp * p.ldx;
        p.offB = p.offG + R * p.Qp * p.ldg;
        p.offC = p.offB + s.m1 * p.ldt;
        p.offU = p.offC + s.r * p.Pp * p.ldc;
        p.offT = p.offU + R * p.Pp * p.ldt;
        p.offS = p.offT + R * p.Pp * p.ldt;
        for (int slots = R; slots >= 1; --slots) {
            p.slots = slots;
            p.offD = p.offS + slots * sums;
            const int64_t words = p.offD + s.d_out() + tail;
            if (words * 4 > kMaxSmem) continue;
            p.smem = (int)words * 4;
            *b = p;
            return true;
        }
    }
    return false;
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
    cudaError_t e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    launch_step() = "gated launch";
    f<<<dim3((unsigned)p.grid, (unsigned)p.nks), kThreads, p.smem, st>>>(
        (const float *)x, (const float *)S, (const float *)A, (const float *)B,
        (const float *)bias, (const float *)dH, (float *)out0, (float *)out1, s, p, activation);
    return cudaGetLastError();
}

cudaError_t f32_backward_pair(const void *x, const void *S, const void *A, const void *B,
                              const void *G0, const void *G1, void *dX0, void *dX1, float *ws,
                              int max_parts, int *parts, const Shape &s, cudaStream_t st) {
    BPlan p;
    // the compiled shape has kernels of its own, faster where rows are many: 2000 rows 335 us here
    // for the whole backward call and 351 there, 2368 rows 384 and 355, 20000 rows 2778 and 2281
    const bool own = s.p == 32 && s.q == 32 && s.m1 == 32 && s.m2 == 32 && s.r == 4 &&
                     s.N >= kCompiledRows;
    if (own || !backward_plan(&p, s, max_parts)) {
        *parts = max_parts;
        return simt_backward_pair(x, S, A, B, G0, G1, dX0, dX1, ws, max_parts, s, st);
    }
    *parts = p.parts;
    launch_step() = "shared memory size";
    cudaError_t e = cudaFuncSetAttribute(glu_f32_backward_kernel,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    launch_step() = "backward launch";
    glu_f32_backward_kernel<<<dim3((unsigned)p.parts, 2), kBackThreads, p.smem, st>>>(
        (const float *)x, (const float *)S, (const float *)A, (const float *)B, (const float *)G0,
        (const float *)G1, (float *)dX0, (float *)dX1, ws, partial_stride(s), s, p);
    return cudaGetLastError();
}

}  // namespace glu
}  // namespace kron
