// glu_wgrad.cu -- factor gradients of the gated Kronecker feed-forward half, BF16.
//
// With dW = x^T d (d = dg or du), block (a, c) of dW the m1 x m2 matrix dW[a,.,c,.]:
//   dC_i[a,c] = sum_(j,k) B_i[j,k] dW[a,j,c,k]     dA_i = dC_i (.) S, dS = sum_i dC_i (.) A_i
//   dB_i[j,k] = sum_(a,c) C_i[a,c] dW[a,j,c,k]     dbias = column sums of d
// dW is formed densely by one tcgen05 product over the rows (both operands as they lie in
// memory, MN-major), then contracted with the factors in fp32.  The vec trick's own order (T = X B
// against d, C d against X) takes 2 r (1/q + 1/m1) of dW's multiply-adds, and T and C d of every
// row through registers and shared memory; dW is a plain product at the tensor cores' rate.  That
// ratio is 1/2 for 1024 x 1024, 32 x 32 blocks and r = 4, but 1/16 for 4096 x 4096, 64 x 64 blocks
// and r = 1: wide layers of low rank pay for dW, as no kernel here takes the other order above
// eight rows (backward of 16384 rows of 4096: 1135 us for r = 1, 2017 for r = 8).  The workspace
// holds dW of both projections in fp32 (134 MB at 4096 x 4096).
// Rows are split into ranges whose dW are added in order: bitwise reproducible.
// 20000 rows, 1024 x 1024: dW 72 us, 1.2 PFLOP/s on 128 of the 148 SMs (76% of the tensor pipe's
// cycles on them), the contraction 19 us, a read of 34 MB from L2 and HBM.  1021 rows, 768 x 2048:
// 20 and 18 us, both short of work for the SMs: 16 steps of 64 rows, and the latency of its loads.
#include "glu.h"
#include "tc_gen_common.cuh"

#include <cuda_bf16.h>

namespace kron {
namespace glu {

using namespace tc;
using namespace tc::gen;

namespace {

// ---- dW = x^T [dg | du]: tiles of 256 x 256 (two M = 128 accumulators, all of TMEM), K = 64
// rows per stage.  A stage brings 64 KB for 1024 cycles of MMA; with 128 x 256 tiles it was
// 48 KB for 512, and the reads from L2 (96 B per cycle and SM) took twice the MMAs' time.
constexpr int kTM = 256, kTN = 256, kTK = 64, kStages = 3;
constexpr int kABytes = kTM * kTK * 2, kBBytes = kTN * kTK * 2, kStageBytes = kABytes + kBBytes;
constexpr int kBoxBytes = 64 * kTK * 2;        // one TMA box: 64 columns x 64 rows
constexpr int kDwThreads = 320;                // TMA, MMA, eight epilogue warps (four also sum
                                               // the columns of d)
constexpr size_t kDwSmem = (size_t)kStages * kStageBytes + 1024 + 256;

struct DwArgs {
    float *part;
    size_t part_floats;
    int64_t N, rows_per_split;
    int din, dout, mt, nt;       // tiles along din, and along dout of one projection
    int tm;                      // rows of dW per tile: 256, or 128 where the tiles are few
    int sums;                    // whether the column sums are wanted
    const __nv_bfloat16 *S, *A;
    float *ct;                   // C_i[f] as [proj][f = (a, c)][rp], for the contraction
    int pq, r, rp;
    int *device_error;
};

enum { kFull = 0, kEmpty = kStages, kDone = 2 * kStages, kDwBars = 2 * kStages + 1 };

__global__ void __launch_bounds__(kDwThreads, 1)
glu_dw_kernel(const __grid_constant__ CUtensorMap mx, const __grid_constant__ CUtensorMap mg,
              const __grid_constant__ CUtensorMap mu, const DwArgs g) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw), base = (raw + 1023u) & ~1023u;
    const uint32_t tail = base + kStages * kStageBytes;
    uint8_t *tail_ptr = smem_raw + (tail - raw);
    auto bar = [&](int i) { return tail + 8u * i; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail_ptr + kDwBars * 8);
    const Abort ab{reinterpret_cast<volatile int *>(tail_ptr + kDwBars * 8 + 8), g.device_error};
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    const int tiles = g.mt * g.nt * 2;
    const int split = blockIdx.x / tiles, tile = blockIdx.x % tiles;
    const int m0 = (tile % g.mt) * g.tm, proj = tile / (g.mt * g.nt);
    const int n0 = (tile / g.mt) % g.nt * kTN;
    const int64_t r0 = split * g.rows_per_split;
    const int64_t r1 = min(g.N, r0 + g.rows_per_split);
    const int steps = (int)((r1 - r0 + kTK - 1) / kTK);
    const bool sums = g.sums && m0 == 0;
    // whether the tile's lower half has rows of dW
    const bool second = g.tm == kTM && m0 + 128 < g.din;
    const int a_boxes = second ? 4 : 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(bar(kFull + s), 1);
            mbar_init(bar(kEmpty + s), sums ? 5 : 1);
        }
        mbar_init(bar(kDone), 1);
        *ab.flag = 0;
        mbar_init_fence();
        prefetch_tmap(&mx);
        prefetch_tmap(proj ? &mu : &mg);
    }
    if (warp == 1) tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)), 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool done = true;

    if (warp == 0) {
        if (lane == 0) {
            int u = 0;
            for (; u < steps; ++u) {
                const int s = u % kStages;
                if (!mbar_wait(bar(kEmpty + s), ((u / kStages) & 1) ^ 1, ab)) break;
                const uint32_t a = base + s * kStageBytes, b = a + kABytes;
                const int row = (int)(r0 + (int64_t)u * kTK);
                mbar_arrive_expect_tx(bar(kFull + s), kBBytes + a_boxes * kBoxBytes);
                for (int i = 0; i < a_boxes; ++i)
                    tma_load_2d(a + i * kBoxBytes, &mx, m0 + i * 64, row, bar(kFull + s));
                for (int i = 0; i < kTN / 64; ++i)
                    tma_load_2d(b + i * kBoxBytes, proj ? &mu : &mg, n0 + i * 64, row,
                                bar(kFull + s));
            }
            for (int v = u > kStages ? u - kStages : 0; v < u; ++v)
                mbar_wait_drain(bar(kFull + v % kStages), (v / kStages) & 1);
        }
    } else if (warp == 1) {
        // both operands MN-major (bits 15 and 16): K runs down the rows of a box
        constexpr uint32_t idesc = idesc_f32acc(128, kTN, 1) | (1u << 15) | kBMajorMN;
        for (int u = 0; u < steps; ++u) {
            const int s = u % kStages;
            if (!warp_wait(bar(kFull + s), (u / kStages) & 1, ab)) break;
            tc_fence_after();
            if (elect_one()) {
                const uint32_t a = base + s * kStageBytes;
                const uint64_t ad = sdesc_mn(a, layout_type(128), kBoxBytes, 1024);
                const uint64_t bd = sdesc_mn(a + kABytes, layout_type(128), kBoxBytes, 1024);
#pragma unroll
                for (int kk = 0; kk < kTK / 16; ++kk)
                    mma_ss<false>(tmem, desc_add(ad, kk * 2048), desc_add(bd, kk * 2048), idesc,
                                  (u > 0 || kk > 0) ? 1u : 0u);
                if (second)
#pragma unroll
                    for (int kk = 0; kk < kTK / 16; ++kk)
                        mma_ss<false>(tmem + 256, desc_add(ad, 2 * kBoxBytes + kk * 2048),
                                      desc_add(bd, kk * 2048), idesc,
                                      (u > 0 || kk > 0) ? 1u : 0u);
                mma_commit(bar(kEmpty + s));
            }
            __syncwarp();
        }
        if (elect_one()) mma_commit(bar(kDone));
        __syncwarp();
        if (lane == 0) mbar_wait_drain(bar(kDone), 0);
        __syncwarp();
    } else {
        const int quad = warp & 3, t = (warp - 2) * 32 + lane;
        float *part = g.part + (size_t)split * g.part_floats;
        const int half = (warp - 2) >> 2;
        if (half == 1) {      // meanwhile: the factors side by side for the contraction
            for (int e = blockIdx.x * 128 + t - 128; e < 2 * g.pq; e += gridDim.x * 128) {
                const int proj2 = e >= g.pq, f = e - proj2 * g.pq;
                const float sv = __bfloat162float(g.S[e]);
                for (int i = 0; i < g.rp; ++i)
                    g.ct[(size_t)e * g.rp + i] =
                        i < g.r
                            ? sv * __bfloat162float(g.A[((size_t)proj2 * g.r + i) * g.pq + f])
                            : 0.f;
            }
        }
        if (sums && half == 0) {
            // columns 2t and 2t + 1 of the d tile, rows in order
            float s0 = 0.f, s1 = 0.f;
            const int col = 2 * t, box = col / 64, inb = (col % 64) * 2;
            bool ok = true;
            for (int u = 0; u < steps; ++u) {
                const int s = u % kStages;
                if (!warp_wait(bar(kFull + s), (u / kStages) & 1, ab)) {
                    ok = false;
                    break;
                }
                const uint32_t b = base + s * kStageBytes + kABytes + box * kBoxBytes;
#pragma unroll 16
                for (int r = 0; r < kTK; ++r) {
                    uint32_t w;
                    asm volatile("ld.shared.b32 %0, [%1];"
                                 : "=r"(w)
                                 : "r"(b + swz((uint32_t)(r * 128 + inb), 128))
                                 : "memory");
                    s0 += __uint_as_float(w << 16);
                    s1 += __uint_as_float(w & 0xFFFF0000u);
                }
                mbar_arrive_warp(bar(kEmpty + s));
            }
            if (ok) {
                float *dst = part + (size_t)2 * g.din * g.dout + (size_t)proj * g.dout + n0 + col;
                if (n0 + col < g.dout) dst[0] = s0;
                if (n0 + col + 1 < g.dout) dst[1] = s1;
            }
        }
        done = warp_wait(bar(kDone), 0, ab);
        tc_fence_after();
        if (done) {
            // the halves of the warps take the two accumulators, or every second column group
            const int acc = second ? half : 0, step = second ? 1 : 2;
            const int row = m0 + acc * 128 + quad * 32 + lane;
            float *dst = part + ((size_t)proj * g.din + row) * g.dout + n0;
            for (int cg = second ? 0 : half; cg < kTN / 32; cg += step) {
                if (n0 + cg * 32 >= g.dout) break;
                uint32_t v[32];
                tmem_load32(tmem + ((uint32_t)(quad * 32) << 16) + acc * 256 + cg * 32, v);
                if (row < g.din) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        if (n0 + cg * 32 + i < g.dout)
                            *reinterpret_cast<uint4 *>(dst + cg * 32 + i) =
                                make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                }
                __syncwarp();
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

// ---- contraction with the factors ----
// dW is read as float4 along k, twice (second time from L2): once with a block per few (a, c)
// for dC, once with a block per eight (j, k) for dB; a third kind of block adds dbias.
constexpr int kCt = 256;      // threads
constexpr int kW = 2;         // places of dW read at a time
constexpr int kJs = 4;        // parts of j (dC)

struct CtArgs {
    const float *part;
    size_t part_floats;
    int splits;
    const __nv_bfloat16 *S, *A, *B;
    __nv_bfloat16 *dS, *dA, *dB, *dbias;
    const float *sums;           // column sums of d, first split: [2][dout]
    const float *ct;             // the factors as the first kernel left them
    int rp;
    int p, q, m1, m2, r, dout;
    int tk, cpb;                 // threads along k (m2 / 4), columns c per block (dC)
    int dc_blocks, db_blocks;    // blocks of the first two kinds
};

// dW at W places, the splits added in order: 2 W loads in flight.
template <int W>
__device__ __forceinline__ void dw4(const CtArgs &g, const size_t (&o)[W], float4 (&v)[W]) {
    auto add = [](float4 &x, const float4 &y) {
        x.x += y.x;
        x.y += y.y;
        x.z += y.z;
        x.w += y.w;
    };
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const float *p = g.part;
    int s = 0;
    for (; s + 1 < g.splits; s += 2, p += 2 * g.part_floats) {
        float4 x[W], y[W];
#pragma unroll
        for (int i = 0; i < W; ++i) {
            x[i] = __ldg(reinterpret_cast<const float4 *>(p + o[i]));
            y[i] = __ldg(reinterpret_cast<const float4 *>(p + g.part_floats + o[i]));
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
            add(v[i], x[i]);
            add(v[i], y[i]);
        }
    }
    if (s < g.splits) {
        float4 x[W];
#pragma unroll
        for (int i = 0; i < W; ++i) x[i] = __ldg(reinterpret_cast<const float4 *>(p + o[i]));
#pragma unroll
        for (int i = 0; i < W; ++i) add(v[i], x[i]);
    }
}

// dC, dA, dS: a block per (projection, a, cpb columns c); a thread has four k of one c and a
// quarter of the j, and the threads of one c are added in order.
template <int kRc>   // ranks summed at a time
__device__ void dc_role(const CtArgs &g) {
    __shared__ float acc_s[kRc][kCt];
    const int ncb = cdiv(g.q, g.cpb), blk = blockIdx.x;
    const int c0 = blk % ncb * g.cpb, a = blk / ncb % g.p, proj = blk / ncb / g.p;
    const int kk = threadIdx.x % g.tk, rest = threadIdx.x / g.tk;
    const int cl = rest % g.cpb, js = rest / g.cpb;
    const bool live = js < kJs && c0 + cl < g.q;
    const int per_j = cdiv(g.m1, kJs), j0 = js * per_j, j1 = min(g.m1, j0 + per_j);
    const size_t o0 = ((size_t)proj * g.p + a) * g.m1 * g.dout + (size_t)(c0 + cl) * g.m2 + 4 * kk;
    const size_t mm = (size_t)g.m1 * g.m2, pq = (size_t)g.p * g.q;
    float ds = 0.f;
    for (int i0 = 0; i0 < g.r; i0 += kRc) {
        const int ni = min(kRc, g.r - i0);
        float acc[kRc] = {};
        if (live) {
            const __nv_bfloat16 *Bi = g.B + ((size_t)proj * g.r + i0) * mm + 4 * kk;
            for (int j = j0; j < j1; j += kW) {
                size_t o[kW];
                float4 v[kW];
#pragma unroll
                for (int t = 0; t < kW; ++t) o[t] = o0 + (size_t)min(j + t, j1 - 1) * g.dout;
                dw4(g, o, v);
#pragma unroll
                for (int t = 0; t < kW; ++t)
                    if (j + t < j1)
#pragma unroll
                        for (int i = 0; i < kRc; ++i)
                            if (i < ni) {
                                const uint2 w = __ldg(reinterpret_cast<const uint2 *>(
                                    Bi + i * mm + (size_t)(j + t) * g.m2));
                                acc[i] = fmaf(v[t].x, __uint_as_float(w.x << 16), acc[i]);
                                acc[i] = fmaf(v[t].y, __uint_as_float(w.x & 0xFFFF0000u), acc[i]);
                                acc[i] = fmaf(v[t].z, __uint_as_float(w.y << 16), acc[i]);
                                acc[i] = fmaf(v[t].w, __uint_as_float(w.y & 0xFFFF0000u), acc[i]);
                            }
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRc; ++i) acc_s[i][threadIdx.x] = acc[i];
        __syncthreads();
        // thread (i, c): the sum of its c's threads in order, into the first of them
        for (int e = threadIdx.x; e < ni * g.cpb; e += kCt) {
            const int i = e / g.cpb, c = e % g.cpb;
            float v = 0.f;
            for (int u = 0; u < kJs; ++u)
                for (int t = 0; t < g.tk; ++t) v += acc_s[i][(u * g.cpb + c) * g.tk + t];
            acc_s[i][c * g.tk] = v;
            if (c0 + c < g.q) {
                const size_t pos = (size_t)a * g.q + c0 + c;
                g.dA[((size_t)proj * g.r + i0 + i) * pq + pos] =
                    __float2bfloat16_rn(v * __bfloat162float(g.S[proj * pq + pos]));
            }
        }
        __syncthreads();
        if (threadIdx.x < g.cpb && c0 + (int)threadIdx.x < g.q) {
            float af[kRc];
#pragma unroll
            for (int i = 0; i < kRc; ++i)
                af[i] = i < ni ? __bfloat162float(g.A[((size_t)proj * g.r + i0 + i) * pq +
                                                      (size_t)a * g.q + c0 + threadIdx.x])
                               : 0.f;
#pragma unroll
            for (int i = 0; i < kRc; ++i)
                if (i < ni) ds = fmaf(acc_s[i][threadIdx.x * g.tk], af[i], ds);
        }
    }
    if (threadIdx.x < g.cpb && c0 + (int)threadIdx.x < g.q)
        g.dS[proj * pq + (size_t)a * g.q + c0 + threadIdx.x] = __float2bfloat16_rn(ds);
}

// dB: a block per (projection, ranks, kDbE float4 of (j, k)); kCt / kDbE threads share a float4, each
// with a range of the (a, c), and their sums are added in order.
template <int kRc, int kDbE>
__device__ void db_role(const CtArgs &g, int blk) {
    constexpr int kDbR = kCt / kDbE;
    __shared__ float red[kDbR][kDbE * kRc * 4 + 1];
    const int n4 = g.m1 * g.tk, eb = cdiv(n4, kDbE), ib = cdiv(g.r, kRc);
    const int el = threadIdx.x % kDbE, range = threadIdx.x / kDbE;
    const int e0 = blk % eb * kDbE, e = e0 + el;
    blk /= eb;
    const int i0 = blk % ib * kRc, proj = blk / ib;
    const int ni = min(kRc, g.r - i0), pq = g.p * g.q;
    const size_t mm = (size_t)g.m1 * g.m2;
    const int f0 = (int)((int64_t)pq * range / kDbR), f1 = (int)((int64_t)pq * (range + 1) / kDbR);
    float acc[kRc][4] = {};
    if (e < n4) {
        const int j = e / g.tk, k = 4 * (e - j * g.tk);
        int a = f0 / g.q, c = f0 - a * g.q;
        const size_t o0 = ((size_t)proj * g.p * g.m1 + j) * g.dout + k;
        const float *ct = g.ct + (size_t)proj * pq * g.rp + i0;
        for (int f = f0; f < f1; f += kW) {
            size_t o[kW];
            float4 v[kW], x[kW][kRc / 4];
#pragma unroll
            for (int t = 0; t < kW; ++t) {
                o[t] = o0 + (size_t)a * g.m1 * g.dout + (size_t)c * g.m2;
                const int ft = min(f + t, f1 - 1);
#pragma unroll
                for (int u = 0; u < kRc / 4; ++u)
                    x[t][u] = f + t < f1 ? __ldg(reinterpret_cast<const float4 *>(
                                               ct + (size_t)ft * g.rp + 4 * u))
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
                if (f + t + 1 < f1 && ++c == g.q) c = 0, ++a;
            }
            dw4(g, o, v);
#pragma unroll
            for (int t = 0; t < kW; ++t)
#pragma unroll
                for (int i = 0; i < kRc; ++i) {
                    const float4 &xi = x[t][i / 4];
                    const float w = i % 4 == 0 ? xi.x : i % 4 == 1 ? xi.y : i % 4 == 2 ? xi.z : xi.w;
                    acc[i][0] = fmaf(v[t].x, w, acc[i][0]);
                    acc[i][1] = fmaf(v[t].y, w, acc[i][1]);
                    acc[i][2] = fmaf(v[t].z, w, acc[i][2]);
                    acc[i][3] = fmaf(v[t].w, w, acc[i][3]);
                }
        }
    }
#pragma unroll
    for (int i = 0; i < kRc; ++i)
#pragma unroll
        for (int t = 0; t < 4; ++t) red[range][(i * kDbE + el) * 4 + t] = acc[i][t];
    __syncthreads();
    // a float4 of (j, k) is four neighbours of dB
    for (int u = threadIdx.x; u < ni * kDbE * 4; u += kCt) {
        const int i = u / (kDbE * 4), w = u % (kDbE * 4);
        if (e0 * 4 + w >= n4 * 4) continue;
        float v = 0.f;
#pragma unroll 8
        for (int s = 0; s < kDbR; ++s) v += red[s][u];
        g.dB[((size_t)proj * g.r + i0 + i) * mm + (size_t)e0 * 4 + w] = __float2bfloat16_rn(v);
    }
}

// dbias: the splits' column sums added in order.
__device__ void bias_role(const CtArgs &g, int blk) {
    const size_t e = (size_t)blk * kCt + threadIdx.x;
    if (e >= (size_t)2 * g.dout) return;
    float v = 0.f;
#pragma unroll 4
    for (int s = 0; s < g.splits; ++s) v += g.sums[(size_t)s * g.part_floats + e];
    g.dbias[e] = __float2bfloat16_rn(v);
}

template <int kRc, int kDbE>
__global__ void __launch_bounds__(kCt, kRc == 4 ? 4 : 3) glu_contract_kernel(const CtArgs g) {
    const int blk = blockIdx.x;
    if (blk < g.dc_blocks) dc_role<kRc>(g);
    else if (blk < g.dc_blocks + g.db_blocks) db_role<kRc, kDbE>(g, blk - g.dc_blocks);
    else bias_role(g, blk - g.dc_blocks - g.db_blocks);
}

// ---- few rows: the vec trick's own order, without dW ----
// dC_i[a,c] = sum_(n,k) T_i[n,a,k] d[n,c,k] with T = X B, dB_i[j,k] = sum_(n,a) X[n,a,j] U_i[n,a,k]
// with U = C d, in fp32 on the CUDA cores, and nothing of dW's size is written or read.  Whole
// backward calls, through dW and this way: 1 row of 4096 x 4096, r = 8: 324 and 61 us; 8 rows 328
// and 135; 1 row of 2784 x 3192, r = 2: 123 and 53; 8 rows of 1024 x 1024, r = 4: 57 and 52; 8
// rows of 1024 x 1280, r = 8: 65 and 59.  At 32 rows dW was faster for all of them.
constexpr int kSmallRows = 8;
constexpr int kSmallSmem = 100 * 1024;      // two blocks per SM

struct SmArgs {
    const __nv_bfloat16 *x, *d[2], *S, *A, *B;
    __nv_bfloat16 *dS, *dA, *dB, *dbias;
    int N, p, q, m1, m2, r;
    int dc_blocks, db_blocks;
};

size_t small_smem(int N, int p, int m1, int m2, int r) {
    const size_t dc = (size_t)N * ((size_t)r * m2 + m1), db = (size_t)N * p * 8;
    return 4 * (dc > db ? dc : db);
}

// A block per (projection, a): T of this a for every term in shared memory, then a warp per c.
__device__ void small_dc(const SmArgs &g, float *smem) {
    const int a = blockIdx.x % g.p, proj = blockIdx.x / g.p, Nk = g.N * g.m2;
    const int din = g.p * g.m1, dout = g.q * g.m2, pq = g.p * g.q, mm = g.m1 * g.m2;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    float *T = smem, *X = smem + g.r * Nk;
    for (int e = threadIdx.x; e < g.N * g.m1; e += kCt) {
        const int n = e / g.m1, j = e - n * g.m1;
        X[e] = __bfloat162float(g.x[(size_t)n * din + a * g.m1 + j]);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < g.r * Nk; e += kCt) {
        const int i = e / Nk, rest = e - i * Nk, n = rest / g.m2, k = rest - n * g.m2;
        const __nv_bfloat16 *b = g.B + ((size_t)proj * g.r + i) * mm + k;
        float v = 0.f;
#pragma unroll 8
        for (int j = 0; j < g.m1; ++j)
            v = fmaf(X[n * g.m1 + j], __bfloat162float(b[(size_t)j * g.m2]), v);
        T[e] = v;
    }
    __syncthreads();
    for (int c = warp; c < g.q; c += kCt / 32) {
        const __nv_bfloat16 *d = g.d[proj] + c * g.m2;
        const size_t pos = (size_t)proj * pq + a * g.q + c;
        const float sv = __bfloat162float(g.S[pos]);
        float ds = 0.f;
        for (int i0 = 0; i0 < g.r; i0 += 4) {
            float acc[4] = {};
            for (int e = 2 * lane; e < Nk; e += 64) {
                const int n = e / g.m2, k = e - n * g.m2;
                const uint32_t w =
                    *reinterpret_cast<const uint32_t *>(d + (size_t)n * dout + k);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (i0 + i < g.r) {
                        const float2 t = *reinterpret_cast<const float2 *>(T + (i0 + i) * Nk + e);
                        acc[i] = fmaf(t.x, __uint_as_float(w << 16), acc[i]);
                        acc[i] = fmaf(t.y, __uint_as_float(w & 0xFFFF0000u), acc[i]);
                    }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i0 + i < g.r) {
                    for (int o = 16; o; o >>= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
                    const size_t ai = ((size_t)proj * g.r + i0 + i) * pq + a * g.q + c;
                    if (lane == 0) g.dA[ai] = __float2bfloat16_rn(acc[i] * sv);
                    ds = fmaf(acc[i], __bfloat162float(g.A[ai]), ds);
                }
        }
        if (lane == 0) g.dS[pos] = __float2bfloat16_rn(ds);
    }
}

// A block per (projection, term, eight k): U of these k in shared memory, then a thread per (j, k).
__device__ void small_db(const SmArgs &g, int blk, float *U) {
    const int k8 = g.m2 / 8, k0 = blk % k8 * 8, f = blk / k8, proj = f / g.r;   // f: flat term
    const int din = g.p * g.m1, dout = g.q * g.m2, pq = g.p * g.q;
    const __nv_bfloat16 *S = g.S + (size_t)proj * pq, *A = g.A + (size_t)f * pq;
    for (int e = threadIdx.x; e < g.N * g.p; e += kCt) {
        const int n = e / g.p, a = e - n * g.p;
        const __nv_bfloat16 *d = g.d[proj] + (size_t)n * dout + k0;
        float acc[8] = {};
#pragma unroll 4
        for (int c = 0; c < g.q; ++c) {
            const float w =
                __bfloat162float(S[a * g.q + c]) * __bfloat162float(A[a * g.q + c]);
            const uint4 v = *reinterpret_cast<const uint4 *>(d + (size_t)c * g.m2);
            const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                acc[2 * t] = fmaf(w, __uint_as_float(u[t] << 16), acc[2 * t]);
                acc[2 * t + 1] = fmaf(w, __uint_as_float(u[t] & 0xFFFF0000u), acc[2 * t + 1]);
            }
        }
#pragma unroll
        for (int t = 0; t < 8; ++t) U[e * 8 + t] = acc[t];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < g.m1 * 8; e += kCt) {
        const int j = e >> 3, t = e & 7;
        float v = 0.f;
        for (int n = 0; n < g.N; ++n) {
            const __nv_bfloat16 *x = g.x + (size_t)n * din + j;
#pragma unroll 8
            for (int a = 0; a < g.p; ++a)
                v = fmaf(__bfloat162float(x[a * g.m1]), U[(n * g.p + a) * 8 + t], v);
        }
        g.dB[((size_t)f * g.m1 + j) * g.m2 + k0 + t] = __float2bfloat16_rn(v);
    }
}

__global__ void __launch_bounds__(kCt) glu_small_grad_kernel(const SmArgs g) {
    extern __shared__ __align__(16) float small_mem[];
    const int blk = blockIdx.x;
    if (blk < g.dc_blocks) {
        small_dc(g, small_mem);
    } else if (blk < g.dc_blocks + g.db_blocks) {
        small_db(g, blk - g.dc_blocks, small_mem);
    } else {
        const int dout = g.q * g.m2, e = (blk - g.dc_blocks - g.db_blocks) * kCt + threadIdx.x;
        if (e >= 2 * dout) return;
        const __nv_bfloat16 *d = e < dout ? g.d[0] + e : g.d[1] + e - dout;
        float v = 0.f;
        for (int n = 0; n < g.N; ++n) v += __bfloat162float(d[(size_t)n * dout]);
        g.dbias[e] = __float2bfloat16_rn(v);
    }
}

size_t pad64(size_t n) { return (n + 63) & ~(size_t)63; }

}  // namespace

static int ranks_at_a_time(int r) { return r <= 4 ? 4 : 8; }

WgradPlan wgrad_plan(const Shape &s, int sms) {
    WgradPlan pl{};
    // few rows take the direct kernel, as long as its tiles fit two blocks of shared memory per SM
    if (s.N <= kSmallRows && small_smem((int)s.N, s.p, s.m1, s.m2, s.r) <= kSmallSmem) {
        pl.direct = 1;
        return pl;
    }
    const int din = (int)s.d_in(), dout = (int)s.d_out();
    const int64_t tiles = (int64_t)cdiv(din, kTM) * 2 * cdiv(dout, kTN);
    int64_t splits = sms / tiles;
    // a range costs a write and two reads of dW: at least 16 stages of rows for it
    const int64_t most = (s.N + 1023) / 1024;
    if (splits > most) splits = most;
    if (splits < 1) splits = 1;
    pl.rows_per_split = ((s.N + splits - 1) / splits + kTK - 1) / kTK * kTK;
    if (pl.rows_per_split < kTK) pl.rows_per_split = kTK;
    pl.splits = (int)((s.N + pl.rows_per_split - 1) / pl.rows_per_split);
    if (pl.splits < 1) pl.splits = 1;
    pl.tm = 2 * tiles * pl.splits <= sms ? 128 : kTM;
    pl.part_floats = pad64((size_t)2 * din * dout + 2 * (size_t)dout);
    pl.ws_bytes = 4 * (pl.part_floats * pl.splits +
                       pad64((size_t)2 * s.p * s.q * up(s.r, ranks_at_a_time(s.r))));
    return pl;
}

cudaError_t wgrad_run(const WgradPlan &pl, const void *x, const void *dg, const void *du,
                      const void *S, const void *A, const void *B, void *dS, void *dA, void *dB,
                      void *dbias, void *ws, const Shape &s, cudaStream_t st) {
    const int din = (int)s.d_in(), dout = (int)s.d_out();
    cudaError_t e;
    if (pl.direct) {
        SmArgs m{};
        m.x = static_cast<const __nv_bfloat16 *>(x);
        m.d[0] = static_cast<const __nv_bfloat16 *>(dg);
        m.d[1] = static_cast<const __nv_bfloat16 *>(du);
        m.S = static_cast<const __nv_bfloat16 *>(S);
        m.A = static_cast<const __nv_bfloat16 *>(A);
        m.B = static_cast<const __nv_bfloat16 *>(B);
        m.dS = static_cast<__nv_bfloat16 *>(dS);
        m.dA = static_cast<__nv_bfloat16 *>(dA);
        m.dB = static_cast<__nv_bfloat16 *>(dB);
        m.dbias = static_cast<__nv_bfloat16 *>(dbias);
        m.N = (int)s.N;
        m.p = s.p;
        m.q = s.q;
        m.m1 = s.m1;
        m.m2 = s.m2;
        m.r = s.r;
        m.dc_blocks = 2 * s.p;
        m.db_blocks = 2 * s.r * (s.m2 / 8);
        const size_t smem = small_smem(m.N, s.p, s.m1, s.m2, s.r);
        launch_step() = "shared memory size";
        e = cudaFuncSetAttribute(glu_small_grad_kernel,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallSmem);
        if (e != cudaSuccess) return e;
        launch_step() = "factor-gradient launch";
        const int blocks = m.dc_blocks + m.db_blocks + (dbias ? cdiv(2 * dout, kCt) : 0);
        glu_small_grad_kernel<<<(unsigned)blocks, kCt, smem, st>>>(m);
        return cudaGetLastError();
    }
    CUtensorMap mx, mg, mu;
    launch_step() = "tensor map";
    e = make_tmap_2d(&mx, x, true, s.N, din, 64, kTK, 128, false);
    if (e == cudaSuccess) e = make_tmap_2d(&mg, dg, true, s.N, dout, 64, kTK, 128, false);
    if (e == cudaSuccess) e = make_tmap_2d(&mu, du, true, s.N, dout, 64, kTK, 128, false);
    if (e != cudaSuccess) return e;
    DwArgs g{};
    g.part = static_cast<float *>(ws);
    g.part_floats = pl.part_floats;
    g.N = s.N;
    g.rows_per_split = pl.rows_per_split;
    g.din = din;
    g.dout = dout;
    g.tm = pl.tm;
    g.mt = cdiv(din, pl.tm);
    g.nt = cdiv(dout, kTN);
    g.sums = dbias != nullptr;
    g.S = static_cast<const __nv_bfloat16 *>(S);
    g.A = static_cast<const __nv_bfloat16 *>(A);
    g.ct = g.part + pl.part_floats * pl.splits;
    g.pq = s.p * s.q;
    g.r = s.r;
    g.rp = up(s.r, ranks_at_a_time(s.r));
    launch_step() = "device error word";
    g.device_error = device_error_ptr();
    if (!g.device_error) return cudaErrorInvalidSymbol;
    launch_step() = "shared memory size";
    e = cudaFuncSetAttribute(glu_dw_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)kDwSmem);
    if (e != cudaSuccess) return e;
    launch_step() = "weight-gradient launch";
    const int64_t grid = (int64_t)g.mt * g.nt * 2 * pl.splits;
    glu_dw_kernel<<<(unsigned)grid, kDwThreads, kDwSmem, st>>>(mx, mg, mu, g);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    CtArgs c{};
    c.part = g.part;
    c.part_floats = pl.part_floats;
    c.splits = pl.splits;
    c.S = static_cast<const __nv_bfloat16 *>(S);
    c.A = static_cast<const __nv_bfloat16 *>(A);
    c.B = static_cast<const __nv_bfloat16 *>(B);
    c.dS = static_cast<__nv_bfloat16 *>(dS);
    c.dA = static_cast<__nv_bfloat16 *>(dA);
    c.dB = static_cast<__nv_bfloat16 *>(dB);
    c.dbias = static_cast<__nv_bfloat16 *>(dbias);
    c.sums = g.part + (size_t)2 * din * dout;
    c.ct = g.ct;
    c.rp = g.rp;
    c.p = s.p;
    c.q = s.q;
    c.m1 = s.m1;
    c.m2 = s.m2;
    c.r = s.r;
    c.dout = dout;
    c.tk = s.m2 / 4;
    c.cpb = kCt / (c.tk * kJs);
    if (c.cpb < 1) return cudaErrorInvalidValue;       // m2 <= 256: checked by the entry points
    if (c.cpb > s.q) c.cpb = s.q;
    c.dc_blocks = 2 * s.p * cdiv(s.q, c.cpb);
    // dB: eight float4 per block where that still makes blocks for every SM, else two (32-byte
    // reads of dW, four times the blocks): 1024 x 1024, r = 4 takes 20 us with two and 34 with eight
    const int rc = ranks_at_a_time(s.r), n4 = s.m1 * s.m2 / 4, per = 2 * cdiv(s.r, rc);
    const bool wide = per * cdiv(n4, 8) >= kRowParts;
    c.db_blocks = per * cdiv(n4, wide ? 8 : 2);
    const int blocks = c.dc_blocks + c.db_blocks + (dbias ? cdiv(2 * dout, kCt) : 0);
    launch_step() = "factor-gradient launch";
    auto *f = rc == 4 ? (wide ? glu_contract_kernel<4, 8> : glu_contract_kernel<4, 2>)
                      : (wide ? glu_contract_kernel<8, 8> : glu_contract_kernel<8, 2>);
    f<<<(unsigned)blocks, kCt, 0, st>>>(c);
    return cudaGetLastError();
}

}  // namespace glu
}  // namespace kron
