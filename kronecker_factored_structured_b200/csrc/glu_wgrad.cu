// glu_wgrad.cu -- factor gradients of the gated Kronecker feed-forward half, BF16.
//
// With dW = x^T d (d = dg or du), block (a, c) of dW the m1 x m2 matrix dW[a,.,c,.]:
//   dC_i[a,c] = sum_(j,k) B_i[j,k] dW[a,j,c,k]     dA_i = dC_i (.) S, dS = sum_i dC_i (.) A_i
//   dB_i[j,k] = sum_(a,c) C_i[a,c] dW[a,j,c,k]     dbias = column sums of d
// dW is formed densely by one tcgen05 product over the rows (both operands as they lie in
// memory, MN-major), then contracted with the factors in fp32.  For the vec trick's own order
// (T = X B against d, C d against X) the row sums take r (1/q + 1/m1) of dW's multiply-adds,
// twice, but T and C d of every row have to go through registers and shared memory, which is
// what bounds those kernels; dW is a plain product that runs at the tensor cores' rate.
// Rows are split into ranges whose dW are added in order: bitwise reproducible.
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
    const bool second = g.tm == kTM && m0 + 128 < g.din;      // whether the tile's lower half has rows of dW
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
// for dC, once with a thread per four (j, k) for dB.
constexpr int kCt = 256;      // threads
constexpr int kW = 2;         // places of dW read at a time
constexpr int kJs = 4;        // parts of j (dC)

struct CtArgs {
    const float *part;
    size_t part_floats;
    int splits;
    const __nv_bfloat16 *S, *A, *B;
    __nv_bfloat16 *dS, *dA;
    float *dbp;                  // [dbs][2][r][m1][m2]
    int p, q, m1, m2, r, dout, dbs;
    int tk, cpb;                 // threads along k (m2 / 4), columns c per block (dC)
    int dc_blocks;               // blocks of the first role
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

// dB partial sums: a thread per four (j, k), a block per (projection, range of (a, c), ranks)
template <int kRc>
__device__ void db_role(const CtArgs &g, int blk) {
    __shared__ float cs[kRc][64];      // C_i of up to 64 (a, c)
    const int n4 = g.m1 * g.tk, eb = cdiv(n4, kCt), ib = cdiv(g.r, kRc);
    const int e = blk % eb * kCt + threadIdx.x;
    blk /= eb;
    const int i0 = (blk % ib) * kRc;
    blk /= ib;
    const int range = blk % g.dbs, proj = blk / g.dbs;
    const int ni = min(kRc, g.r - i0), pq = g.p * g.q;
    const int f0 = (int)((int64_t)pq * range / g.dbs), f1 = (int)((int64_t)pq * (range + 1) / g.dbs);
    const bool live = e < n4;
    const int j = live ? e / g.tk : 0, k = live ? 4 * (e - j * g.tk) : 0;
    float acc[kRc][4] = {};
    for (int f = f0; f < f1; f += 64) {
        const int nf = min(64, f1 - f);
        __syncthreads();
        for (int u = threadIdx.x; u < kRc * 64; u += kCt) {
            const int i = u >> 6, w = u & 63;
            cs[i][w] = i < ni && w < nf
                           ? __bfloat162float(g.S[(size_t)proj * pq + f + w]) *
                                 __bfloat162float(g.A[((size_t)proj * g.r + i0 + i) * pq + f + w])
                           : 0.f;
        }
        __syncthreads();
        if (live) {
            int a = f / g.q, c = f - a * g.q;
            const size_t o0 = ((size_t)proj * g.p * g.m1 + j) * g.dout + k;
            for (int w = 0; w < nf; w += kW) {
                size_t o[kW];
                float4 v[kW];
#pragma unroll
                for (int t = 0; t < kW; ++t) {
                    o[t] = o0 + (size_t)a * g.m1 * g.dout + (size_t)c * g.m2;
                    if (w + t + 1 < nf && ++c == g.q) c = 0, ++a;
                }
                dw4(g, o, v);
#pragma unroll
                for (int t = 0; t < kW; ++t)
                    if (w + t < nf)
#pragma unroll
                        for (int i = 0; i < kRc; ++i) {
                            const float x = cs[i][w + t];
                            acc[i][0] = fmaf(v[t].x, x, acc[i][0]);
                            acc[i][1] = fmaf(v[t].y, x, acc[i][1]);
                            acc[i][2] = fmaf(v[t].z, x, acc[i][2]);
                            acc[i][3] = fmaf(v[t].w, x, acc[i][3]);
                        }
            }
        }
    }
    if (live)
#pragma unroll
        for (int i = 0; i < kRc; ++i)
            if (i < ni)
                *reinterpret_cast<float4 *>(
                    g.dbp + (((size_t)range * 2 + proj) * g.r + i0 + i) * g.m1 * g.m2 +
                    (size_t)j * g.m2 + k) =
                    make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
}

template <int kRc>
__global__ void __launch_bounds__(kCt, 4) glu_contract_kernel(const CtArgs g) {
    if ((int)blockIdx.x < g.dc_blocks) dc_role<kRc>(g);
    else db_role<kRc>(g, blockIdx.x - g.dc_blocks);
}

// dB and dbias: the ranges and splits, eight threads per value, each adding every eighth in
// order, then their sums in order.
__global__ void __launch_bounds__(kCt)
glu_finish_kernel(const float *dbp, int dbs, size_t nb, __nv_bfloat16 *dB, const float *sums,
                  size_t part_floats, int splits, size_t nbias, __nv_bfloat16 *dbias) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, part = threadIdx.x >> 5;
    const size_t e = (size_t)blockIdx.x * 32 + lane;
    float v = 0.f;
    if (e < nb) {
#pragma unroll 4
        for (int s = part; s < dbs; s += 8) v += dbp[(size_t)s * nb + e];
    } else if (e - nb < nbias) {
        for (int s = part; s < splits; s += 8) v += sums[(size_t)s * part_floats + e - nb];
    }
    red[part][lane] = v;
    __syncthreads();
    if (part == 0 && e < nb + nbias) {
        v = 0.f;
#pragma unroll
        for (int t = 0; t < 8; ++t) v += red[t][lane];
        if (e < nb) dB[e] = __float2bfloat16_rn(v);
        else dbias[e - nb] = __float2bfloat16_rn(v);
    }
}

size_t pad64(size_t n) { return (n + 63) & ~(size_t)63; }

}  // namespace

static int ranks_at_a_time(int r) { return r <= 4 ? 4 : 8; }

WgradPlan wgrad_plan(const Shape &s, int sms) {
    WgradPlan pl{};
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
    // dB: ranges of (a, c) for about four blocks per SM, at most 128 (their sums are added again)
    const int64_t per = (int64_t)cdiv(s.m1 * s.m2 / 4, kCt) * cdiv(s.r, ranks_at_a_time(s.r)) * 2;
    int64_t dbs = (4 * sms + per - 1) / per;
    if (dbs > 128) dbs = 128;
    if (dbs > (int64_t)s.p * s.q) dbs = (int64_t)s.p * s.q;
    pl.dbs = (int)dbs;
    pl.ws_bytes = 4 * (pl.part_floats * pl.splits +
                       pad64((size_t)pl.dbs * 2 * s.r * s.m1 * s.m2));
    return pl;
}

cudaError_t wgrad_run(const WgradPlan &pl, const void *x, const void *dg, const void *du,
                      const void *S, const void *A, const void *B, void *dS, void *dA, void *dB,
                      void *dbias, void *ws, const Shape &s, cudaStream_t st) {
    const int din = (int)s.d_in(), dout = (int)s.d_out();
    CUtensorMap mx, mg, mu;
    launch_step() = "tensor map";
    cudaError_t e = make_tmap_2d(&mx, x, true, s.N, din, 64, kTK, 128, false);
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
    c.dbp = g.part + pl.part_floats * pl.splits;
    c.p = s.p;
    c.q = s.q;
    c.m1 = s.m1;
    c.m2 = s.m2;
    c.r = s.r;
    c.dout = dout;
    c.dbs = pl.dbs;
    c.tk = s.m2 / 4;
    c.cpb = kCt / (c.tk * kJs);
    if (c.cpb < 1) return cudaErrorInvalidValue;       // m2 <= 256: checked by the entry points
    if (c.cpb > s.q) c.cpb = s.q;
    c.dc_blocks = 2 * s.p * cdiv(s.q, c.cpb);
    const int db_blocks = cdiv(s.m1 * s.m2 / 4, kCt) * cdiv(s.r, ranks_at_a_time(s.r)) * pl.dbs * 2;
    launch_step() = "factor-gradient launch";
    if (ranks_at_a_time(s.r) == 4)
        glu_contract_kernel<4><<<(unsigned)(c.dc_blocks + db_blocks), kCt, 0, st>>>(c);
    else
        glu_contract_kernel<8><<<(unsigned)(c.dc_blocks + db_blocks), kCt, 0, st>>>(c);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const size_t nb = (size_t)2 * s.r * s.m1 * s.m2, nbias = dbias ? (size_t)2 * dout : 0;
    launch_step() = "final sums launch";
    glu_finish_kernel<<<(unsigned)((nb + nbias + 31) / 32), kCt, 0, st>>>(
        c.dbp, pl.dbs, nb, static_cast<__nv_bfloat16 *>(dB),
        g.part + (size_t)2 * din * dout, pl.part_floats, pl.splits, nbias,
        static_cast<__nv_bfloat16 *>(dbias));
    return cudaGetLastError();
}

}  // namespace glu
}  // namespace kron
