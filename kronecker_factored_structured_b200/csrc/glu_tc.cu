// glu_tc.cu -- the gated Kronecker feed-forward half on the sm_100a tensor cores, BF16: both
// projections, the activation and the product in one kernel (forward), the gradients of both
// pre-activations from one recompute (kPre), and dX as the sum over both projections (kInput).
//
// Every projection is the vec trick Y_n = sum_i C_i^T (X_n B_i), C_i = S (.) A_i, in two
// chained products per tile of NT rows of x; the sizes are run-time values, only the padded
// width MP of a k slice is compiled (16, 32, 64 or 128 columns k of B_i):
//   stage 1 (chunk)  T[(i,k),(n,a)] = sum_j B_i[j,k] X_n[a,j]   M = 128 lanes: RB = 128/MP ranks i
//                                                              x MP columns k; N = NT x AC <= 128
//   stage 2          Y[(n,k),c]   += sum_(i,a) T[(n,k),(i,a)] C_i[a,c]   M = 128: NT = RB rows n
//                                                              x MP; K = RB x AC <= 128
// The 2r ranks of gate and up are one list: a chunk's K steps of gate ranks go to one
// accumulator and those of up ranks to another, so that x is read once for both.  Epilogue 1
// (8 warps) moves a chunk TMEM -> bf16 -> shared memory, which is the permute of the vec trick;
// epilogue 2 (8 warps) has g and u of one (n, k, c) side by side.  For kInput the kernel runs
// with transposed factors, dg against the gate's and du against the up's ranks, all into one
// accumulator.  T is rounded to BF16 between the stages, as in the layer's own kernels: half
// a step, 2^-8 of each term.
//
// A CTA holds the factors of one (k slice, c slice) in shared memory for its life and streams
// row tiles; slices exist where the factors do not fit at once, and for few rows, where the
// set-up of the factors is what takes the time.  Stage 1 is repeated for each c slice.
// Bound by shared memory: per chunk 32 KB of T stored and 32 KB read back, 512 of about 770
// cycles at 128 B/clk for the 32 x 32 blocks, against 256 cycles of MMA.
#include "glu.h"
#include "tc_gen_common.cuh"

#include <cuda_bf16.h>
#include <cudaTypedefs.h>

namespace kron {
namespace tc {
PFN_cuTensorMapEncodeTiled_v12000 get_encode();
}

namespace glu {

using namespace tc;
using namespace tc::gen;

namespace {

constexpr int kThreads = 608;          // TMA, two MMA issuers, 8 + 8 epilogue warps
constexpr int kMaxStages = 6;
constexpr int kTailBytes = 512;        // barriers, TMEM address, abort flag
constexpr int kSmemMax = 232448 - 1024 - kTailBytes;
constexpr int kTmD1 = 0, kTmY = 256;   // TMEM columns: two D1 buffers of 128, then Y

struct KArgs {
    Plan pl;
    const __nv_bfloat16 *S, *A, *B, *bias, *dH;
    __nv_bfloat16 *out0, *out1;
    int64_t N;
    int sBi, sBo, sCa, sCc;    // strides of B along (in, out) and of C along (a, c)
    int pq, mm;                // elements of one S or A_i, and of one B_i
    int out_ld;
    int *device_error;
};

// Barriers, in 8-byte words from the tail's start.
enum { kXFull = 0, kXEmpty = kMaxStages, kD1Full = 2 * kMaxStages, kD1Empty = kD1Full + 2,
       kTFull = kD1Empty + 2, kTEmpty = kTFull + 2, kYFull = kTEmpty + 2, kYEmpty = kYFull + 2,
       kDrain = kYEmpty + 2, kBars = kDrain + 2 };
static_assert(kBars * 8 + 16 <= kTailBytes, "tail");

template <int ACT, bool PRE>
__device__ __forceinline__ void gated(float g, float u, float dh, float &o0, float &o1) {
    if constexpr (PRE) {
        float d;
        const float f = act_fast<ACT>(g, &d);
        o0 = dh * u * d;
        o1 = dh * f;
    } else {
        o0 = act_fast<ACT>(g, nullptr) * u;
    }
}

// 16 columns of one epilogue-2 group.
template <bool PRE>
__device__ __forceinline__ void gate16(int act, const uint32_t (&g)[16], const uint32_t (&u)[16],
                                       const float (&bg)[16], const float (&bu)[16],
                                       const float (&dh)[16], float (&o0)[16], float (&o1)[16]) {
#define KRON_GATE(ACT)                                                                        \
    _Pragma("unroll") for (int t = 0; t < 16; ++t)                                            \
        gated<ACT, PRE>(__uint_as_float(g[t]) + bg[t], __uint_as_float(u[t]) + bu[t], dh[t],  \
                        o0[t], o1[t])
    switch (act) {
        case KRON_ACT_SILU: KRON_GATE(KRON_ACT_SILU); break;
        case KRON_ACT_GELU: KRON_GATE(KRON_ACT_GELU); break;
        case KRON_ACT_GELU_TANH: KRON_GATE(KRON_ACT_GELU_TANH); break;
        default: KRON_GATE(KRON_ACT_SIGMOID); break;
    }
#undef KRON_GATE
}

template <int MP, int MODE>
__global__ void __launch_bounds__(kThreads, 1)
glu_tc_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
              const __grid_constant__ KArgs g, int act) {
    constexpr int RB = 128 / MP, NT = RB;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    const Plan &pl = g.pl;
    const uint32_t sB = base, sC = base + pl.off_c, sT = base + pl.off_t, sX = base + pl.off_x;
    const uint32_t tail = base + pl.smem;
    uint8_t *tail_ptr = smem_raw + (tail - raw);
    auto bar = [&](int i) { return tail + 8u * i; };
    volatile uint32_t *tmem_slot = reinterpret_cast<volatile uint32_t *>(tail_ptr + kBars * 8);
    const Abort ab{reinterpret_cast<volatile int *>(tail_ptr + kBars * 8 + 8), g.device_error};

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nslices = pl.nqs * pl.nks;
    const int slice = blockIdx.x % nslices, group = blockIdx.x / nslices;
    const int k0 = (slice / pl.nqs) * MP, c0 = (slice % pl.nqs) * pl.qc;
    const int N1 = NT * pl.AC;
    const int nchunks = pl.nac * pl.nblk;      // stage-1 / stage-2 chunks of a tile

    // flat rank of block `b` of source `src`, position il (-1: none): rank i of gate is i, of
    // up r + i, the order of A and B in memory
    auto flat_rank = [&](int b, int il) {
        const int src = b / pl.nblk_src, i = (b % pl.nblk_src) * RB + il;
        return i < pl.ranks ? src * pl.ranks + i : -1;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < pl.stages; ++s) {
            mbar_init(bar(kXFull + s), 1);
            mbar_init(bar(kXEmpty + s), 1);
        }
        for (int d = 0; d < 2; ++d) {
            mbar_init(bar(kD1Full + d), 1);
            mbar_init(bar(kD1Empty + d), 8);
            mbar_init(bar(kTFull + d), 8);
            mbar_init(bar(kTEmpty + d), 1);
            mbar_init(bar(kYFull + d), 1);
            mbar_init(bar(kYEmpty + d), 8);
            mbar_init(bar(kDrain + d), 1);
        }
        *ab.flag = 0;
        mbar_init_fence();
        prefetch_tmap(&map0);
        if (pl.nsrc > 1) prefetch_tmap(&map1);
    }
    if (warp == 1) tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)), 512);

    // stage-1 A operand: row L = (il, k) of block b holds B_i[., k0 + k], zero past the sizes
    {
        const int nk8 = pl.kb / 16;
        for (int e = threadIdx.x; e < pl.nblk * nk8 * 128; e += kThreads) {
            const int L = e & 127, rest = e >> 7, j8 = (rest % nk8) * 8, b = rest / nk8;
            const int F = flat_rank(b, L / MP), k = k0 + L % MP;
            uint32_t w[4] = {0, 0, 0, 0};
            if (F >= 0 && k < pl.M2) {
                const __nv_bfloat16 *src = g.B + (size_t)F * g.mm + (size_t)k * g.sBo;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const int j = j8 + 2 * t;
                    const uint32_t lo =
                        j < pl.M1 ? __bfloat16_as_ushort(src[(size_t)j * g.sBi]) : 0u;
                    const uint32_t hi =
                        j + 1 < pl.M1 ? __bfloat16_as_ushort(src[(size_t)(j + 1) * g.sBi]) : 0u;
                    w[t] = lo | (hi << 16);
                }
            }
            st_shared_v4(sB + b * 128 * pl.kb + kmaj(L, j8 * 2, 128, pl.sw), w[0], w[1], w[2],
                         w[3]);
        }
    }
    // stage-2 B operand of chunk (ac, b): row c, K position il*AC + a: C_i[ac*AC + a][c0 + c]
    {
        const int na8 = pl.AC / 8;
        const int per = pl.rbl * na8 * pl.qcp;
        for (int e = threadIdx.x; e < nchunks * per; e += kThreads) {
            const int ch = e / per, rem = e % per;
            const int c = rem % pl.qcp, kk = rem / pl.qcp, a8 = (kk % na8) * 8, il = kk / na8;
            const int ac = ch / pl.nblk, b = ch % pl.nblk;
            const int F = flat_rank(b, il);
            float v[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const int a = ac * pl.AC + a8 + t;
                v[t] = 0.f;
                if (F >= 0 && c < pl.qc && c0 + c < pl.Q && a < pl.P) {
                    const size_t o = (size_t)a * g.sCa + (size_t)(c0 + c) * g.sCc;
                    v[t] = __bfloat162float(g.S[(size_t)(F / pl.r) * g.pq + o]) *
                           __bfloat162float(g.A[(size_t)F * g.pq + o]);
                }
            }
            st_shared_v4(sC + ch * pl.c_chunk + kmaj(c, (il * pl.AC + a8) * 2, pl.qcp, 128),
                         pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                         pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
        }
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    const int x_chunks = pl.nsrc * pl.nac;     // ring items of a tile

    if (warp == 0) {
        // ---------------- TMA producer: x chunk (source, ac) of NT rows ----------------
        if (lane == 0) {
            int u = 0;
            bool ok = true;
            for (int t = group; t < pl.ntiles && ok; t += pl.groups) {
                for (int xc = 0; xc < x_chunks; ++xc, ++u) {
                    const int s = u % pl.stages;
                    if (!mbar_wait(bar(kXEmpty + s), ((u / pl.stages) & 1) ^ 1, ab)) {
                        ok = false;
                        break;
                    }
                    const CUtensorMap *map = xc < pl.nac ? &map0 : &map1;
                    mbar_arrive_expect_tx(bar(kXFull + s), N1 * pl.kb);
                    for (int kc = 0; kc < pl.kch; ++kc)
                        asm volatile(
                            "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::"
                            "complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                                sX + s * pl.x_bytes + kc * N1 * pl.sw),
                            "l"(reinterpret_cast<uint64_t>(map)), "r"(kc * (pl.sw / 2)),
                            "r"((xc % pl.nac) * pl.AC), "r"(t * NT), "r"(bar(kXFull + s))
                            : "memory");
                }
            }
            for (int v = u > pl.stages ? u - pl.stages : 0; v < u; ++v)
                mbar_wait_drain(bar(kXFull + v % pl.stages), (v / pl.stages) & 1);
        }
    } else if (warp == 1) {
        // ---------------- stage 1 ----------------
        const uint32_t idesc = idesc_f32acc(128, N1, 1);
        const int ksteps = (pl.M1 + 15) / 16;
        int u = 0, v = 0;
        bool ok = true;
        for (int t = group; t < pl.ntiles && ok; t += pl.groups) {
            for (int xc = 0; xc < x_chunks && ok; ++xc, ++u) {
                const int s = u % pl.stages, src = xc / pl.nac;
                if (!warp_wait(bar(kXFull + s), (u / pl.stages) & 1, ab)) {
                    ok = false;
                    break;
                }
                const uint64_t bd0 = sdesc_kmajor(sX + s * pl.x_bytes, pl.sw);
                for (int b = 0; b < pl.nblk_src; ++b, ++v) {
                    const int d1 = v & 1;
                    if (!warp_wait(bar(kD1Empty + d1), ((v >> 1) & 1) ^ 1, ab)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint64_t ad0 =
                            sdesc_kmajor(sB + (src * pl.nblk_src + b) * 128 * pl.kb, pl.sw);
                        for (int kk = 0; kk < ksteps; ++kk) {
                            const int kb = kk * 32, ch = kb / pl.sw, in = kb % pl.sw;
                            mma_ss<false>(tmem + kTmD1 + d1 * 128,
                                          desc_add(ad0, ch * 128 * pl.sw + in),
                                          desc_add(bd0, ch * N1 * pl.sw + in), idesc, kk > 0);
                        }
                        mma_commit(bar(kD1Full + d1));
                        if (b == pl.nblk_src - 1) mma_commit(bar(kXEmpty + s));
                    }
                    __syncwarp();
                }
            }
        }
        if (elect_one()) mma_commit(bar(kDrain + 0));
        __syncwarp();
        if (lane == 0) mbar_wait_drain(bar(kDrain + 0), 0);
        __syncwarp();
    } else if (warp == 2) {
        // ---------------- stage 2 ----------------
        const uint32_t idesc = idesc_f32acc(128, pl.qcp, 1);
        int v = 0, ti = 0;
        bool ok = true;
        for (int t = group; t < pl.ntiles && ok; t += pl.groups, ++ti) {
            const int y = ti % pl.ybufs;
            if (!warp_wait(bar(kYEmpty + y), ((ti / pl.ybufs) & 1) ^ 1, ab)) break;
            const uint32_t yb = tmem + kTmY + y * pl.nacc * pl.qcp;
            uint32_t acc0 = 0, acc1 = 0;      // whether an accumulator holds something
            for (int xc = 0; xc < x_chunks && ok; ++xc) {
                const int src = xc / pl.nac, ac = xc % pl.nac;
                for (int bs = 0; bs < pl.nblk_src; ++bs, ++v) {
                    const int tb = v & 1, b = src * pl.nblk_src + bs;
                    if (!warp_wait(bar(kTFull + tb), (v >> 1) & 1, ab)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const int live = min(RB, pl.ranks - bs * RB);
                    const int steps = live * pl.AC / 16;
                    // K steps below `split` belong to gate ranks
                    const int split =
                        MODE == kInput ? steps
                                       : min(live, max(0, pl.r - bs * RB)) * pl.AC / 16;
                    if (elect_one()) {
                        const uint64_t ad0 = sdesc_kmajor(sT + tb * pl.t_bytes, 128);
                        const uint64_t bd0 =
                            sdesc_kmajor(sC + (ac * pl.nblk + b) * pl.c_chunk, 128);
                        for (int ks = 0; ks < steps; ++ks) {
                            const int ch = ks >> 2, in = (ks & 3) * 32;
                            const bool up = ks >= split;
                            mma_ss<false>(up ? yb + pl.qcp : yb,
                                          desc_add(ad0, ch * 128 * 128 + in),
                                          desc_add(bd0, ch * pl.qcp * 128 + in), idesc,
                                          up ? (acc1 | (uint32_t)(ks > split))
                                             : (acc0 | (uint32_t)(ks > 0)));
                        }
                        mma_commit(bar(kTEmpty + tb));
                        if (xc == x_chunks - 1 && bs == pl.nblk_src - 1)
                            mma_commit(bar(kYFull + y));
                    }
                    __syncwarp();
                    if (split > 0) acc0 = 1;
                    if (split < steps) acc1 = 1;
                }
            }
        }
        if (elect_one()) mma_commit(bar(kDrain + 1));
        __syncwarp();
        if (lane == 0) mbar_wait_drain(bar(kDrain + 1), 0);
        __syncwarp();
    } else if (warp < 11) {
        // ---------------- epilogue 1: D1 -> T ----------------
        const int quad = warp & 3, wi = (warp - 3) >> 2;
        const int L = quad * 32 + lane, il = L / MP, k = L % MP;
        const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
        // byte offsets in T of this lane's stores: columns (n, a..a+7) go to row (n, k), K
        // position il*AC + a; the warp takes the 32-column groups wi and wi + 2
        uint32_t soff[2][4];
#pragma unroll
        for (int gi = 0; gi < 2; ++gi)
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const int f = (wi + 2 * gi) * 32 + t * 8, n = f / pl.AC, a = f % pl.AC;
                soff[gi][t] =
                    f < N1 ? kmaj(n * MP + k, (il * pl.AC + a) * 2, 128, 128) : 0xFFFFFFFFu;
            }
        int v = 0;
        bool ok = true;
        for (int t = group; t < pl.ntiles && ok; t += pl.groups) {
            for (int ch = 0; ch < nchunks; ++ch, ++v) {
                const int d = v & 1, bs = ch % pl.nblk_src;
                if (!warp_wait(bar(kD1Full + d), (v >> 1) & 1, ab) ||
                    !warp_wait(bar(kTEmpty + d), ((v >> 1) & 1) ^ 1, ab)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                // a warp's lanes hold one rank, or two (MP = 16): live is per lane
                const bool live = bs * RB + il < pl.ranks;
                if (__any_sync(0xffffffffu, live)) {
#pragma unroll
                    for (int gi = 0; gi < 2; ++gi) {
                        const int cg = wi + 2 * gi;
                        if (cg * 32 < N1) {
                            uint32_t r[32];
                            tmem_load32(tmem + lane_addr + kTmD1 + d * 128 + cg * 32, r);
                            if (live) {
#pragma unroll
                                for (int q = 0; q < 4; ++q)
                                    if (soff[gi][q] != 0xFFFFFFFFu)
                                        st_op16<__nv_bfloat16>(sT + d * pl.t_bytes + soff[gi][q],
                                                               &r[q * 8]);
                            }
                        }
                    }
                }
                tc_fence_before();
                fence_proxy_async();
                mbar_arrive_warp(bar(kD1Empty + d));
                mbar_arrive_warp(bar(kTFull + d));
            }
        }
    } else {
        // ---------------- epilogue 2: Y (and bias, dH) -> outputs ----------------
        const int quad = warp & 3, wi = (warp - 11) >> 2;
        const int L = quad * 32 + lane, n_l = L / MP, k = k0 + L % MP;
        const uint32_t lane_addr = (uint32_t)(quad * 32) << 16;
        const bool k_ok = k < pl.M2;
        const int ng = pl.qcp / 16;
        const int qmax = min(pl.qc, pl.Q - c0);        // columns of this slice
        int ti = 0;
        bool ok = true;
        for (int t = group; t < pl.ntiles && ok; t += pl.groups, ++ti) {
            const int y = ti % pl.ybufs;
            const int64_t n = (int64_t)t * NT + n_l;
            const bool row_ok = n < g.N && k_ok;
            const size_t obase = (size_t)n * g.out_ld + (size_t)c0 * pl.M2 + k;
            bool waited = false;
            for (int cg = wi; cg < ng; cg += 2) {
                const int cb = cg * 16;
                float bg[16], bu[16], dh[16];
                if constexpr (MODE != kInput) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const bool in = row_ok && cb + i < qmax;
                        const size_t bo = (size_t)(c0 + cb + i) * pl.M2 + k;
                        bg[i] = g.bias && in ? __bfloat162float(__ldg(g.bias + bo)) : 0.f;
                        bu[i] = g.bias && in ? __bfloat162float(__ldg(g.bias + g.out_ld + bo))
                                             : 0.f;
                        if constexpr (MODE == kPre)
                            dh[i] = in ? __bfloat162float(
                                             __ldg(g.dH + obase + (size_t)(cb + i) * pl.M2))
                                       : 0.f;
                    }
                }
                if (!waited) {
                    if (!warp_wait(bar(kYFull + y), (ti / pl.ybufs) & 1, ab)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    waited = true;
                }
                __syncwarp();
                const uint32_t ya = tmem + lane_addr + kTmY + y * pl.nacc * pl.qcp + cb;
                uint32_t v0[16];
                tmem_load_n<16>(ya, v0);
                float o0[16], o1[16];
                if constexpr (MODE == kInput) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) o0[i] = __uint_as_float(v0[i]);
                } else {
                    uint32_t v1[16];
                    tmem_load_n<16>(ya + pl.qcp, v1);
                    gate16<MODE == kPre>(act, v0, v1, bg, bu, dh, o0, o1);
                }
                if (row_ok) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (cb + i < qmax) {
                            const size_t o = obase + (size_t)(cb + i) * pl.M2;
                            g.out0[o] = __float2bfloat16_rn(o0[i]);
                            if constexpr (MODE == kPre) g.out1[o] = __float2bfloat16_rn(o1[i]);
                        }
                }
                __syncwarp();
            }
            if (!ok) break;
            if (!waited) {     // no columns for this warp: only keep the phases in step
                if (!warp_wait(bar(kYFull + y), (ti / pl.ybufs) & 1, ab)) break;
            }
            tc_fence_before();
            mbar_arrive_warp(bar(kYEmpty + y));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

cudaError_t map_rows(CUtensorMap *map, const void *base, int64_t N, const Plan &pl) {
    auto enc = get_encode();
    if (!enc) return cudaErrorNotSupported;
    cuuint64_t dims[3] = {(cuuint64_t)pl.M1, (cuuint64_t)pl.P, (cuuint64_t)N};
    cuuint64_t strides[2] = {(cuuint64_t)pl.M1 * 2, (cuuint64_t)pl.P * pl.M1 * 2};
    cuuint32_t box[3] = {(cuuint32_t)pl.sw / 2, (cuuint32_t)pl.AC, (cuuint32_t)pl.NT};
    cuuint32_t es[3] = {1, 1, 1};
    const CUtensorMapSwizzle sw = pl.sw == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : pl.sw == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                : CU_TENSOR_MAP_SWIZZLE_32B;
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims,
                           strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
                           CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int MP>
const void *kernel_of(Mode m) {
    return m == kForward ? (const void *)glu_tc_kernel<MP, kForward>
           : m == kPre   ? (const void *)glu_tc_kernel<MP, kPre>
                         : (const void *)glu_tc_kernel<MP, kInput>;
}

}  // namespace

// Chooses MP, the c slices and the ring by an estimate of the kernel's time: per chunk the
// larger of its shared-memory cycles (128 B each) and its MMA cycles (4096 multiply-adds each)
// and about 80 of hand-over, per tile at least epilogue 2's time, per CTA the packing of the
// factors.  More slices mean less packing per CTA and room for the factors, and more repeats of
// stage 1 and of the reads of x.
bool tc_plan(Plan *best, const Shape &s, Mode mode, int sms) {
    double best_cost = 0;
    bool found = false;
    const bool tr = mode == kInput;
    for (int MP = 16; MP <= 128; MP *= 2) {
        Plan p{};
        p.P = tr ? s.q : s.p;
        p.M1 = tr ? s.m2 : s.m1;
        p.Q = tr ? s.p : s.q;
        p.M2 = tr ? s.m1 : s.m2;
        p.r = s.r;
        p.nsrc = tr ? 2 : 1;
        p.ranks = tr ? s.r : 2 * s.r;
        p.nacc = tr ? 1 : 2;
        if (MP > 16 && MP >= 2 * p.M2) continue;
        p.MP = MP;
        p.NT = p.RB = 128 / MP;
        p.nac = cdiv(p.P, MP);
        p.AC = up(cdiv(p.P, p.nac), 8);
        p.nblk_src = cdiv(p.ranks, p.RB);
        p.nblk = p.nsrc * p.nblk_src;
        // whole K steps of 16 for every block's ranks and for the gate's part of them
        bool whole = (p.NT * p.AC) % 16 == 0;
        for (int b = 0; b < p.nblk_src; ++b) {
            const int live = gmin(p.RB, p.ranks - b * p.RB);
            const int gate = tr ? live : gmin(live, gmax(0, s.r - b * p.RB));
            whole = whole && (live * p.AC) % 16 == 0 && (gate * p.AC) % 16 == 0;
        }
        if (!whole) p.AC = up(p.AC, 16);
        const int rowb = up(p.M1, 16) * 2;
        p.sw = rowb <= 32 ? 32 : rowb <= 64 ? 64 : 128;
        p.kch = cdiv(rowb, p.sw);
        p.kb = p.kch * p.sw;
        p.nks = cdiv(p.M2, MP);
        p.rbl = gmin(p.RB, p.ranks);
        const int K2 = p.rbl * p.AC, K2b = up(K2 * 2, 128), N1 = p.NT * p.AC;
        p.t_bytes = 128 * K2b;
        p.x_bytes = up(N1 * p.kb, 1024);
        const int64_t tiles = (s.N + p.NT - 1) / p.NT;
        if (tiles > 0x7fffffff / 4 || p.kb > 1024) continue;
        p.ntiles = (int)tiles;
        for (int nqs = 1; nqs <= p.Q; ++nqs) {
            p.qc = cdiv(p.Q, nqs);
            p.qcp = up(p.qc, 16);
            if (cdiv(p.Q, p.qc) != nqs || p.nacc * p.qcp > 256) continue;
            if (nqs > 1 && p.qc < 8) break;
            p.nqs = nqs;
            p.ybufs = 2 * p.nacc * p.qcp <= 256 ? 2 : 1;
            p.c_chunk = up(p.qcp * K2b, 1024);
            const int64_t bytes_b = (int64_t)p.nblk * 128 * p.kb;
            const int64_t bytes_c = (int64_t)p.nac * p.nblk * p.c_chunk;
            const int64_t fixed = bytes_b + bytes_c + 2 * p.t_bytes;
            if (fixed + 2 * p.x_bytes > kSmemMax) continue;
            p.stages = (int)((kSmemMax - fixed) / p.x_bytes);
            if (p.stages > kMaxStages) p.stages = kMaxStages;
            p.off_c = (int)bytes_b;
            p.off_t = (int)(bytes_b + bytes_c);
            p.off_x = p.off_t + 2 * p.t_bytes;
            p.smem = p.off_x + p.stages * p.x_bytes;
            const int slices = p.nqs * p.nks;
            p.groups = (int)(tiles < sms / slices ? tiles : sms / slices);
            if (p.groups < 1) p.groups = 1;
            const double mem = 4.0 * K2 + (128.0 + N1) * p.kb / 128 + 2.0 * K2 * p.qcp / 128 +
                               (double)N1 * p.kb / 128 / p.nblk_src;
            const double mma = 128.0 * N1 * p.kb / 2 / 4096 + 128.0 * K2 * p.qcp / 4096;
            const double tile = p.nac * p.nblk * ((mem > mma ? mem : mma) + 80);
            const double epi = p.qc * (mode == kPre ? 40.0 : 20.0);
            const double pack = 2000 + (bytes_b + 2.0 * bytes_c) / 2 / kThreads * 12;
            const double waves = (double)((tiles + p.groups - 1) / p.groups) *
                                 (slices > sms ? cdiv(slices, sms) : 1);
            const double cost = pack + waves * (tile > epi ? tile : epi) + 1500;
            if (!found || cost < best_cost) {
                best_cost = cost;
                *best = p;
                found = true;
            }
        }
    }
    return found;
}

cudaError_t tc_run(const Plan &pl, const TcArgs &a, Mode mode, cudaStream_t st) {
    launch_step() = "tensor map";
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaSetDevice(dev);   // binds the context for the driver call
    CUtensorMap m0, m1;
    if (e == cudaSuccess) e = map_rows(&m0, a.src0, a.N, pl);
    if (e == cudaSuccess) e = map_rows(&m1, mode == kInput ? a.src1 : a.src0, a.N, pl);
    if (e != cudaSuccess) return e;
    KArgs k{};
    k.pl = pl;
    k.S = static_cast<const __nv_bfloat16 *>(a.S);
    k.A = static_cast<const __nv_bfloat16 *>(a.A);
    k.B = static_cast<const __nv_bfloat16 *>(a.B);
    k.bias = mode == kInput ? nullptr : static_cast<const __nv_bfloat16 *>(a.bias);
    k.dH = static_cast<const __nv_bfloat16 *>(a.dH);
    k.out0 = static_cast<__nv_bfloat16 *>(a.out0);
    k.out1 = static_cast<__nv_bfloat16 *>(a.out1);
    k.N = a.N;
    const bool tr = mode == kInput;
    const int m2 = tr ? pl.M1 : pl.M2, q = tr ? pl.P : pl.Q;   // the layer's m2 and q
    k.sBi = tr ? 1 : m2;
    k.sBo = tr ? m2 : 1;
    k.sCa = tr ? 1 : q;
    k.sCc = tr ? q : 1;
    k.pq = pl.P * pl.Q;
    k.mm = pl.M1 * pl.M2;
    k.out_ld = pl.Q * pl.M2;
    launch_step() = "device error word";
    k.device_error = device_error_ptr();
    if (!k.device_error) return cudaErrorInvalidSymbol;
    const void *f = pl.MP == 16   ? kernel_of<16>(mode)
                    : pl.MP == 32 ? kernel_of<32>(mode)
                    : pl.MP == 64 ? kernel_of<64>(mode)
                                  : kernel_of<128>(mode);
    const size_t smem = (size_t)pl.smem + kTailBytes + 1024;
    launch_step() = "shared memory size";
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    launch_step() = "kernel launch";
    int act = a.activation;
    void *params[] = {&m0, &m1, &k, &act};
    return cudaLaunchKernel(f, dim3((unsigned)(pl.groups * pl.nqs * pl.nks)), dim3(kThreads),
                            params, smem, st);
}

}  // namespace glu
}  // namespace kron
