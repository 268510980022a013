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
// (12 warps) moves a chunk TMEM -> bf16 -> shared memory, which is the permute of the vec trick;
// epilogue 2 (16 warps) has g and u of one (n, k, c) side by side.  For kInput the kernel runs
// with transposed factors, dg against the gate's and du against the up's ranks, and the two
// accumulators are added.  T is rounded to BF16 between the stages and C_i = S (.) A_i as it is
// packed, as in the layer's own kernels, because the MMA takes BF16 operands: each half a step,
// 2^-8 of a term.
//
// A CTA holds the factors of one (k slice, c slice) in shared memory for its life and streams
// row tiles; slices exist where the factors do not fit at once, and for few rows, where the
// set-up of the factors is what takes the time.  Stage 1 is repeated for each c slice.
// Bound by the SM's shared-memory pipe and issue slots: per chunk 32 KB of T are stored and read
// back beside the MMAs' other operands, 512 cycles at 128 B/clk for the 32 x 32 blocks against
// 256 cycles of MMA.  20000 x 1024, r = 4: 45 us, 73% of the pipe's cycles (35 the warps', 38 the
// tensor core's), 74% of the issue slots, 0.91 TB/s of HBM.  Backward of these rows:
// pre-activations' gradients 67 us (epilogue 2's latency: three reads and two stores per element),
// dX 44.
// Wide layers whose factors of both projections exceed one SM's shared memory (64 x 64 blocks, r =
// 8: 262 KB) are bound by repeats instead: two slices of c, so that every T is formed, stored and
// read back twice, and stage-2 MMAs of N = 32, which take 74 cycles where 16 is the rate.  16384 x
// 4096, r = 8: 391 us, 703 TFLOP/s, from a cool GPU and 450 us, 611 TFLOP/s, under the power cap;
// two forward calls of the layer (176 us each) and an elementwise gate (62 us of HBM traffic) take
// as long.
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

constexpr int kE1 = 12, kE2 = 16;      // epilogue warps
constexpr int kG1 = kE1 / 4;           // groups of epilogue-1 warps, one chunk each at a time
constexpr int kThreads = 32 * (4 + kE1 + kE2);   // and TMA and three MMA issuers
constexpr int kMaxStages = 6;
constexpr int kTailBytes = 512;        // barriers, TMEM address, abort flag
constexpr int kSmemMax = 232448 - 1024 - kTailBytes;
constexpr int kMaxT = 4, kMaxD = 3;    // T buffers, D1 buffers (128 TMEM columns each)

struct KArgs {
    Plan pl;
    const __nv_bfloat16 *S, *A, *B, *bias, *dH;
    __nv_bfloat16 *out0, *out1;
    int64_t N;
    int pq, mm;                // elements of one S or A_i, and of one B_i
    int out_ld;
    int *device_error;
};

// Barriers, in 8-byte words from the tail's start.
enum { kXFull = 0, kXEmpty = kMaxStages, kD1Full = 2 * kMaxStages, kD1Empty = kD1Full + kMaxD,
       kTFull = kD1Empty + kMaxD, kTEmpty = kTFull + kMaxT, kYFull = kTEmpty + kMaxT,
       kYEmpty = kYFull + 2, kDrain = kYEmpty + 2, kBars = kDrain + 3 };
static_assert(kBars * 8 + 16 <= kTailBytes, "tail");

// A shared-memory descriptor from its low word (address) and the high word of its layout: steps
// along an operand then change one 32-bit word.
__device__ __forceinline__ uint64_t desc_of(uint32_t lo, uint32_t hi) {
    return ((uint64_t)hi << 32) | lo;
}

// The two bfloat16 of a word, or of two words the lower or upper ones side by side, in fp32.
__device__ __forceinline__ f2 lower2(uint32_t a, uint32_t b) {
    return pack2(__uint_as_float(a << 16), __uint_as_float(b << 16));
}
__device__ __forceinline__ f2 upper2(uint32_t a, uint32_t b) {
    return pack2(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u));
}

// One epilogue-2 item: accumulators r (gate) and q (up) of four columns at k and k + 1, two columns
// side by side in packed arithmetic: pair (rep, kk) holds the columns 2 rep and 2 rep + 1 at
// k + kk.  w0 and w1 get the outputs of each column as a pair (k, k + 1).
template <int ACT, bool PRE>
__device__ __forceinline__ void gate_item(const uint32_t (&r)[8], const uint32_t (&q)[8],
                                          const uint32_t (&bg)[4], const uint32_t (&bu)[4],
                                          const uint32_t (&dh)[4], uint32_t (&w0)[4],
                                          uint32_t (&w1)[4]) {
#pragma unroll
    for (int rep = 0; rep < 2; ++rep) {
        float o[2][2], p[2][2];      // [kk][column]
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            const int i = 4 * rep + 2 * kk, c = 2 * rep;
            const f2 g = add2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                              kk ? upper2(bg[c], bg[c + 1]) : lower2(bg[c], bg[c + 1]));
            const f2 u = add2(pack2(__uint_as_float(q[i]), __uint_as_float(q[i + 1])),
                              kk ? upper2(bu[c], bu[c + 1]) : lower2(bu[c], bu[c + 1]));
            f2 d;
            const f2 f = act2<ACT, PRE>(g, d);
            if constexpr (PRE) {
                const f2 h = kk ? upper2(dh[c], dh[c + 1]) : lower2(dh[c], dh[c + 1]);
                unpack2(mul2(mul2(h, u), d), o[kk][0], o[kk][1]);
                unpack2(mul2(h, f), p[kk][0], p[kk][1]);
            } else {
                unpack2(mul2(f, u), o[kk][0], o[kk][1]);
            }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            w0[2 * rep + c] = pack_bf16x2(o[0][c], o[1][c]);
            if constexpr (PRE) w1[2 * rep + c] = pack_bf16x2(p[0][c], p[1][c]);
        }
    }
}

// Accumulator column (row of the packed C') that holds column c of a slice: in each group of 16 the
// thread tq of a 16x256b load has the columns 2 tq, 2 tq + 1, 2 tq + 8 and 2 tq + 9, and these
// hold c = tq, tq + 4, tq + 8 and tq + 12, so that one store of a warp covers four adjacent c.
__device__ __forceinline__ int acc_column(int c) {
    const int i = (c >> 2) & 3;
    return (c & ~15) + 8 * (i >> 1) + 2 * (c & 3) + (i & 1);
}

// 16 lanes x 16 columns in the 16x256b pattern (tmem_load16x256_x4 with two repetitions) of two
// accumulators, one wait for both.
__device__ __forceinline__ void tmem_load16x256_x2(uint32_t ta, uint32_t tb, uint32_t (&r)[8],
                                                   uint32_t (&q)[8]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%16];\n\t"
        "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%17];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(q[0]), "=r"(q[1]), "=r"(q[2]), "=r"(q[3]), "=r"(q[4]), "=r"(q[5]),
          "=r"(q[6]), "=r"(q[7])
        : "r"(ta), "r"(tb)
        : "memory");
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

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int nslices = pl.nqs * pl.nks;
    const int slice = blockIdx.x % nslices, group = blockIdx.x / nslices;
    const int k0 = (slice / pl.nqs) * MP, c0 = (slice % pl.nqs) * pl.qc;
    const int N1 = NT * pl.AC;
    const int nchunks = pl.nac * pl.nblk;      // stage-1 / stage-2 chunks of a tile

    constexpr bool TR = MODE == kInput;
    const int x_chunks = pl.nsrc * pl.nac;     // ring items of a tile

    // x chunk (ac, source) of tile t into ring slot s, by one thread
    auto issue_x = [&](int t, int ac, int src, int s) {
        const CUtensorMap *map = src ? &map1 : &map0;
        mbar_arrive_expect_tx(bar(kXFull + s), N1 * pl.kb);
        for (int kc = 0; kc < pl.kch; ++kc)
            asm volatile(
                "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes "
                "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(sX + s * pl.x_bytes + kc * N1 * pl.sw),
                "l"(reinterpret_cast<uint64_t>(map)), "r"(kc * (pl.sw >> 1)), "r"(ac * pl.AC),
                "r"(t * NT), "r"(bar(kXFull + s))
                : "memory");
    };
    // the producer's position: ring slot and parity, tile, chunk (warp 0 lane 0)
    int xs = 0, xph = 1, xt = group, xac = 0, xsrc = 0, xissued = 0;
    auto advance_x = [&]() {
        if (++xsrc == pl.nsrc) {
            xsrc = 0;
            if (++xac == pl.nac) xac = 0, xt += pl.groups;
        }
        if (++xs == pl.stages) xs = 0, xph ^= 1;
        ++xissued;
    };

    if (threadIdx.x == 0) {
        for (int s = 0; s < pl.stages; ++s) {
            mbar_init(bar(kXFull + s), 1);
            mbar_init(bar(kXEmpty + s), 1);
        }
        for (int d = 0; d < kMaxD; ++d) {
            mbar_init(bar(kD1Full + d), 1);
            mbar_init(bar(kD1Empty + d), 4);
        }
        for (int d = 0; d < kMaxT; ++d) {
            mbar_init(bar(kTFull + d), 4);
            mbar_init(bar(kTEmpty + d), 2);
        }
        for (int d = 0; d < 2; ++d) {
            mbar_init(bar(kYFull + d), 2);
            mbar_init(bar(kYEmpty + d), kE2);
            mbar_init(bar(kDrain + d), 1);
        }
        mbar_init(bar(kDrain + 2), 1);
        *ab.flag = 0;
        mbar_init_fence();
        prefetch_tmap(&map0);
        if (pl.nsrc > 1) prefetch_tmap(&map1);
    }
    if (warp == 1) tmem_alloc(smem_u32(const_cast<uint32_t *>(tmem_slot)), 512);

    // ---- factors to shared memory, zero past the sizes, eight values of the index that is
    // contiguous in memory per thread and step.  The loops are kept small: a CTA runs them once
    // or twice, and fetching their instructions takes longer than their loads (unrolled to
    // sixteen loads in flight the same packing took 17,000 cycles instead of 11,000).
    // The ranks of gate and up are one list f in the order of A and B in memory; kInput has
    // them by source.  Warp 0 fills the x ring meanwhile.
    if (!pl.exact) zero_smem(sB, pl.off_t);
    __syncthreads();
    if (warp == 0) {
        if (lane == 0)
            for (int i = 0; i < pl.stages && xt < pl.ntiles; ++i) {
                issue_x(xt, xac, xsrc, xs);
                advance_x();
            }
        __syncwarp();
    } else {
        const int nranks = pl.nsrc * pl.ranks;               // 2 r
        // rank f: (source, block, position)
        auto place = [&](int f, int &so, int &bs, int &il) {
            so = TR && f >= pl.ranks ? 1 : 0;
            const int i = f - so * pl.ranks;
            bs = i / RB;
            il = i % RB;
        };
        // stage-1 A operand: row L = (il, l) of a block holds B_i[., k0 + k] with
        // k = pair_lane_index(l): epilogue 2 then finds k and k + 1 in one thread
        {
            const int swl = 31 - __clz(pl.sw);
            const uint32_t xmask = (uint32_t)(pl.sw >> 4) - 1;
            // TR: eight j (all of K's row: 16 bytes); else eight k (two or four bytes apart in l)
            const int inner = (TR ? pl.M1 : MP) >> 3, outer = TR ? MP : pl.M1;
            for (int e = threadIdx.x - 32; e < nranks * outer * inner; e += kThreads - 32) {
                const int rest = e / inner, in8 = (e - rest * inner) * 8;
                const int f = rest / outer, row = rest - f * outer;
                const int k = k0 + (TR ? pair_lane_index(row) : in8);
                if (k >= pl.M2) continue;
                const uint4 v = *reinterpret_cast<const uint4 *>(
                    g.B + (size_t)f * g.mm + (TR ? k * pl.M1 + in8 : row * pl.M2 + k));
                int so, bs, il;
                place(f, so, bs, il);
                const uint32_t jb = 2u * (uint32_t)(TR ? in8 : row);
                const uint32_t blk = sB + (so * pl.nblk_src + bs) * 128 * pl.kb;
                const uint32_t at = ((jb >> swl) * 128u << swl) + (jb & (uint32_t)(pl.sw - 1)) +
                                    (uint32_t)(il * MP) * pl.sw;
                if constexpr (TR) {
                    const uint32_t off = at + row * pl.sw;
                    st_shared_v4(blk + (off ^ ((off >> 7 & xmask) << 4)), v.x, v.y, v.z, v.w);
                } else {
                    // k = in8 + t lies in lane (in8 & ~15) + (k & 15) / 2 + 8 (k & 1)
                    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
                    const int l0 = (in8 & ~15) + ((in8 & 8) >> 1);
#pragma unroll
                    for (int t = 0; t < 8; ++t) {
                        const uint32_t off = at + (uint32_t)(l0 + (t >> 1) + 8 * (t & 1)) * pl.sw;
                        st_shared_u16(blk + (off ^ ((off >> 7 & xmask) << 4)),
                                      (uint16_t)(w[t >> 1] >> (16 * (t & 1))));
                    }
                }
            }
        }
        // stage-2 B operand of chunk ch = (ac, source, block), in the order of the tile's
        // chunks: row acc_column(c), K position il*AC + a % AC: C_i[a][c0 + c]
        {
            const int cmax = min(pl.qc, pl.Q - c0);
            const int outer = TR ? cmax : pl.P, len = TR ? pl.P : cmax, inner = (len + 7) >> 3;
            // rows of S and A_i start on 16 bytes, and so do the slices of them
            const bool vec = TR ? pl.P % 8 == 0 : pl.Q % 8 == 0 && c0 % 8 == 0;
            for (int e = threadIdx.x - 32; e < nranks * outer * inner; e += kThreads - 32) {
                const int rest = e / inner, in8 = (e - rest * inner) * 8;
                const int f = rest / outer, row = rest - f * outer;
                const size_t o = TR ? (size_t)(c0 + row) * pl.P + in8
                                    : (size_t)row * pl.Q + c0 + in8;
                const __nv_bfloat16 *pa = g.A + (size_t)f * g.pq + o;
                const __nv_bfloat16 *ps = g.S + (f >= pl.r ? g.pq : 0) + o;
                const int left = len - in8;
                uint32_t wa[4] = {0, 0, 0, 0}, ws[4] = {0, 0, 0, 0};
                if (vec && left >= 8) {
                    const uint4 va = *reinterpret_cast<const uint4 *>(pa);
                    const uint4 vs = *reinterpret_cast<const uint4 *>(ps);
                    wa[0] = va.x, wa[1] = va.y, wa[2] = va.z, wa[3] = va.w;
                    ws[0] = vs.x, ws[1] = vs.y, ws[2] = vs.z, ws[3] = vs.w;
                } else {
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        if (t < left) {
                            wa[t >> 1] |= (uint32_t)__bfloat16_as_ushort(pa[t]) << (16 * (t & 1));
                            ws[t >> 1] |= (uint32_t)__bfloat16_as_ushort(ps[t]) << (16 * (t & 1));
                        }
                }
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    wa[t] = pack_bf16x2(
                        __uint_as_float(wa[t] << 16) * __uint_as_float(ws[t] << 16),
                        __uint_as_float(wa[t] & 0xFFFF0000u) *
                            __uint_as_float(ws[t] & 0xFFFF0000u));
                int so, bs, il;
                place(f, so, bs, il);
                const int a = TR ? in8 : row, ac = a / pl.AC;
                const uint32_t kb = (uint32_t)(il * pl.AC + a - ac * pl.AC) * 2u;
                const uint32_t at = sC + ((ac * pl.nsrc + so) * pl.nblk_src + bs) * pl.c_chunk +
                                    (kb >> 7) * (uint32_t)pl.qcp * 128u;
                const uint32_t in = kb & 127u;
                if constexpr (TR) {      // zeros behind p: inside the chunk's padding
                    const int c = acc_column(row);
                    st_shared_v4(at + c * 128 + (in ^ ((c & 7) << 4)), wa[0], wa[1], wa[2], wa[3]);
                } else {
#pragma unroll
                    for (int t = 0; t < 8; ++t)
                        if (t < left) {
                            const int c = acc_column(in8 + t);
                            st_shared_u16(at + c * 128 + (in ^ ((c & 7) << 4)),
                                          (uint16_t)(wa[t >> 1] >> (16 * (t & 1))));
                        }
                }
            }
        }
    }
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;

    if (warp == 0) {
        // ---------------- TMA producer ----------------
        if (lane == 0) {
            while (xt < pl.ntiles) {
                if (!mbar_wait(bar(kXEmpty + xs), xph, ab)) break;
                issue_x(xt, xac, xsrc, xs);
                advance_x();
            }
            for (int v = xissued > pl.stages ? xissued - pl.stages : 0; v < xissued; ++v)
                mbar_wait_drain(bar(kXFull + v % pl.stages), (v / pl.stages) & 1);
        }
    } else if (warp == 1) {
        // ---------------- stage 1 ----------------
        const uint32_t idesc = idesc_f32acc(128, N1, 1);
        const int ksteps = (pl.M1 + 15) >> 4;
        const int per_ch = pl.sw >> 5;                 // K steps per chunk of an x row
        const int kfirst = min(ksteps, per_ch);
        const uint64_t bdx = sdesc_kmajor(sX, pl.sw);
        const uint32_t hi = (uint32_t)(bdx >> 32), x_lo = (uint32_t)bdx;
        const uint32_t b_lo = (uint32_t)sdesc_kmajor(sB, pl.sw);
        const uint32_t a_ch = 8u * pl.sw, b_ch = (uint32_t)(N1 * pl.sw) >> 4;   // per chunk
        const uint32_t a_blk = 8u * pl.kb, x_stage = (uint32_t)pl.x_bytes >> 4;
        int s = 0, ph = 0, d1 = 0, dph = 1;
        bool ok = true;
        for (int t = group; t < pl.ntiles && ok; t += pl.groups) {
            for (int xc = 0; xc < x_chunks && ok; ++xc) {
                if (!warp_wait(bar(kXFull + s), ph, ab)) {
                    ok = false;
                    break;
                }
                const uint32_t bd0 = x_lo + s * x_stage;
                uint32_t ad0 = b_lo + (TR && (xc & 1) ? pl.nblk_src * a_blk : 0u);
                for (int b = 0; b < pl.nblk_src; ++b, ad0 += a_blk) {
                    if (!warp_wait(bar(kD1Empty + d1), dph, ab)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t dst = tmem + d1 * 128;
                    if (elect_one()) {
                        mma_ss<false>(dst, desc_of(ad0, hi), desc_of(bd0, hi), idesc, 0);
#pragma unroll
                        for (int kk = 1; kk < 4; ++kk)      // the first chunk: 64 columns j
                            if (kk < kfirst)
                                mma_ss<false>(dst, desc_of(ad0 + kk * 2, hi),
                                              desc_of(bd0 + kk * 2, hi), idesc, 1);
                        for (int kk = per_ch; kk < ksteps; ++kk) {
                            const uint32_t ch = kk / per_ch, in = (kk % per_ch) * 2;
                            mma_ss<false>(dst, desc_of(ad0 + ch * a_ch + in, hi),
                                          desc_of(bd0 + ch * b_ch + in, hi), idesc, 1);
                        }
                        mma_commit(bar(kD1Full + d1));
                        if (b == pl.nblk_src - 1) mma_commit(bar(kXEmpty + s));
                    }
                    __syncwarp();
                    if (++d1 == pl.dbufs) d1 = 0, dph ^= 1;
                }
                if (++s == pl.stages) s = 0, ph ^= 1;
            }
        }
        if (elect_one()) mma_commit(bar(kDrain + 0));
        __syncwarp();
        if (lane == 0) mbar_wait_drain(bar(kDrain + 0), 0);
        __syncwarp();
    } else if (warp < 4) {
        // ---------------- stage 2: one warp per accumulator ----------------
        // Gate's ranks (kInput: dg) and up's (du) go to accumulators of their own, each issued by
        // one warp, so that one's waits and descriptors overlap the other's MMAs.  Both follow
        // every chunk (an arrival in place of the MMAs of the other's), so that neither falls a
        // phase behind.
        const int me = warp - 2;
        const uint32_t idesc = idesc_f32acc(128, pl.qcp, 1);
        const uint64_t adt = sdesc_kmajor(sT, 128);
        const uint32_t hi = (uint32_t)(adt >> 32), t_lo = (uint32_t)adt;
        const uint32_t c_lo = (uint32_t)sdesc_kmajor(sC, 128);
        const uint32_t t_buf = (uint32_t)pl.t_bytes >> 4, c_step = (uint32_t)pl.c_chunk >> 4;
        const uint32_t c_ch = 8u * pl.qcp;
        const int a16 = pl.AC >> 3;              // half K steps per rank
        const int steps_full = (RB * a16) >> 1;
        const int steps_last = ((pl.ranks - (pl.nblk_src - 1) * RB) * a16) >> 1;
        // K steps [lo, hi) of a block are this warp's: with gate and up in one list, blocks below
        // r / RB are gate's, the one at it may be both, the rest up's
        const int edge = pl.r / RB, split = ((pl.r % RB) * a16) >> 1;
        int tb = 0, tph = 0, y = 0, yph = 1;
        bool ok = true;
        for (int t = group; t < pl.ntiles && ok; t += pl.groups) {
            if (!warp_wait(bar(kYEmpty + y), yph, ab)) break;
            const uint32_t dst = tmem + pl.tm_y + (2 * y + me) * pl.qcp;
            uint32_t acc = 0;                    // whether the accumulator holds something
            uint32_t bd0 = c_lo;
            for (int ch = 0, bs = 0, src = 0; ch < nchunks; ++ch, bd0 += c_step) {
                const int steps = bs == pl.nblk_src - 1 ? steps_last : steps_full;
                int k_lo = 0, k_hi = steps;
                if (TR) {
                    if (src != me) k_hi = 0;
                } else if (me == 0) {
                    if (bs >= edge) k_hi = bs == edge ? split : 0;
                } else {
                    if (bs <= edge) k_lo = bs == edge ? split : steps;
                }
                const uint32_t ad0 = t_lo + tb * t_buf;
                if (!warp_wait(bar(kTFull + tb), tph, ab)) {
                    ok = false;
                    break;
                }
                if (k_lo < k_hi) {
                    tc_fence_after();
                    if (elect_one()) {
                        if (k_hi - k_lo == 8) {
                            mma_ss<false>(dst, desc_of(ad0, hi), desc_of(bd0, hi), idesc, acc);
#pragma unroll
                            for (int ks = 1; ks < 8; ++ks)
                                mma_ss<false>(
                                    dst, desc_of(ad0 + (ks >> 2) * 1024 + (ks & 3) * 2, hi),
                                    desc_of(bd0 + (ks >> 2) * c_ch + (ks & 3) * 2, hi), idesc, 1);
                        } else {
                            for (int ks = k_lo; ks < k_hi; ++ks)
                                mma_ss<false>(
                                    dst, desc_of(ad0 + (ks >> 2) * 1024 + (ks & 3) * 2, hi),
                                    desc_of(bd0 + (ks >> 2) * c_ch + (ks & 3) * 2, hi), idesc,
                                    acc | (uint32_t)(ks > k_lo));
                        }
                        mma_commit(bar(kTEmpty + tb));
                    }
                    acc = 1;
                } else if (elect_one()) {
                    mbar_arrive(bar(kTEmpty + tb));
                }
                __syncwarp();
                if (++tb == pl.tbufs) tb = 0, tph ^= 1;
                if (++bs == pl.nblk_src) {
                    bs = 0;
                    if (TR) src ^= 1;
                }
            }
            if (!ok) break;
            if (elect_one()) mma_commit(bar(kYFull + y));
            __syncwarp();
            if (++y == pl.ybufs) y = 0, yph ^= 1;
        }
        if (elect_one()) mma_commit(bar(kDrain + 1 + me));
        __syncwarp();
        if (lane == 0) mbar_wait_drain(bar(kDrain + 1 + me), 0);
        __syncwarp();
    } else if (warp < 4 + kE1) {
        // ---------------- epilogue 1: D1 -> T ----------------
        // Groups of four warps, one per lane quadrant, take the chunks in turn: a chunk's loads,
        // conversions and stores take longer than its MMAs, and up to three are in flight.  No
        // more groups than buffers of D1 and of T: a group that waits for a buffer has then
        // seen the use before the last one end (it ended before the group's own last chunk was
        // stored), so the parity it waits for cannot be an older phase's.
        const int quad = warp & 3, mine = (warp - 4) >> 2;
        const int L = quad * 32 + lane, il = L / MP, l = L % MP;
        const uint32_t d1_addr = tmem + ((uint32_t)(quad * 32) << 16);
        // columns (n, a..a+7) of this lane go to row (n, l) of T, K position il*AC + a; with AC =
        // MP that is one of MP/8 addresses and a constant (the swizzle depends on l alone)
        const bool full = pl.AC == MP;
        uint32_t soff[MP / 8];
#pragma unroll
        for (int j = 0; j < MP / 8; ++j) soff[j] = sT + kmaj(l, (il * MP + j * 8) * 2, 128, 128);
        int d = mine, dph = 0, tb = mine, tph = 1, t = group, bs = mine, ch = mine;
        auto wrap = [&]() {
            while (d >= pl.dbufs) d -= pl.dbufs, dph ^= 1;
            while (tb >= pl.tbufs) tb -= pl.tbufs, tph ^= 1;
            while (bs >= pl.nblk_src) bs -= pl.nblk_src;
            while (ch >= nchunks) ch -= nchunks, t += pl.groups;
        };
        wrap();
        while (mine < pl.g1 && t < pl.ntiles) {
            if (!warp_wait(bar(kD1Full + d), dph, ab) || !warp_wait(bar(kTEmpty + tb), tph, ab))
                break;
            tc_fence_after();
            // a warp's lanes hold one rank, or two (MP = 16): live is per lane
            const bool live = bs * RB + il < pl.ranks;
            const bool some = __any_sync(0xffffffffu, live);
            const uint32_t to = tb * pl.t_bytes;
            if (some && full) {
                // AC = MP: column group f lies in row n = f / MP, at a = f % MP
                uint32_t base8[MP / 8];
#pragma unroll
                for (int j = 0; j < MP / 8; ++j) base8[j] = soff[j] + to;
#pragma unroll
                for (int gi = 0; gi < 4; ++gi) {
                    uint32_t r[32];
                    tmem_load32(d1_addr + d * 128 + gi * 32, r);
                    if (live) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int f = gi * 32 + q * 8;
                            st_op16<__nv_bfloat16>(base8[f % MP / 8] + f / MP * MP * 128, &r[q * 8]);
                        }
                    }
                }
            } else if (some) {
#pragma unroll 1
                for (int gi = 0; gi * 32 < N1; ++gi) {
                    uint32_t r[32];
                    tmem_load32(d1_addr + d * 128 + gi * 32, r);
                    if (live) {
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int f = gi * 32 + q * 8, n = f / pl.AC, a = f - n * pl.AC;
                            if (f < N1)
                                st_op16<__nv_bfloat16>(
                                    sT + to + kmaj(n * MP + l, (il * pl.AC + a) * 2, 128, 128),
                                    &r[q * 8]);
                        }
                    }
                }
            }
            tc_fence_before();
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(kD1Empty + d));
                mbar_arrive(bar(kTFull + tb));
            }
            d += pl.g1;
            tb += pl.g1;
            bs += pl.g1;
            ch += pl.g1;
            wrap();
        }
    } else {
        // ---------------- epilogue 2: Y (and bias, dH) -> outputs ----------------
        // A warp has 16 lanes of its quadrant and every second 16-column group; its items are
        // (tile, group).  A thread holds, for the columns c = tq, tq + 4, tq + 8 and tq + 12 of the
        // group, the pair of values k, k + 1.  For kPre the dH of an item are fetched two items
        // ahead.
        const int quad = warp & 3, wi = (warp - 4 - kE1) >> 2, w0c = wi >> 1;
        const int L16 = quad * 32 + (wi & 1) * 16, n_l = L16 / MP;
        const int kl = L16 % MP + 2 * (lane >> 2), k = k0 + kl, tq = lane & 3;
        const uint32_t y_addr = tmem + ((uint32_t)L16 << 16) + pl.tm_y;
        const bool k_ok = k < pl.M2;
        const int ni = ((pl.qcp >> 4) + 1 - w0c) >> 1;     // items per tile
        const int qmax = min(pl.qc, pl.Q - c0) - tq;   // columns of this slice, from tq on
        const size_t lane_off =
            (size_t)n_l * g.out_ld + (size_t)(c0 + tq + 16 * w0c) * pl.M2 + k;
        const size_t tile_step = (size_t)NT * g.out_ld * pl.groups;   // to this CTA's next tile
        const size_t item_step = (size_t)32 * pl.M2;
        const int nlast = (int)g.N - n_l;                   // rows t NT below it exist
        uint32_t dh[2][4] = {};
        int ft = group, fi = 0;                        // next item to fetch
        const __nv_bfloat16 *fsrc =
            MODE == kPre ? g.dH + (size_t)group * NT * g.out_ld + lane_off : nullptr;
        auto fetch_next = [&](uint32_t (&to)[4]) {
            if (ft >= pl.ntiles) return;
            const bool row_ok = ft * NT < nlast && k_ok;
            const __nv_bfloat16 *src = fsrc + (size_t)fi * item_step;
            const int left = row_ok ? qmax - (w0c + 2 * fi) * 16 : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = 4 * i;
                to[i] = c < left ? __ldg(reinterpret_cast<const unsigned int *>(src + c * pl.M2))
                                 : 0u;
            }
            if (++fi == ni) fi = 0, ft += pl.groups, fsrc += tile_step;
        };
        __nv_bfloat16 *p0 = g.out0 + (size_t)group * NT * g.out_ld + lane_off;
        __nv_bfloat16 *p1 =
            MODE == kPre ? g.out1 + (size_t)group * NT * g.out_ld + lane_off : nullptr;
        // biases of an item's four pairs: kept in registers where a warp has one item per tile,
        // read again for each otherwise (from shared memory they took a seventh of its cycles)
        uint32_t bias_g[4] = {}, bias_u[4] = {};
        auto load_bias = [&](int item) {
            const __nv_bfloat16 *p =
                g.bias + (size_t)(c0 + tq + 16 * w0c + 32 * item) * pl.M2 + k;
            const int left = k_ok ? qmax - (w0c + 2 * item) * 16 : 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = 4 * i;
                if (c < left) {
                    bias_g[i] = __ldg(reinterpret_cast<const unsigned int *>(p + c * pl.M2));
                    bias_u[i] =
                        __ldg(reinterpret_cast<const unsigned int *>(p + g.out_ld + c * pl.M2));
                }
            }
        };
        const bool biased = MODE != kInput && g.bias != nullptr;
        if (biased && ni > 0) load_bias(0);
        int t = group, item = 0, y = 0, yph = 0;
        // one item; false when the pipeline gave up
        auto process = [&](uint32_t (&d)[4]) -> bool {
            if (biased && ni > 1) load_bias(item);
            if (item == 0) {
                if (!warp_wait(bar(kYFull + y), yph, ab)) return false;
                tc_fence_after();
            }
            const int cb = (w0c + 2 * item) * 16;
            const uint32_t ya = y_addr + 2 * y * pl.qcp + cb;
            uint32_t w0[4], w1[4];
            // registers 4 rep + (0, 1) hold k at the accumulator columns 8 rep + 2 tq (+ 1), that
            // is at the i-th c for i = 2 rep (+ 1), and 4 rep + (2, 3) hold k + 1
            if constexpr (MODE == kInput) {
                uint32_t r[8], q[8];
                tmem_load16x256_x2(ya, ya + pl.qcp, r, q);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int o = 4 * (i >> 1) + (i & 1);
                    w0[i] = pack_bf16x2(__uint_as_float(r[o]) + __uint_as_float(q[o]),
                                        __uint_as_float(r[o + 2]) + __uint_as_float(q[o + 2]));
                }
            } else {
                uint32_t r[8], q[8];
                tmem_load16x256_x2(ya, ya + pl.qcp, r, q);
                constexpr bool PRE = MODE == kPre;
                switch (act) {
                    case KRON_ACT_SILU:
                        gate_item<KRON_ACT_SILU, PRE>(r, q, bias_g, bias_u, d, w0, w1);
                        break;
                    case KRON_ACT_GELU:
                        gate_item<KRON_ACT_GELU, PRE>(r, q, bias_g, bias_u, d, w0, w1);
                        break;
                    case KRON_ACT_GELU_TANH:
                        gate_item<KRON_ACT_GELU_TANH, PRE>(r, q, bias_g, bias_u, d, w0, w1);
                        break;
                    default: gate_item<KRON_ACT_SIGMOID, PRE>(r, q, bias_g, bias_u, d, w0, w1); break;
                }
            }
            if (item == ni - 1) {
                tc_fence_before();
                mbar_arrive_warp(bar(kYEmpty + y));
            }
            if (t * NT < nlast && k_ok) {
                const size_t o = (size_t)item * item_step;
                const int left = qmax - cb;
                if (left >= 13) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = 4 * i;
                        *reinterpret_cast<uint32_t *>(p0 + o + c * pl.M2) = w0[i];
                        if constexpr (MODE == kPre)
                            *reinterpret_cast<uint32_t *>(p1 + o + c * pl.M2) = w1[i];
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = 4 * i;
                        if (c < left) {
                            *reinterpret_cast<uint32_t *>(p0 + o + c * pl.M2) = w0[i];
                            if constexpr (MODE == kPre)
                                *reinterpret_cast<uint32_t *>(p1 + o + c * pl.M2) = w1[i];
                        }
                    }
                }
            }
            __syncwarp();
            if (++item == ni) {
                item = 0;
                t += pl.groups;
                p0 += tile_step;
                if constexpr (MODE == kPre) p1 += tile_step;
                if (++y == pl.ybufs) y = 0, yph ^= 1;
            }
            return true;
        };
        if (MODE == kPre && ni > 0) {
            fetch_next(dh[0]);
            fetch_next(dh[1]);
        }
        if (ni == 0)      // no columns for this warp (qcp = 16): only the phases
            for (; t < pl.ntiles; t += pl.groups) {
                if (!warp_wait(bar(kYFull + y), yph, ab)) break;
                mbar_arrive_warp(bar(kYEmpty + y));
                if (++y == pl.ybufs) y = 0, yph ^= 1;
            }
        while (t < pl.ntiles && ni > 0) {
            if (!process(dh[0])) break;
            if constexpr (MODE == kPre) {
                fetch_next(dh[0]);
                if (t >= pl.ntiles) break;
                if (!process(dh[1])) break;
                fetch_next(dh[1]);
            }
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

// Cycles of one M = 128, K = 16 MMA with both operands in shared memory, as measured back to
// back: 74 at N = 32, 77 at 64, 85 at 128, 97 at 192, 129 at 256.  Below N = 192 reading the
// 128 rows of A is what takes the time.
static double mma_cycles(int n) { return n > 208 ? n * 0.5 : 70 + n * 0.13; }

// Chooses MP, the c slices and the ring by an estimate of the kernel's time: per chunk the
// larger of its shared-memory cycles (128 B each) and its MMA cycles and about 80 of hand-over,
// per tile at least epilogue 2's time, per CTA the packing of the factors.  More slices mean less
// packing per CTA and room for the factors, and more repeats of stage 1 and of the reads of x.
static bool find_plan(Plan *best, const Shape &s, Mode mode, int sms) {
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
            if (cdiv(p.Q, p.qc) != nqs || 2 * p.qcp > 256) continue;
            if (nqs > 1 && p.qc < 8) break;
            p.nqs = nqs;
            p.ybufs = 4 * p.qcp <= 256 ? 2 : 1;
            p.c_chunk = up(p.qcp * K2b, 1024);
            const int64_t bytes_b = (int64_t)p.nblk * 128 * p.kb;
            const int64_t bytes_c = (int64_t)p.nac * p.nblk * p.c_chunk;
            int64_t left =
                kSmemMax - (bytes_b + bytes_c + 2 * p.t_bytes + 2 * (int64_t)p.x_bytes);
            if (left < 0) continue;
            p.tbufs = p.stages = 2;
            // what is left over: a third T buffer, two more x stages, a fourth T buffer, x stages
            for (bool more = true; more;) {
                more = false;
                const bool t_next = p.tbufs < kMaxT && (p.tbufs == 2 || p.stages >= 4);
                if (t_next && left >= p.t_bytes) {
                    ++p.tbufs;
                    left -= p.t_bytes;
                    more = true;
                } else if (p.stages < kMaxStages && left >= p.x_bytes) {
                    ++p.stages;
                    left -= p.x_bytes;
                    more = true;
                }
            }
            // nothing is padded: the packing writes every byte of the operands
            p.exact = p.M1 * 2 == p.kb && p.M2 % MP == 0 && p.ranks % p.RB == 0 &&
                      p.P == p.nac * p.AC && (p.AC * p.RB) % 64 == 0 && p.qc == p.qcp &&
                      p.Q % p.qc == 0;
            p.tm_y = 512 - p.ybufs * 2 * p.qcp;
            p.dbufs = gmin(kMaxD, p.tm_y / 128);
            p.g1 = gmin(kG1, gmin(p.dbufs, p.tbufs));
            p.off_c = (int)bytes_b;
            p.off_t = (int)(bytes_b + bytes_c);
            p.off_x = p.off_t + p.tbufs * p.t_bytes;
            p.smem = p.off_x + p.stages * p.x_bytes;
            const int slices = p.nqs * p.nks;
            p.groups = (int)(tiles < sms / slices ? tiles : sms / slices);
            if (p.groups < 1) p.groups = 1;
            const double mem = 4.0 * K2 + (128.0 + N1) * p.kb / 128 + 2.0 * K2 * p.qcp / 128 +
                               (double)N1 * p.kb / 128 / p.nblk_src;
            const double mma = up(p.M1, 16) / 16 * mma_cycles(N1) + K2 / 16 * mma_cycles(p.qcp);
            // with two buffers, two groups of epilogue-1 warps work instead of three
            const double chunk = ((mem > mma ? mem : mma) + 80) * (p.g1 < kG1 ? 1.4 : 1.0);
            const double tile = p.nac * p.nblk * chunk * (MP == 16 ? 1.15 : 1.0);
            const double epi = p.qc * (mode == kPre ? 40.0 : 20.0);
            const double pack = 4000 + (bytes_b + 2.0 * bytes_c) / 2 / kThreads * 10;
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

// The search takes a microsecond and a call needs three plans: the last ones are kept.
bool tc_plan(Plan *best, const Shape &s, Mode mode, int sms) {
    struct Kept {
        Shape s;
        int mode, sms, ok;
        Plan pl;
    };
    static thread_local Kept kept[8] = {};
    static thread_local int next = 0;
    for (const Kept &k : kept)
        if (k.sms == sms && k.mode == (int)mode && k.s.N == s.N && k.s.p == s.p && k.s.q == s.q &&
            k.s.m1 == s.m1 && k.s.m2 == s.m2 && k.s.r == s.r) {
            *best = k.pl;
            return k.ok != 0;
        }
    Kept &k = kept[next];
    next = (next + 1) % 8;
    k.sms = 0;
    k.ok = find_plan(&k.pl, s, mode, sms) ? 1 : 0;
    k.s = s;
    k.mode = (int)mode;
    k.sms = sms;
    *best = k.pl;
    return k.ok != 0;
}

cudaError_t tc_run(const Plan &pl, const TcArgs &a, Mode mode, cudaStream_t st) {
    // the error word's look-up binds a context to this thread, which the encoder needs
    launch_step() = "device error word";
    int *const device_error = device_error_ptr();
    if (!device_error) return cudaErrorInvalidSymbol;
    launch_step() = "tensor map";
    CUtensorMap m0, m1;
    cudaError_t e = map_rows(&m0, a.src0, a.N, pl);
    if (e == cudaSuccess && mode == kInput) e = map_rows(&m1, a.src1, a.N, pl);
    if (e != cudaSuccess) return e;
    if (mode != kInput) m1 = m0;
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
    k.pq = pl.P * pl.Q;
    k.mm = pl.M1 * pl.M2;
    k.out_ld = pl.Q * pl.M2;
    k.device_error = device_error;
    const void *f = pl.MP == 16   ? kernel_of<16>(mode)
                    : pl.MP == 32 ? kernel_of<32>(mode)
                    : pl.MP == 64 ? kernel_of<64>(mode)
                                  : kernel_of<128>(mode);
    const size_t smem = (size_t)pl.smem + kTailBytes + 1024;
    // the limit belongs to the kernel, whoever calls it: the same for all sizes (another host
    // thread may set it between this one's setting and its launch)
    launch_step() = "shared memory size";
    e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmemMax + kTailBytes + 1024);
    if (e != cudaSuccess) return e;
    launch_step() = "kernel launch";
    int act = a.activation;
    void *params[] = {&m0, &m1, &k, &act};
    return cudaLaunchKernel(f, dim3((unsigned)(pl.groups * pl.nqs * pl.nks)), dim3(kThreads),
                            params, smem, st);
}

}  // namespace glu
}  // namespace kron
