// la_tc_decay.cu - linear attention with a decay for each head on tensor cores
// (tcgen05 + TMA): bf16 rows on 16-byte boundaries.
//
// One CTA walks over one segment of one head of one sweep (la_decay.h) for 64
// columns of z, in chunks of C = 128 tokens.  With rows x_i, y_i, z_i of the
// chunk, its n tokens (C but for a sequence's last) and the state S, forwards:
//   P    = x y^T                                    (C x C, fp32 in TMEM)
//   A_ij = a^(i-j) P_ij (j <= i), rounded to bf16   (TMEM)
//   out  = c_intra A z + c_inter a^(i+1) x S        (two accumulators, fp32)
//   S    = a^n S + c_state y^T (a^(n-1-j) z_j)
// and backwards in time the same with j >= i, a^(n-1-i) and a^(j+1).
//
// Accuracy: the decays multiply the scores and the rows of x S in fp32, never
// as a^i a^-j, which overflows.  The score and the state (as an operand) are
// each rounded to bf16 once; the state itself stays in fp32 registers, and the
// rows that enter it are exact: y as it came, a^(n-1-j) z_j as three bf16 parts
// (8 bits each), so that a state carried over thousands of tokens is as good
// as fp32 sums.
//
// Masked places hold zeros, but 0 times a z_j that is not finite is NaN: a chunk
// whose z holds such a value computes A z row by row from the tiles instead.
//
// Roles (512 threads): warp 0 loads (TMA), warps 1-3 issue the MMAs of P, of the
// outputs and of the state's increments, 4-7 decay and mask the scores, 8-11
// weigh z, 12-15 keep the state and write the outputs.  Tiles are 128-byte
// swizzled; every wait is bounded.
#include <algorithm>

#include "la_common.cuh"
#include "la_decay.h"
#include "la_pair.cuh"
#include "tc_host.h"
#include "tc_ptx.cuh"
#include "tc_kernels.cuh"

namespace la {
namespace {

using namespace tc;

constexpr int kMB = 64;                    // columns of z that a CTA takes
constexpr int kDecayThreads = 512;
constexpr int kTile = kC * 128;            // 128 rows of 64 bf16 values

struct TcSweep {
    CUtensorMap x, y, z, out;
    const float *start;
    float *end;
    int D, M, blocks;                      // blocks of kMB columns
    int transposed, backwards, has_out;
    float c_intra, c_inter, c_state;
};

struct TcDecayArgs {
    TcSweep sweep[kDecayMaxSweeps];
    const float *log_decay;
    const int *lens;
    int *err;
    int H, N, segs, seg_tokens, sums, starts, sweeps, blocks;
};

template <int DP> struct DecayCfg {
    static constexpr int SUB = DP / 64;                 // 64-column sub-tiles of x and y
    static constexpr int STAGE = (2 * SUB + 1) * kTile;
    static constexpr int NS = DP == 64 ? 3 : 2;
    static constexpr int NSNAP = DP == 64 ? 2 : 1;      // state snapshots that fit
    static constexpr int SNAP = DP * 128;
    static constexpr int OFF_ZW = NS * STAGE;           // three parts of the weighted z
    static constexpr int OFF_SNAP = OFF_ZW + 3 * kTile;
    static constexpr int OFF_TAB = OFF_SNAP + NSNAP * SNAP;
    // a^-32..a^128 (0 below 0), then a block's column factors
    static constexpr int TAB = 32 + kC + 4;
    static constexpr int OFF_COL = OFF_TAB + TAB * 4 + (16 - TAB * 4 % 16) % 16;
    static constexpr int OFF_FLAG = OFF_COL + 32 * 4;   // [4 chunks][4 warps]: z not finite
    static constexpr int NBARS = 2 * NS + 2 * 5 + 1 + 1 + 2 * 2 + 2 + 1;
    static constexpr int OFF_BAR = OFF_FLAG + 64;
    static constexpr int OFF_TSLOT = OFF_BAR + 8 * NBARS;
    static constexpr int SMEM = OFF_TSLOT + 16;
    static_assert(OFF_BAR % 8 == 0 && SMEM <= (int)kSmemMax, "shared memory budget");
    // TMEM: two buffers of P (128 columns; then A as bf16 in the first 64, A z in
    // the others) and x S (64); two increments of the state (64)
    static __device__ __forceinline__ uint32_t col_p(int b) { return 192u * b; }
    static __device__ __forceinline__ uint32_t col_az(int b) { return 192u * b + 64u; }
    static __device__ __forceinline__ uint32_t col_xs(int b) { return 192u * b + 128u; }
    static __device__ __forceinline__ uint32_t col_ds(int b) { return 384u + 64u * b; }
};

__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, uint64_t *bar, int x, int t, int h, int b) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(t), "r"(h), "r"(b), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tma_store_4d(const void *tmap, const void *src, int x, int t, int h, int b) {
    asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(tmap)),
                 "r"(smem_u32(src)), "r"(x), "r"(t), "r"(h), "r"(b)
                 : "memory");
}

__device__ __forceinline__ void state_sync() { asm volatile("bar.sync 2, 128;" ::: "memory"); }

// The output row of a chunk whose z is not finite: A z from the tiles, without
// the rows that the mask hides, and x S from TMEM (xs); the row goes where its x
// lay, after its last read of it.  Whole warps call it.
template <int DP>
__device__ __noinline__ void row_by_hand(uint8_t *xt, const uint8_t *yt, const uint8_t *zt, const float *w, uint32_t xs,
                                         int r, int rows, bool backwards, float intra, float inter) {
    uint32_t out[kMB / 2];
    const int j0 = backwards ? r : 0, j1 = r >= rows ? j0 : backwards ? rows : r + 1;
    for (int c0 = 0; c0 < kMB; c0 += 16) {
        float o[16];
        for (int i = 0; i < 16; i++) o[i] = 0.f;
        for (int j = j0; j < j1; j++) {
            float p = 0.f;
            for (int c = 0; c < DP; c += 2) {
                const uint32_t off = (c / 64) * kTile;
                const uint32_t a = *reinterpret_cast<const uint32_t *>(xt + off + sw128_offset(r, c % 64));
                const uint32_t b = *reinterpret_cast<const uint32_t *>(yt + off + sw128_offset(j, c % 64));
                p = fmaf(bf16lo(a), bf16lo(b), fmaf(bf16hi(a), bf16hi(b), p));
            }
            p = __bfloat162float(__float2bfloat16_rn(p * w[backwards ? j - r : r - j]));
            for (int i = 0; i < 16; i += 2) {
                const uint32_t z = *reinterpret_cast<const uint32_t *>(zt + sw128_offset(j, c0 + i));
                o[i] = fmaf(p, bf16lo(z), o[i]);
                o[i + 1] = fmaf(p, bf16hi(z), o[i + 1]);
            }
        }
        __syncwarp();
        uint32_t x[16];
        tmem_ld16(xs + c0, x);
        tmem_wait_ld();
        for (int i = 0; i < 8; i++)
            out[c0 / 2 + i] = r < rows ? pack_bf16x2(fmaf(intra, o[2 * i], inter * __uint_as_float(x[2 * i])),
                                                     fmaf(intra, o[2 * i + 1], inter * __uint_as_float(x[2 * i + 1])))
                                       : 0u;
    }
    for (int c = 0; c < kMB; c += 8)
        *reinterpret_cast<uint4 *>(xt + sw128_offset(r, c)) =
            make_uint4(out[c / 2], out[c / 2 + 1], out[c / 2 + 2], out[c / 2 + 3]);
}

template <int DP>
__global__ void __launch_bounds__(kDecayThreads, 1) decay_tc_kernel(const __grid_constant__ TcDecayArgs args) {
    using C = DecayCfg<DP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_TSLOT + 4);
    // neighbouring CTAs share their rows: column blocks and sweeps first, then segments, then heads
    int blk = blockIdx.x % args.blocks, k = 0;
    for (; k + 1 < args.sweeps && blk >= args.sweep[k].blocks; k++) blk -= args.sweep[k].blocks;
    const TcSweep &sw = args.sweep[k];
    const int rest = blockIdx.x / args.blocks, seg = rest % args.segs, bh = rest / args.segs;
    const int h = bh % args.H, b = bh / args.H, m0 = blk * kMB;
    const bool backwards = sw.backwards != 0, out = sw.has_out != 0;

    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *full = bar, *empty = full + C::NS, *p_full = empty + C::NS, *a_ready = p_full + 2, *xs_full = a_ready + 2,
             *o_full = xs_full + 2, *o_free = o_full + 2, *zw_ready = o_free + 2, *tail_ready = zw_ready + 1,
             *ds_full = tail_ready + 1, *ds_free = ds_full + 2, *snap_ready = ds_free + 2, *drain = snap_ready + 2;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + C::OFF_TSLOT);
    float *w = reinterpret_cast<float *>(smem + C::OFF_TAB) + 32, *colf = reinterpret_cast<float *>(smem + C::OFF_COL);
    volatile int *flag = reinterpret_cast<volatile int *>(smem + C::OFF_FLAG);
    uint8_t *zw = smem + C::OFF_ZW;
    auto snap = [&](int j) { return smem + C::OFF_SNAP + (j % C::NSNAP) * C::SNAP; };
    auto stage = [&](int it) { return smem + (it % C::NS) * C::STAGE; };
    constexpr int OFF_Y = C::SUB * kTile, OFF_Z = 2 * C::SUB * kTile;

    pdl_launch_dependents();
    if (tid == 0) {
        *abort = (smem_u32(smem) & 1023u) ? 1 : 0;   // the swizzled layouts need a 1024-byte aligned base
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], out ? 3 : 1);       // increment MMAs; output MMAs; output rows stored
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&p_full[i], 1);
            mbar_init(&a_ready[i], kGrp);
            mbar_init(&xs_full[i], 1);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_free[i], kGrp);
            mbar_init(&ds_full[i], 1);
            mbar_init(&ds_free[i], kGrp);
            mbar_init(&snap_ready[i], kGrp);
        }
        mbar_init(zw_ready, kGrp);
        mbar_init(tail_ready, kGrp);
        mbar_init(drain, 3);
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    pdl_wait_cta();   // from here on the previous launch's writes are visible
    tc_fence_after();
    const uint32_t tmem = *tslot;

    const float g = args.log_decay[h];
    const int len = args.lens ? max(0, min(args.N, args.lens[b])) : args.N;
    const int first = seg * args.seg_tokens;
    const int tokens = max(0, min(len - first, args.seg_tokens));
    const int n = (tokens + kC - 1) / kC;                       // chunks
    const int tail = tokens - (n - 1) * kC;                     // tokens of the last one
    auto chunk_of = [&](int it) { return backwards ? n - 1 - it : it; };
    auto rows_of = [&](int it) { return chunk_of(it) == n - 1 ? tail : kC; };
    for (int i = tid; i < C::TAB; i += kDecayThreads) {
        const int e = i - 32;   // a^0 is 1 also where g is -infinity
        w[e] = e < 0 ? 0.f : e == 0 ? 1.f : expf(g * (float)e);
    }
    if (tid < 32) {
        const int e = backwards ? tid : 31 - tid;
        colf[tid] = e == 0 ? 1.f : expf(g * (float)e);
    }
    __syncthreads();

    if (warp == 0) {
        // ------------------------------------------------------ producer
        if (lane == 0 && !*abort) {
            prefetch_tmap(&sw.y);
            prefetch_tmap(&sw.z);
            if (out) prefetch_tmap(&sw.x);
            int issued = 0;
            for (int it = 0; it < n; ++it) {
                const int s = it % C::NS;
                if (it >= C::NS && !wait_bar(&empty[s], (it / C::NS - 1) & 1, abort)) break;
                uint8_t *st = stage(it);
                const int t0 = first + chunk_of(it) * kC;
                mbar_arrive_expect_tx(&full[s], ((out ? 2 : 1) * C::SUB + 1) * kTile);
#pragma unroll
                for (int j = 0; j < C::SUB; ++j) {
                    if (out) tma_load_4d(st + j * kTile, &sw.x, &full[s], j * 64, t0, h, b);
                    tma_load_4d(st + OFF_Y + j * kTile, &sw.y, &full[s], j * 64, t0, h, b);
                }
                tma_load_4d(st + OFF_Z, &sw.z, &full[s], m0, t0, h, b);
                ++issued;
            }
            if (*abort)   // let the copies in flight land before the CTA exits
                for (int it = max(0, issued - C::NS); it < issued; ++it)
                    mbar_wait_bounded(&full[it % C::NS], (it / C::NS) & 1, now_ns() + kWaitNs, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ scores: P = x y^T
        if (lane == 0 && !*abort && out) {
            constexpr uint32_t ID = idesc_bf16(128, kC, 0, 0);
            for (int it = 0; it < n; ++it) {
                const int s = it % C::NS, pb = it & 1;
                if (!wait_bar(&full[s], (it / C::NS) & 1, abort)) break;
                if (rows_of(it) < kC && !wait_bar(tail_ready, 0, abort)) break;   // rows past the end are zeros now
                if (it >= 2 && !wait_bar(&o_free[pb], (it / 2 - 1) & 1, abort)) break;
                tc_fence_after();
                const uint32_t st = smem_u32(stage(it));
                const uint64_t dx = kmajor_base(st), dy = kmajor_base(st + OFF_Y);
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks)
                    mma_f16_ss(tmem + C::col_p(pb), dx + kmajor_step(ks), dy + kmajor_step(ks), ID, ks > 0);
                mma_commit(&p_full[pb]);
            }
        }
        if (lane == 0) mma_commit(drain);
    } else if (warp == 2) {
        // ------------------------------------------------------ outputs: x S, A z
        if (lane == 0 && !*abort && out) {
            constexpr uint32_t ID = idesc_bf16(128, kMB, 0, 1);
            for (int it = 0; it < n; ++it) {
                const int s = it % C::NS, pb = it & 1;
                if (!wait_bar(&full[s], (it / C::NS) & 1, abort)) break;
                if (!wait_bar(&snap_ready[it & 1], (it >> 1) & 1, abort)) break;
                if (it >= 2 && !wait_bar(&o_free[pb], (it / 2 - 1) & 1, abort)) break;
                tc_fence_after();
                const uint32_t st = smem_u32(stage(it));
                const uint64_t dx = kmajor_base(st), ds = smem_desc(smem_u32(snap(it)), 0, 1024);
#pragma unroll
                for (int ks = 0; ks < DP / 16; ++ks)
                    mma_f16_ss(tmem + C::col_xs(pb), dx + kmajor_step(ks), ds + mnmajor_step(ks), ID, ks > 0);
                mma_commit(&xs_full[pb]);
                if (!wait_bar(&a_ready[pb], (it >> 1) & 1, abort)) break;
                tc_fence_after();
                const uint64_t dz = smem_desc(st + OFF_Z, 0, 1024);
#pragma unroll
                for (int ks = 0; ks < kC / 16; ++ks)
                    mma_f16_ts(tmem + C::col_az(pb), tmem + C::col_p(pb) + ks * 8, dz + mnmajor_step(ks), ID, ks > 0);
                mma_commit(&o_full[pb]);
                mma_commit(&empty[s]);
            }
        }
        if (lane == 0) mma_commit(drain);
    } else if (warp == 3) {
        // ------------------------------------------------------ increments: y^T (weighted z)
        if (lane == 0 && !*abort) {
            constexpr uint32_t ID = idesc_bf16(128, kMB, 1, 1);
            for (int it = 0; it < n; ++it) {
                const int s = it % C::NS, db = it & 1;
                if (!wait_bar(&full[s], (it / C::NS) & 1, abort)) break;
                if (!wait_bar(zw_ready, it & 1, abort)) break;
                if (it >= 2 && !wait_bar(&ds_free[db], (it / 2 - 1) & 1, abort)) break;
                tc_fence_after();
                // y^T read MN-major; 64 columns wide it is repeated (M-atom stride 0), so
                // that lanes 64-127 hold a second copy
                const uint64_t dy = smem_desc(smem_u32(stage(it)) + OFF_Y, DP == 64 ? 0 : kTile, 1024);
#pragma unroll
                for (int part = 0; part < 3; ++part) {
                    const uint64_t dz = smem_desc(smem_u32(zw) + part * kTile, 0, 1024);
#pragma unroll
                    for (int ks = 0; ks < kC / 16; ++ks)
                        mma_f16_ss(tmem + C::col_ds(db), dy + mnmajor_step(ks), dz + mnmajor_step(ks), ID,
                                   part > 0 || ks > 0);
                }
                mma_commit(&ds_full[db]);
                mma_commit(&empty[s]);
            }
        }
        if (lane == 0) mma_commit(drain);
    } else if (warp < 8) {
        // ------------------------------------------------------ scores: decayed, masked, bf16
        const int q4 = warp & 3, r = 32 * q4 + lane;
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const float4 *col4 = reinterpret_cast<const float4 *>(colf);
        for (int it = 0; it < (out ? n : 0); ++it) {
            const int pb = it & 1;
            if (wait_bar_warp(&p_full[pb], (it >> 1) & 1, abort)) {
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < kC; c0 += 32) {
                    uint32_t a[16];
                    if (backwards ? c0 < 32 * q4 : c0 > 32 * q4) {   // hidden from every row of this warp
#pragma unroll
                        for (int j = 0; j < 16; ++j) a[j] = 0u;
                    } else {
                        float x[32];
                        tmem_ld32f(tmem + lane_off + C::col_p(pb) + c0, x);
                        if (c0 == 32 * q4) {
                            const float *wr = backwards ? w - lane : w + lane;
#pragma unroll
                            for (int j = 0; j < 32; ++j) {
                                const float f = backwards ? wr[j] : wr[-j];
                                x[j] = (backwards ? j >= lane : j <= lane) ? x[j] * f : 0.f;
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j) a[j] = pack_bf16x2(x[2 * j], x[2 * j + 1]);
                        } else {
                            // a^(distance) = a^(row to the block's near edge) a^(edge to column): no power grows
                            const float rf = backwards ? w[c0 - r] : w[r - c0 - 31];
                            const float2 rf2 = make_float2(rf, rf);
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float4 f = col4[j];
                                const float2 u = mul_pair(make_float2(x[4 * j], x[4 * j + 1]),
                                                          mul_pair(make_float2(f.x, f.y), rf2));
                                const float2 v = mul_pair(make_float2(x[4 * j + 2], x[4 * j + 3]),
                                                          mul_pair(make_float2(f.z, f.w), rf2));
                                a[2 * j] = pack_bf16x2(u.x, u.y);
                                a[2 * j + 1] = pack_bf16x2(v.x, v.y);
                            }
                        }
                    }
                    tmem_st16(tmem + lane_off + C::col_p(pb) + c0 / 2, a);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            mbar_arrive(&a_ready[pb]);
        }
    } else if (warp < 12) {
        // ------------------------------------------------------ z weighed, in three bf16 parts
        const int r = tid - 256;
        for (int it = 0; it < n; ++it) {
            const int s = it % C::NS, rows = rows_of(it);
            bool ok = wait_bar_warp(&full[s], (it / C::NS) & 1, abort);
            // the last increment has read the parts
            if (it > 0) ok = ok && wait_bar_warp(&ds_full[(it - 1) & 1], ((it - 1) >> 1) & 1, abort);
            if (ok) {
                uint8_t *st = stage(it), *zt = st + OFF_Z;
                if (rows < kC) {   // rows past the end: nothing, whatever they hold
                    if (r >= rows) {
                        for (int c = 0; c < 64; c += 8) {
                            *reinterpret_cast<uint4 *>(zt + sw128_offset(r, c)) = make_uint4(0u, 0u, 0u, 0u);
                            for (int j = 0; j < C::SUB; ++j)
                                *reinterpret_cast<uint4 *>(st + OFF_Y + j * kTile + sw128_offset(r, c)) =
                                    make_uint4(0u, 0u, 0u, 0u);
                        }
                    }
                }
                const float wr = r < rows ? w[backwards ? r + 1 : rows - 1 - r] : 0.f;
                uint32_t most = 0u;
#pragma unroll 2
                for (int c = 0; c < 64; c += 8) {
                    const uint32_t off = sw128_offset(r, c);
                    const uint4 v = *reinterpret_cast<const uint4 *>(zt + off);
                    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                    uint32_t hi[4], mid[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        most = __vmaxu2(most, in[i] & 0x7fff7fffu);
                        float2 f = mul_pair(get_pair(in[i]), make_float2(wr, wr));
                        hi[i] = put_pair(f);
                        float2 e = get_pair(hi[i]);
                        f = make_float2(f.x - e.x, f.y - e.y);
                        mid[i] = put_pair(f);
                        e = get_pair(mid[i]);
                        lo[i] = put_pair(make_float2(f.x - e.x, f.y - e.y));
                    }
                    *reinterpret_cast<uint4 *>(zw + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(zw + kTile + off) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                    *reinterpret_cast<uint4 *>(zw + 2 * kTile + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
                const bool bad = (most & 0xffffu) >= 0x7f80u || (most >> 16) >= 0x7f80u;
                const bool any = __any_sync(0xffffffffu, bad);
                if (lane == 0) flag[(it & 3) * 4 + (warp & 3)] = any;
                __threadfence_block();
            }
            fence_proxy_async();
            if (rows < kC) mbar_arrive(tail_ready);
            mbar_arrive(zw_ready);
        }
    } else {
        // ------------------------------------------------------ state and output rows
        // DP = 64: thread (q4, lane) keeps row 32 (q4 & 1) + lane of the state, columns
        // 32 (q4 / 2) on; DP = 128: row 32 q4 + lane, all columns
        constexpr int NC = DP == 64 ? 32 : 64;
        const int q4 = warp & 3, r = 32 * q4 + lane;
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const int d = DP == 64 ? 32 * (q4 & 1) + lane : r, cb = DP == 64 ? 32 * (q4 >> 1) : 0;
        const bool leader = tid == 384;
        const int D = sw.D, M = sw.M;
        const size_t DM = (size_t)D * M;
        float sv[NC];
        auto state_at = [&](const float *p, int j) {   // element of column cb + j
            return p + (sw.transposed ? (size_t)(m0 + cb + j) * D + d : (size_t)d * M + m0 + cb + j);
        };
        const float *start = args.sums || sw.start == nullptr
                                 ? nullptr
                                 : sw.start + (args.starts ? (size_t)bh * args.segs + seg : (size_t)bh) * DM;
        // 16-byte accesses where a row of the state has them
        auto wide = [&](const float *p) { return !sw.transposed && M % 4 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
        if (start && wide(start)) {
#pragma unroll
            for (int j = 0; j < NC; j += 4) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (d < D && m0 + cb + j < M) v = *reinterpret_cast<const float4 *>(state_at(start, j));
                sv[j] = v.x, sv[j + 1] = v.y, sv[j + 2] = v.z, sv[j + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int j = 0; j < NC; ++j) sv[j] = start && d < D && m0 + cb + j < M ? *state_at(start, j) : 0.f;
        }
        auto put_snap = [&](int it) {
#pragma unroll
            for (int j = 0; j < NC; j += 32) store_snap32<DP>(snap(it), d, cb + j, sv + j);
            fence_proxy_async();
            mbar_arrive(&snap_ready[it & 1]);
        };
        if (out) put_snap(0);
        const float2 kept_whole = kept(g, kC), kept_tail = kept(g, tail);
        for (int it = 0; it < n; ++it) {
            const int db = it & 1, pb = it & 1, rows = rows_of(it);
            bool ok = wait_bar_warp(&ds_full[db], (it >> 1) & 1, abort);
            if (ok) {
                tc_fence_after();
                const float2 a = rows == kC ? kept_whole : kept_tail;
#pragma unroll
                for (int j = 0; j < NC; j += 16) {
                    uint32_t v[16];
                    tmem_ld16(tmem + lane_off + C::col_ds(db) + cb + j, v);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        sv[j + i] = fmaf(sw.c_state, __uint_as_float(v[i]), keep(a, sv[j + i]));
                }
            }
            tc_fence_before();
            mbar_arrive(&ds_free[db]);
            if (!out) continue;
            // the snapshot of chunk it - 1 was read before its output rows were, with
            // room for one alone chunk it's has to be read first
            if (C::NSNAP == 1) ok = ok && wait_bar_warp(&xs_full[pb], (it >> 1) & 1, abort);
            if (it + 1 < n) put_snap(it + 1);
            ok = ok && wait_bar_warp(&o_full[pb], (it >> 1) & 1, abort);
            uint8_t *st = stage(it);   // x is dead: its first sub-tile takes the output rows
            if (ok) {
                tc_fence_after();
                const volatile int *f = flag + (it & 3) * 4;
                const bool by_hand = f[0] | f[1] | f[2] | f[3];
                const float inter = sw.c_inter * w[r < rows ? (backwards ? rows - 1 - r : r + 1) : 0];
                if (by_hand) {
                    row_by_hand<DP>(st, st + OFF_Y, st + OFF_Z, w, tmem + lane_off + C::col_xs(pb), r, rows, backwards,
                                    sw.c_intra, inter);
                } else {
#pragma unroll
                    for (int c0 = 0; c0 < kMB; c0 += 16) {
                        uint32_t az[16], xs[16], o[8];
                        tmem_ld16(tmem + lane_off + C::col_az(pb) + c0, az);
                        tmem_ld16(tmem + lane_off + C::col_xs(pb) + c0, xs);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float u = fmaf(sw.c_intra, __uint_as_float(az[2 * i]), inter * __uint_as_float(xs[2 * i]));
                            const float v =
                                fmaf(sw.c_intra, __uint_as_float(az[2 * i + 1]), inter * __uint_as_float(xs[2 * i + 1]));
                            o[i] = r < rows ? pack_bf16x2(u, v) : 0u;
                        }
                        *reinterpret_cast<uint4 *>(st + sw128_offset(r, c0)) = make_uint4(o[0], o[1], o[2], o[3]);
                        *reinterpret_cast<uint4 *>(st + sw128_offset(r, c0 + 8)) = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
            }
            tc_fence_before();
            mbar_arrive(&o_free[pb]);
            fence_proxy_async();
            state_sync();
            if (leader) {
                if (ok) {
                    tma_store_4d(&sw.out, st, m0, first + chunk_of(it) * kC, h, b);
                    tma_store_commit();
                }
                tma_store_wait_read0();
                mbar_arrive(&empty[it % C::NS]);
            }
        }
        // chunks past the length: rows of zeros (no load is on its way any more)
        const int chunks = (min(first + args.seg_tokens, args.N) - first + kC - 1) / kC;
        if (out && n < chunks) {
            state_sync();   // the leader's last store has read its tile
            for (int c = 0; c < 64; c += 8) *reinterpret_cast<uint4 *>(smem + sw128_offset(r, c)) = make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async();
            state_sync();
            if (leader && !*abort) {
                for (int c = n; c < chunks; ++c) tma_store_4d(&sw.out, smem, m0, first + c * kC, h, b);
                tma_store_commit();
            }
        }
        if (leader && out) tma_store_wait_all0();
        // the state leaves where the sequence's last segment (backwards: its first) ends
        const int last = max(0, (len + args.seg_tokens - 1) / args.seg_tokens - 1);
        if (sw.end && !*abort && (args.sums || seg == (backwards ? 0 : last))) {
            float *end = sw.end + (args.sums ? (size_t)bh * args.segs + seg : (size_t)bh) * DM;
            if (wide(end)) {
#pragma unroll
                for (int j = 0; j < NC; j += 4)
                    if (d < D && m0 + cb + j < M)
                        *reinterpret_cast<float4 *>(const_cast<float *>(state_at(end, j))) =
                            make_float4(sv[j], sv[j + 1], sv[j + 2], sv[j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < NC; ++j)
                    if (d < D && m0 + cb + j < M) *const_cast<float *>(state_at(end, j)) = sv[j];
            }
        }
    }
    // no MMA may still be running when the CTA frees its TMEM
    if (tid == 0) mbar_wait_bounded(drain, 0, now_ns() + kWaitNs, nullptr);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 3) tmem_dealloc(tmem, 512);
    if (tid == 0 && *abort) record_error(args.err, kErrTimeout);
}

// 16-byte rows: base and strides; dimensions of one do not move.
bool mappable(const la_view &v, int B, int H, int N) {
    auto ok = [](long long stride, int n) { return n <= 1 || (stride % 8 == 0 && stride > 0 && stride < (1LL << 38)); };
    return v.data == nullptr ||
           ((reinterpret_cast<uintptr_t>(v.data) & 15) == 0 && ok(v.sb, B) && ok(v.sh, H) && ok(v.sn, N));
}

// Tensor map of [B][H][N][cols] with the view's strides, boxes of 64 columns x
// 128 rows.  Columns and rows past the tensor read as zeros and are not written.
bool map_of(CUtensorMap *m, const la_view &v, int cols, const DecayLaunch &l) {
    auto fn = encode_fn();
    if (!fn) return false;
    auto bytes = [](long long stride, int n) { return (cuuint64_t)(n > 1 ? stride * 2 : 16); };
    cuuint64_t dims[4] = {(cuuint64_t)cols, (cuuint64_t)l.N, (cuuint64_t)l.H, (cuuint64_t)l.B};
    cuuint64_t strides[3] = {bytes(v.sn, l.N), bytes(v.sh, l.H), bytes(v.sb, l.B)};
    cuuint32_t box[4] = {64, (cuuint32_t)kC, 1, 1}, step[4] = {1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.data, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

template <int DP> cudaError_t launch(const TcDecayArgs &a, long long ctas, cudaStream_t stream) {
    using C = DecayCfg<DP>;
    cudaError_t e = set_smem(decay_tc_kernel<DP>, C::SMEM);
    if (e != cudaSuccess) return e;
    e = launch_pdl(decay_tc_kernel<DP>, dim3((unsigned)ctas), dim3(kDecayThreads), C::SMEM, stream, 0u, a);
    count_launches(1);
    return e;
}

}  // namespace

bool tc_decay_supported(const DecayLaunch &l, la_dtype dtype) {
    if (dtype != LA_DTYPE_BF16) return false;
    for (int i = 0; i < l.sweeps; i++) {
        const DecaySweep &s = l.sweep[i];
        for (const la_view *v : {&s.x, &s.y, &s.z, &s.out})
            if (!mappable(*v, l.B, l.H, l.N)) return false;
    }
    return true;
}

cudaError_t tc_decay(const DecayLaunch &l) {
    const DeviceInfo *dev = device_info();
    if (!dev) return cudaErrorInvalidDevice;
    TcDecayArgs a{};
    int D = 0;
    for (int i = 0; i < l.sweeps; i++) {
        const DecaySweep &s = l.sweep[i];
        TcSweep &t = a.sweep[i];
        if (!map_of(&t.y, s.y, s.D, l) || !map_of(&t.z, s.z, s.M, l)) return cudaErrorInvalidValue;
        if (s.out.data && (!map_of(&t.x, s.x, s.D, l) || !map_of(&t.out, s.out, s.M, l))) return cudaErrorInvalidValue;
        t.start = s.start, t.end = s.end, t.D = s.D, t.M = s.M, t.blocks = (s.M + kMB - 1) / kMB;
        t.transposed = s.transposed, t.backwards = s.backwards, t.has_out = s.out.data != nullptr;
        t.c_intra = s.c_intra, t.c_inter = s.c_inter, t.c_state = s.c_state;
        a.blocks += t.blocks;
        D = std::max(D, s.D);
    }
    a.log_decay = l.log_decay, a.lens = l.lens, a.err = dev->err_word;
    a.H = l.H, a.N = l.N, a.segs = l.segs, a.seg_tokens = l.seg_tokens, a.sums = l.sums, a.starts = l.starts;
    a.sweeps = l.sweeps;
    const long long ctas = (long long)l.B * l.H * l.segs * a.blocks;
    return D <= 64 ? launch<64>(a, ctas, l.stream) : launch<128>(a, ctas, l.stream);
}

}  // namespace la
