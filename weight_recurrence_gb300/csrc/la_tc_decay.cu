// la_tc_decay.cu - linear attention with a decay for each head on tensor cores
// (tcgen05 + TMA): bf16 rows on 16-byte boundaries (the inputs'; outputs lie as they
// may).
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
// each rounded to bf16 once, the type that the tensor cores multiply with rows
// that are bf16 themselves: outputs, rounded to bf16 too, are 0.0023 of their root
// mean square off the sums in 64 bits, where their own rounding alone is 0.0017
// (16 x 8 heads of 4096 tokens).  Two parts of each would take that off for as
// many MMAs again as the outputs take, and a second snapshot's room.  The state
// itself stays in fp32 registers, and the
// rows that enter it are exact: y as it came, a^(n-1-j) z_j as three bf16 parts
// of 8 bits each, so that a state carried over thousands of tokens is as good as
// fp32 sums.  Two parts (16 bits) where no state leaves: bf16 outputs alone see it.
//
// Masked places hold zeros, but 0 times a z_j that is not finite is NaN.  Such
// values are taken out of z (not out of the parts that enter the state), and the
// outputs that see them are made NaN.
//
// Roles (640 threads): warp 0 loads (TMA); warps 1, 2 and 3 issue the MMAs of P, of
// the outputs (x S, A z) and of the state's increments.  Two groups of four warps
// (4-11) decay and mask the scores and make the output rows, each for half of the
// columns, and store them from registers; two more (12-19) weigh z, by halves of its
// rows, and keep the state.  Tiles are 128-byte swizzled; every wait is bounded.
//
// 64 columns of z a CTA: the three parts of z, two snapshots and three chunks of
// tiles fill the shared memory (one snapshot, two chunks at 128 channels); 128
// columns would leave one chunk.  The CTAs of a head's column blocks and of the
// backward's three sweeps are neighbours and share their rows through the L2.
//
// Measured: 128 heads of 4096 tokens, D = M = 64, forward 76 us (272 MB, 3.6 TB/s,
// 113 TFLOP/s); 16 heads of 65536 tokens, D = M = 128, in 9 segments 491 us; the
// backward's three sweeps of 128 heads of 2048 tokens 105 us.  A chunk takes about
// 3900 clocks, of which HBM would need 2800 (all SMs at the copy's rate), the tensor
// pipe 850, issue 2100.  No unit is full: the weighing of z (14 us of 72 where it was
// left out), the outputs (12), the scores (4) and the increments share the issue slots
// and the shared memory's bandwidth (about 300 KB a chunk).  A CTA's start and end
// take as long as six chunks.
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
constexpr int kDecayThreads = 640;
constexpr int kTile = kC * 128;            // 128 rows of 64 bf16 values

struct TcSweep {
    CUtensorMap x, y, z;
    la_view rows;                          // the output's
    const float *start;
    float *end;
    int D, M, blocks;                      // blocks of kMB columns
    int transposed, backwards, has_out;
    int shared;                            // bits 2 i (heads) and 2 i + 1 (sequences): all of x, y, z's are one
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
    static constexpr int NS = DP == 64 ? 3 : 2;         // chunks whose tiles are held
    static constexpr int NSNAP = DP == 64 ? 2 : 1;      // state snapshots that fit
    static constexpr int SNAP = DP * 128;
    static constexpr int OFF_X = 0;
    static constexpr int OFF_Y = OFF_X + NS * SUB * kTile;
    static constexpr int OFF_Z = OFF_Y + NS * SUB * kTile;
    static constexpr int OFF_ZW = OFF_Z + NS * kTile;   // three parts of the weighted z
    static constexpr int OFF_SNAP = OFF_ZW + 3 * kTile;
    static constexpr int OFF_TAB = OFF_SNAP + NSNAP * SNAP;
    // decays by 0..128 tokens, then the factors of a block's columns, then those of a
    // block on the diagonal by column - row, from -31 on
    static constexpr int TAB = kC + 4;
    static constexpr int OFF_COL = OFF_TAB + TAB * 4;
    static constexpr int OFF_DIAG = OFF_COL + 32 * 4;
    // chunks whose record of values of z that are not finite is held: chunk j's is
    // written again for chunk j + NBAD, which needs z's tile of chunk j + NBAD - NS, so
    // that chunk's A z and the output rows of the chunk before it
    static constexpr int NBAD = 4;
    static constexpr int OFF_FLAG = OFF_DIAG + 64 * 4;     // [NBAD][2 halves][8 warps]
    static constexpr int OFF_BAD = OFF_FLAG + NBAD * 64;   // [NBAD][2][8][16 columns]: first or last row, a byte
    static constexpr int OFF_BAR = OFF_BAD + NBAD * 256;
    static constexpr int NBARS = 6 * NS + 5 * 2 + 4 + 1 + 6 + 2 + 1;
    static constexpr int OFF_TSLOT = OFF_BAR + 8 * NBARS;
    static constexpr int SMEM = OFF_TSLOT + 16;
    static_assert(NBAD > NS && OFF_BAR % 8 == 0 && SMEM <= (int)kSmemMax, "shared memory budget");
    // TMEM: two buffers of P (128 columns; the scores as bf16 take the first half of
    // each 64), x S and A z (64 each), and two of the state's increment (64 each)
    static __device__ __forceinline__ uint32_t col_p(int b) { return 128u * b; }
    static constexpr uint32_t COL_XS = 256, COL_AZ = 320, COL_DS = 384;
};

__device__ __forceinline__ void tma_load_4d(void *dst, const void *tmap, uint64_t *bar, int x, int t, int h, int b) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(x), "r"(t), "r"(h), "r"(b), "r"(smem_u32(bar))
        : "memory");
}
// 32 lanes x 32 bit, 8 consecutive columns a thread.
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}

// A wait that may sleep in the barrier's hardware for up to about 20 us at a time.
// Out of line but for the first try: the roles share one instruction cache.
__device__ __forceinline__ bool try_wait_long(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(20000u)
        : "memory");
    return ok != 0;
}
__device__ __noinline__ bool wait_long(uint64_t *bar, uint32_t parity, volatile int *abort) {
    const uint64_t deadline = now_ns() + kWaitNs;
    while (!*abort) {
        if (try_wait_long(bar, parity)) return true;
        if (now_ns() > deadline) *abort = 1;
    }
    return false;
}
// As wait_bar and wait_bar_warp; a role that gave up raises the abort flag for the others.
__device__ __forceinline__ bool wait_one(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return mbar_try_wait(bar, parity) || wait_long(bar, parity, abort);
}
__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, volatile int *abort) {
    return __all_sync(0xffffffffu, wait_one(bar, parity, abort));
}

// True in one lane of a converged warp.  The MMAs are issued under it by warps that
// walk through their loops as a whole: descriptors then stay in uniform registers
// and an MMA goes out every few clocks; issued by a lane that runs alone, each took 97.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// One arrival for a warp, whose lanes have each done what it stands for (and their
// fences).
__device__ __forceinline__ void arrive_warp(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

__device__ __forceinline__ float2 pair_at(const uint32_t (&v)[16], int i) {
    return make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
}

// The upper halves of two fp32 values: bf16, cut off.
__device__ __forceinline__ uint32_t top_pair(float2 v) {
    return __byte_perm(__float_as_uint(v.x), __float_as_uint(v.y), 0x7632);
}

// Rows of z (16 columns from c0 on) with values that are not finite (any lane of the
// warp has one): they become zeros in the tile, and the warp notes for every column its
// first (backwards: last) row that had one, 255 (0: row + 1) for none.
__device__ __noinline__ void take_out(uint8_t *zt, int r, int c0, uint8_t *note, bool backwards) {
    const int lane = threadIdx.x & 31;
    for (int c = 0; c < 16; ++c) {
        uint16_t *p = reinterpret_cast<uint16_t *>(zt + sw128_offset(r, c0 + c));
        const bool bad = (*p & 0x7fffu) >= 0x7f80u;
        if (bad) *p = 0;
        const uint32_t who = __ballot_sync(0xffffffffu, bad);
        if (lane == 0) {
            const int row = r + (backwards ? 31 - __clz(who) : __ffs(who) - 1);
            note[c] = who == 0u ? (backwards ? 0 : 255) : backwards ? row + 1 : row;
        }
    }
}

// Which of the columns 32 grp..32 grp + 31 of row r see one of them; note: [2][8][16],
// flag: [2][8].  Warps 2q and 2q + 1 wrote columns 16q..16q + 15.
__device__ __noinline__ uint32_t seen_bad(int r, int grp, const uint8_t *note, const volatile int *flag, bool backwards) {
    uint32_t hit = 0u;
    for (int i = 0; i < 16; ++i) {
        const int q = (i & 7) >> 1;
        if (!flag[i] || q >> 1 != grp) continue;
        for (int c = 0; c < 16; ++c)
            if (backwards ? note[i * 16 + c] > r : note[i * 16 + c] <= r) hit |= 1u << (16 * (q & 1) + c);
    }
    return hit;
}

// 16 output values to a row, `cols` of them.
__device__ __noinline__ void store_some(__nv_bfloat16 *row, uint4 a, uint4 b, int cols) {
    for (int i = 0; i < min(cols, 16); i += 8) {
        const uint4 v = i == 0 ? a : b;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t pair = j < 2 ? v.x : j < 4 ? v.y : j < 6 ? v.z : v.w;
            if (i + j < cols) reinterpret_cast<uint16_t *>(row)[i + j] = (uint16_t)(j & 1 ? pair >> 16 : pair);
        }
    }
}
__device__ __forceinline__ void store16(__nv_bfloat16 *row, uint4 a, uint4 b, int cols) {
    if (cols < 16 || (reinterpret_cast<uintptr_t>(row) & 15)) {
        store_some(row, a, b, cols);
    } else if ((reinterpret_cast<uintptr_t>(row) & 31) == 0) {   // a whole 32-byte sector
        st_global_v8(row, a, b);
    } else {
        reinterpret_cast<uint4 *>(row)[0] = a;
        reinterpret_cast<uint4 *>(row)[1] = b;
    }
}

template <int DP>
__global__ void __launch_bounds__(kDecayThreads, 1) decay_tc_kernel(const __grid_constant__ TcDecayArgs args) {
    using C = DecayCfg<DP>;
    extern __shared__ __align__(1024) uint8_t smem[];
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    volatile int *abort = reinterpret_cast<volatile int *>(smem + C::OFF_TSLOT + 4);
    // neighbouring CTAs share their rows: column blocks and sweeps first, then segments, then heads
    int blk = blockIdx.x % args.blocks, k = 0;
    for (; k + 1 < args.sweeps && blk >= args.sweep[k].blocks; k++) blk -= args.sweep[k].blocks;
    const TcSweep &sw = args.sweep[k];
    const int rest = blockIdx.x / args.blocks, seg = rest % args.segs, bh = rest / args.segs;
    const int h = bh % args.H, b = bh / args.H, m0 = blk * kMB;
    const bool backwards = sw.backwards != 0, out = sw.has_out != 0;
    if (args.sums && seg == (backwards ? 0 : args.segs - 1)) {   // nobody asks for that one
        pdl_wait();
        return;
    }
    // a state that leaves is exact; one that bf16 outputs alone see takes two parts of z
    const int parts = sw.end != nullptr ? 3 : 2;

    constexpr int kPair = 8;   // warps of a pair of groups
    uint64_t *bar = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);
    uint64_t *x_full = bar, *x_empty = x_full + C::NS, *y_full = x_empty + C::NS, *y_empty = y_full + C::NS,
             *z_full = y_empty + C::NS, *z_empty = z_full + C::NS;
    uint64_t *p_full = z_empty + C::NS, *a_ready = p_full + 2, *xs_full = a_ready + 2, *o_full = xs_full + 2,
             *o_free = o_full + 2, *zw_ready = o_free + 2, *tail_ready = zw_ready + 4, *half_ready = tail_ready + 1,
             *half_free = half_ready + 1, *ds_full = half_free + 1, *ds_free = ds_full + 2, *snap_ready = ds_free + 2,
             *drain = snap_ready + 2;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(smem + C::OFF_TSLOT);
    float *w = reinterpret_cast<float *>(smem + C::OFF_TAB), *colf = reinterpret_cast<float *>(smem + C::OFF_COL);
    float *diag = reinterpret_cast<float *>(smem + C::OFF_DIAG) + 31;
    volatile int *flag = reinterpret_cast<volatile int *>(smem + C::OFF_FLAG);
    uint8_t *zw = smem + C::OFF_ZW;
    auto snap = [&](int j) { return smem + C::OFF_SNAP + (j % C::NSNAP) * C::SNAP; };
    auto xtile = [&](int it) { return smem + C::OFF_X + (it % C::NS) * C::SUB * kTile; };
    auto ytile = [&](int it) { return smem + C::OFF_Y + (it % C::NS) * C::SUB * kTile; };
    auto ztile = [&](int it) { return smem + C::OFF_Z + (it % C::NS) * kTile; };

    pdl_launch_dependents();
    if (tid == 0) {
        *abort = (smem_u32(smem) & 1023u) ? 1 : 0;   // the swizzled layouts need a 1024-byte aligned base
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(&x_full[s], 1);
            mbar_init(&x_empty[s], 2);               // MMAs of P and of x S
            mbar_init(&y_full[s], 1);
            mbar_init(&y_empty[s], out ? 2 : 1);     // of the increment and of P
            mbar_init(&z_full[s], 1);
            mbar_init(&z_empty[s], out ? 2 : 1);     // of the increment and of A z
        }
        // where a waiter may be a chunk behind, a barrier for each of two (or four, for
        // the weighed z: up to NS chunks) chunks, so that none is two phases ahead of it
        for (int i = 0; i < 2; ++i) {
            mbar_init(&p_full[i], 1);
            mbar_init(&a_ready[i], kPair);
            mbar_init(&xs_full[i], 1);
            mbar_init(&o_full[i], 1);
            mbar_init(&o_free[i], kPair);
            mbar_init(&snap_ready[i], kPair);
            mbar_init(&ds_full[i], 1);
            mbar_init(&ds_free[i], kPair);
        }
        for (int i = 0; i < 4; ++i) mbar_init(&zw_ready[i], kPair);
        mbar_init(half_ready, kPair);
        mbar_init(half_free, 1);
        mbar_init(tail_ready, kPair);
        mbar_init(drain, 3);
        fence_mbar_init();
    }
    if (warp == 3) {
        tmem_alloc(tslot, 512);
        tmem_relinquish();
    }
    if (tid == 32) {
        prefetch_tmap(&sw.y);
        prefetch_tmap(&sw.z);
        if (out) prefetch_tmap(&sw.x);
    }
    tc_fence_before();
    pdl_wait_cta();   // from here on the previous launch's writes are visible
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tslot, 0);

    const float g = args.log_decay[h];
    const int len = args.lens ? max(0, min(args.N, args.lens[b])) : args.N;
    const int first = seg * args.seg_tokens;
    const int tokens = __shfl_sync(0xffffffffu, max(0, min(len - first, args.seg_tokens)), 0);
    const int n = (tokens + kC - 1) / kC;                       // chunks
    const int tail = tokens - (n - 1) * kC;                     // tokens of the last one
    auto chunk_of = [&](int it) { return backwards ? n - 1 - it : it; };
    auto rows_of = [&](int it) { return chunk_of(it) == n - 1 ? tail : kC; };
    auto decayed = [&](int e) { return e == 0 ? 1.f : expf(g * (float)e); };   // a^0 is 1 also where g is -infinity
    // warp 0 goes on to the loads
    if (tid >= 32 && tid <= 32 + kC) w[tid - 32] = decayed(tid - 32);
    else if (tid >= 192 && tid < 224) colf[tid - 192] = decayed(backwards ? tid - 192 : 223 - tid);
    else if (tid >= 224 && tid < 288) {
        const int e = backwards ? tid - 224 - 31 : 31 - (tid - 224);   // hidden places: 0
        diag[tid - 224 - 31] = e < 0 ? 0.f : decayed(e);
    }
    if (warp > 0) asm volatile("bar.sync 2, 608;" ::: "memory");

    if (warp == 0) {
        // ------------------------------------------------------ loads
        if (lane == 0 && !*abort) {
            int ny = 0, nx = 0, nz = 0;
            const int hx = sw.shared & 1 ? 0 : h, bx = sw.shared & 2 ? 0 : b, hy = sw.shared & 4 ? 0 : h;
            const int by = sw.shared & 8 ? 0 : b, hz = sw.shared & 16 ? 0 : h, bz = sw.shared & 32 ? 0 : b;
            for (int it = 0; it < n; ++it) {
                const int s = it % C::NS, t0 = first + chunk_of(it) * kC;
                const uint32_t again = (it / C::NS - 1) & 1;
                if (it >= C::NS && !wait_one(&y_empty[s], again, abort)) break;
                mbar_arrive_expect_tx(&y_full[s], C::SUB * kTile);
#pragma unroll
                for (int j = 0; j < C::SUB; ++j) tma_load_4d(ytile(it) + j * kTile, &sw.y, &y_full[s], j * 64, t0, hy, by);
                ++ny;
                if (out) {
                    if (it >= C::NS && !wait_one(&x_empty[s], again, abort)) break;
                    mbar_arrive_expect_tx(&x_full[s], C::SUB * kTile);
#pragma unroll
                    for (int j = 0; j < C::SUB; ++j)
                        tma_load_4d(xtile(it) + j * kTile, &sw.x, &x_full[s], j * 64, t0, hx, bx);
                    ++nx;
                }
                if (it >= C::NS && !wait_one(&z_empty[s], again, abort)) break;
                mbar_arrive_expect_tx(&z_full[s], kTile);
                tma_load_4d(ztile(it), &sw.z, &z_full[s], m0, t0, hz, bz);
                ++nz;
            }
            if (*abort) {   // let the copies in flight land before the CTA exits
                auto land = [&](uint64_t *full, int issued) {
                    for (int it = max(0, issued - C::NS); it < issued; ++it)
                        mbar_wait_bounded(&full[it % C::NS], (it / C::NS) & 1, now_ns() + kWaitNs, nullptr);
                };
                land(y_full, ny);
                land(x_full, nx);
                land(z_full, nz);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------ scores: P = x y^T
        if (out) {
            constexpr uint32_t ID = idesc_bf16(128, kC, 0, 0);
            for (int it = 0; it < n; ++it) {
                const int s = it % C::NS, pb = it & 1;
                const uint32_t turn = (it / C::NS) & 1;
                if (!wait_warp(&y_full[s], turn, abort) || !wait_warp(&x_full[s], turn, abort)) break;
                if (rows_of(it) < kC && !wait_warp(tail_ready, 0, abort)) break;   // rows past the end are zeros now
                // the scores of two chunks before were read
                if (it >= 2 && !wait_warp(&o_full[pb], (it / 2 - 1) & 1, abort)) break;
                tc_fence_after();
                const uint64_t dx = kmajor_base(smem_u32(xtile(it))), dy = kmajor_base(smem_u32(ytile(it)));
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < DP / 16; ++ks)
                        mma_f16_ss(tmem + C::col_p(pb), dx + kmajor_step(ks), dy + kmajor_step(ks), ID, ks > 0);
                    mma_commit(&p_full[pb]);
                    mma_commit(&x_empty[s]);
                    mma_commit(&y_empty[s]);
                }
            }
        }
        if (elect_one()) mma_commit(drain);
    } else if (warp == 3) {
        // ------------------------------------------------------ increments: y^T (weighted z)
        {
            constexpr uint32_t ID = idesc_bf16(128, kMB, 1, 1);
            for (int it = 0; it < n; ++it) {
                const int s = it % C::NS;
                if (!wait_warp(&y_full[s], (it / C::NS) & 1, abort)) break;
                // the increment of two chunks before has been added to the state
                if (it >= 2 && !wait_warp(&ds_free[it & 1], (it / 2 - 1) & 1, abort)) break;
                // y^T read MN-major; 64 columns wide it is repeated (M-atom stride 0), so
                // that lanes 64-127 hold a second copy.  By halves of the rows, so that the
                // first half's parts can be written anew while the second's are multiplied
                const uint64_t dy = smem_desc(smem_u32(ytile(it)), DP == 64 ? 0 : kTile, 1024);
                const uint64_t dz = smem_desc(smem_u32(zw), 0, 1024);
                constexpr uint64_t part = kTile >> 4;
                const uint32_t to = tmem + C::COL_DS + kMB * (it & 1);
                bool ok = true;
#pragma unroll 1
                for (int k0 = 0; k0 < kC / 16 && ok; k0 += kC / 32) {
                    ok = k0 == 0 ? wait_warp(half_ready, it & 1, abort) : wait_warp(&zw_ready[it & 3], (it >> 2) & 1, abort);
                    if (!ok) break;
                    tc_fence_after();
                    if (elect_one()) {
#pragma unroll
                        for (int i = 0; i < kC / 32; ++i) {
                            const uint64_t step = mnmajor_step(1) * (uint64_t)(k0 + i);
                            mma_f16_ss(to, dy + step, dz + step, ID, k0 + i > 0);
                            mma_f16_ss(to, dy + step, dz + part + step, ID, 1);
                        }
                        if (parts == 3)
#pragma unroll
                            for (int i = 0; i < kC / 32; ++i) {
                                const uint64_t step = mnmajor_step(1) * (uint64_t)(k0 + i);
                                mma_f16_ss(to, dy + step, dz + 2 * part + step, ID, 1);
                            }
                        if (k0 == 0) mma_commit(half_free);
                    }
                }
                if (!ok) break;
                if (elect_one()) {
                    mma_commit(&ds_full[it & 1]);
                    mma_commit(&y_empty[s]);
                    mma_commit(&z_empty[s]);
                }
            }
        }
        if (elect_one()) mma_commit(drain);
    } else if (warp == 2) {
        // ------------------------------------------------------ outputs: x S, A z
        if (out) {
            constexpr uint32_t ID = idesc_bf16(128, kMB, 0, 1);
            for (int it = 0; it < n; ++it) {
                const int s = it % C::NS, pb = it & 1;
                if (!wait_warp(&x_full[s], (it / C::NS) & 1, abort)) break;
                if (!wait_warp(&snap_ready[it & 1], (it >> 1) & 1, abort)) break;
                // the output rows of the chunk before have read x S and A z
                if (it >= 1 && !wait_warp(&o_free[(it - 1) & 1], ((it - 1) >> 1) & 1, abort)) break;
                tc_fence_after();
                const uint64_t dx = kmajor_base(smem_u32(xtile(it))), ds = smem_desc(smem_u32(snap(it)), 0, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < DP / 16; ++ks)
                        mma_f16_ss(tmem + C::COL_XS, dx + kmajor_step(ks), ds + mnmajor_step(ks), ID, ks > 0);
                    mma_commit(&xs_full[pb]);
                    mma_commit(&x_empty[s]);
                }
                // z has no value left that is not finite, and the scores are decayed
                if (!wait_warp(&z_full[s], (it / C::NS) & 1, abort)) break;
                if (!wait_warp(&zw_ready[it & 3], (it >> 2) & 1, abort)) break;
                if (!wait_warp(&a_ready[pb], (it >> 1) & 1, abort)) break;
                tc_fence_after();
                const uint64_t dz = smem_desc(smem_u32(ztile(it)), 0, 1024);
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < kC / 16; ++ks)
                        mma_f16_ts(tmem + C::COL_AZ, tmem + C::col_p(pb) + (ks / 4) * 64 + (ks % 4) * 8, dz + mnmajor_step(ks), ID,
                                   ks > 0);
                    mma_commit(&o_full[pb]);
                    mma_commit(&z_empty[s]);
                }
            }
        }
        if (elect_one()) mma_commit(drain);
    } else if (warp < 12) {
        // ------------------------------------------------------ scores, output rows
        const int q4 = warp & 3, r = 32 * q4 + lane, grp = warp >= 8;
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const float4 *col4 = reinterpret_cast<const float4 *>(colf);
        const float2 intra2 = make_float2(sw.c_intra, sw.c_intra);
        __nv_bfloat16 *rows_out = static_cast<__nv_bfloat16 *>(sw.rows.data) + b * sw.rows.sb + h * sw.rows.sh + m0 + 32 * grp;
        const int cols = sw.M - m0 - 32 * grp;
        // scores of columns 64 grp..64 grp + 63, decayed, masked, rounded to bf16: over the
        // first half of P's own columns, which this thread alone reads
        auto scores = [&](int it) {
            const int pb = it & 1;
            if (wait_warp(&p_full[pb], (it >> 1) & 1, abort)) {
                tc_fence_after();
                const uint32_t tp = tmem + lane_off + C::col_p(pb) + 64 * grp;
#pragma unroll 1
                for (int i = 0; i < 64; i += 16) {
                    const int c0 = 64 * grp + i, block = c0 >> 5;
                    uint32_t x[16], a[8];
                    if (backwards ? block < q4 : block > q4) {   // hidden from every row of this warp
#pragma unroll
                        for (int j = 0; j < 8; ++j) a[j] = 0u;
                    } else {
                        tmem_ld16(tp + i, x);
                        if (block != q4) {
                            // a^(distance) = a^(row to the block's near edge) a^(edge to column): no power grows
                            const float rf = backwards ? w[32 * block - r] : w[r - 32 * block - 31];
                            const float2 rf2 = make_float2(rf, rf);
                            const float4 *f4 = col4 + (i & 16) / 4;
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const float4 f = f4[j];
                                const float2 t = mul_pair(pair_at(x, 4 * j), mul_pair(make_float2(f.x, f.y), rf2));
                                const float2 u = mul_pair(pair_at(x, 4 * j + 2), mul_pair(make_float2(f.z, f.w), rf2));
                                a[2 * j] = pack_bf16x2(t.x, t.y);
                                a[2 * j + 1] = pack_bf16x2(u.x, u.y);
                            }
                        } else {
                            // a select hides what is behind the row's own column (0 times a score
                            // that is not finite is NaN)
                            const float *f = diag + (c0 - r);
                            const int k = backwards ? r - c0 : c0 - r;
                            tmem_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; j += 2) {
                                const float u = __uint_as_float(x[j]) * f[j], v = __uint_as_float(x[j + 1]) * f[j + 1];
                                a[j / 2] = pack_bf16x2(backwards ? (j >= k ? u : 0.f) : (j <= -k ? u : 0.f),
                                                       backwards ? (j + 1 >= k ? v : 0.f) : (j + 1 <= -k ? v : 0.f));
                            }
                        }
                    }
                    tmem_st8(tp + i / 2, a);
                }
                tmem_wait_st();
            }
            tc_fence_before();
            arrive_warp(&a_ready[pb]);
        };
        // output columns 32 grp..32 grp + 31
        auto output = [&](int it) {
            const int pb = it & 1, rows = rows_of(it), t = first + chunk_of(it) * kC + r;
            const bool ok = wait_warp(&o_full[pb], (it >> 1) & 1, abort);
            uint32_t hit = 0u;
            if (ok) {
                tc_fence_after();
                const volatile int *f = flag + it % C::NBAD * 16;
                if (__builtin_expect(__any_sync(0xffffffffu, f[lane & 15]), 0))
                    hit = seen_bad(r, grp, smem + C::OFF_BAD + it % C::NBAD * 256, f, backwards);
                const float by = r < rows ? sw.c_inter * w[backwards ? rows - 1 - r : r + 1] : 0.f;
                const float2 by2 = make_float2(by, by);
                const uint32_t at = tmem + lane_off + 32 * grp;
                __nv_bfloat16 *row = rows_out + (long long)t * sw.rows.sn;
#pragma unroll 1
                for (int c = 0; c < 32; c += 16) {
                    uint32_t az[16], xs[16], o[8];
                    tmem_ld16(at + C::COL_AZ + c, az);
                    tmem_ld16(at + C::COL_XS + c, xs);
                    tmem_wait_ld();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float2 v = fma_pair(pair_at(az, 2 * i), intra2, mul_pair(pair_at(xs, 2 * i), by2));
                        o[i] = pack_bf16x2(v.x, v.y);
                    }
                    if (__builtin_expect(r >= rows || hit, 0)) {
#pragma unroll
                        for (int i = 0; i < 8; ++i)   // zeros past the length, NaN where a value of z that is not finite is seen
                            o[i] = r >= rows ? 0u
                                             : o[i] | (hit >> (c + 2 * i) & 1u ? 0x7fffu : 0u) |
                                                   (hit >> (c + 2 * i + 1) & 1u ? 0x7fff0000u : 0u);
                    }
                    if (t < args.N)
                        store16(row + c, make_uint4(o[0], o[1], o[2], o[3]), make_uint4(o[4], o[5], o[6], o[7]), cols - c);
                }
            }
            tc_fence_before();
            arrive_warp(&o_free[pb]);
        };
        if (out) {
            for (int it = 0; it <= n; ++it) {
                if (it < n) scores(it);
                if (it > 0) output(it - 1);
            }
            // the chunks past the length: zeros
            const uint4 zeros = make_uint4(0u, 0u, 0u, 0u);
            for (int t = first + n * kC + r; t < min(first + args.seg_tokens, args.N); t += kC)
                for (int c = 0; c < 32; c += 16) store16(rows_out + (long long)t * sw.rows.sn + c, zeros, zeros, cols - c);
        }
    } else {
        // ------------------------------------------------------ weighted z, state
        // The state lies in registers: DP = 64: thread (grp, q4, lane) keeps columns
        // 32 (q4 / 2) + 16 grp on of row 32 (q4 & 1) + lane; DP = 128: columns 32 grp on
        // of row 32 q4 + lane
        constexpr int NC = DP == 64 ? 16 : 32;
        const int q4 = warp & 3, r = 32 * q4 + lane, grp = warp >= 16;
        const uint32_t lane_off = (uint32_t)(32 * q4) << 16;
        const int d = DP == 64 ? 32 * (q4 & 1) + lane : r, cb = DP == 64 ? 32 * (q4 >> 1) + 16 * grp : 32 * grp;
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
            // the snapshot that this one replaces has been read by its chunk's x S
            const int old = it - C::NSNAP;
            if (old >= 0) wait_warp(&xs_full[old & 1], (old >> 1) & 1, abort);
#pragma unroll
            for (int j = 0; j < NC; j += 8) {
                uint4 v;
                v.x = pack_bf16x2(sv[j], sv[j + 1]);
                v.y = pack_bf16x2(sv[j + 2], sv[j + 3]);
                v.z = pack_bf16x2(sv[j + 4], sv[j + 5]);
                v.w = pack_bf16x2(sv[j + 6], sv[j + 7]);
                *reinterpret_cast<uint4 *>(snap(it) + sw128_offset(d, cb + j)) = v;
            }
            fence_proxy_async();
            arrive_warp(&snap_ready[it & 1]);
        };
        // z of chunk it: the half of its rows from 64 on or before, by four pieces of 16
        // columns a row (the parts go where the MMAs have read the last chunk's)
        const int zr = (tid - 384) & 63, zc = 16 * ((tid - 384) >> 6);
        auto weigh = [&](int it, int half, bool ok) {
            const int rows = rows_of(it), row = 64 * half + zr;
            uint8_t *zt = ztile(it);
            if (ok) {
                const float wr = row < rows ? w[backwards ? row + 1 : rows - 1 - row] : 0.f;
                const float2 wr2 = make_float2(wr, wr), minus = make_float2(-1.f, -1.f);
                float2 check = make_float2(0.f, 0.f);   // NaN where a value is not finite
#pragma unroll
                for (int c = zc; c < zc + 16; c += 8) {
                    const uint32_t off = sw128_offset(row, c);
                    const uint4 v = *reinterpret_cast<const uint4 *>(zt + off);
                    const uint32_t in[4] = {v.x, v.y, v.z, v.w};
                    uint32_t hi[4], mid[4];
                    float2 rest[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        // the leading 8 bits of each value, cut off, three times: 24 bits, all there are
                        float2 f = mul_pair(get_pair(in[j]), wr2);
                        hi[j] = top_pair(f);
                        f = fma_pair(get_pair(hi[j]), minus, f);
                        check = add_pair(check, f);
                        mid[j] = top_pair(f);
                        rest[j] = f;
                    }
                    *reinterpret_cast<uint4 *>(zw + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4 *>(zw + kTile + off) = make_uint4(mid[0], mid[1], mid[2], mid[3]);
                    if (parts == 3) {
                        uint32_t lo[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) lo[j] = top_pair(fma_pair(get_pair(mid[j]), minus, rest[j]));
                        *reinterpret_cast<uint4 *>(zw + 2 * kTile + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    }
                }
                const int slot = it % C::NBAD * 16 + 8 * half + (warp - 12);
                const float all = check.x + check.y;
                const bool any = __any_sync(0xffffffffu, !(fabsf(all) < __int_as_float(0x7f800000)));
                if (__builtin_expect(any, 0)) take_out(zt, row, zc, smem + C::OFF_BAD + slot * 16, backwards);
                if (lane == 0) flag[slot] = any;
            }
            fence_proxy_async();
            arrive_warp(half ? &zw_ready[it & 3] : half_ready);
        };
        // a sequence's last chunk: rows past the end are nothing, whatever they hold
        auto end_rows = [&](int it) {
            const int rows = rows_of(it);
            const bool ok = wait_warp(&y_full[it % C::NS], (it / C::NS) & 1, abort);
            if (ok && r >= rows) {
                uint8_t *zt = ztile(it), *yt = ytile(it) + (DP == 64 ? 0 : grp * kTile);
                for (int c = 0; c < 32; c += 8)
                    *reinterpret_cast<uint4 *>(zt + sw128_offset(r, 32 * grp + c)) = make_uint4(0u, 0u, 0u, 0u);
                for (int c = 0; c < DP / 2; c += 8)
                    *reinterpret_cast<uint4 *>(yt + sw128_offset(r, (DP == 64 ? 32 * grp : 0) + c)) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async();
            arrive_warp(tail_ready);
            asm volatile("bar.sync 1, 256;" ::: "memory");   // other warps read these rows
            return ok;
        };
        if (out) put_snap(0);
        const float2 kept_whole = kept(g, kC), kept_tail = kept(g, tail), c2 = make_float2(sw.c_state, sw.c_state);
        for (int it = 0; it <= n; ++it) {
            bool ok = true;
            if (it < n) {
                ok = wait_warp(&z_full[it % C::NS], (it / C::NS) & 1, abort);
                if (rows_of(it) < kC) ok = end_rows(it) && ok;
                if (it > 0) ok = wait_warp(half_free, (it - 1) & 1, abort) && ok;
                weigh(it, 0, ok);
            }
            if (it > 0) {   // the increment of the chunk before
                ok = wait_warp(&ds_full[(it - 1) & 1], ((it - 1) >> 1) & 1, abort) && ok;
                if (ok) {
                    tc_fence_after();
                    const float2 a = rows_of(it - 1) == kC ? kept_whole : kept_tail;
                    const uint32_t tds = tmem + lane_off + C::COL_DS + kMB * ((it - 1) & 1) + cb;
#pragma unroll
                    for (int j = 0; j < NC; j += 16) {
                        uint32_t v[16];
                        tmem_ld16(tds + j, v);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; i += 2) {
                            const float2 e = pair_at(v, i);
                            float2 s2 = make_float2(sv[j + i], sv[j + i + 1]);
                            s2 = fma_pair(make_float2(a.y, a.y), s2, mul_pair(make_float2(a.x, a.x), s2));
                            s2 = fma_pair(c2, e, s2);
                            sv[j + i] = s2.x, sv[j + i + 1] = s2.y;
                        }
                    }
                }
                tc_fence_before();
                arrive_warp(&ds_free[(it - 1) & 1]);
            }
            if (it == n) break;
            // z before the snapshot: its increment is what the next round waits for
            weigh(it, 1, ok);
            if (it > 0 && out) put_snap(it);
        }
        // the state leaves where the sequence's last segment (backwards: its first) ends
        if (sw.end && !*abort && (args.sums || seg == (backwards ? 0 : last_segment(len, args.seg_tokens)))) {
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

// 16-byte rows: base and strides; dimensions of one do not move, and heads and
// sequences may be one and the same (stride 0).
bool mappable(const la_view &v, int B, int H, int N) {
    auto ok = [](long long stride, int n) { return n <= 1 || (stride % 8 == 0 && stride > 0 && stride < (1LL << 38)); };
    return v.data == nullptr || ((reinterpret_cast<uintptr_t>(v.data) & 15) == 0 && (v.sb == 0 || ok(v.sb, B)) &&
                                 (v.sh == 0 || ok(v.sh, H)) && ok(v.sn, N));
}
int shared_by(const la_view &v) { return (v.sh == 0 ? 1 : 0) | (v.sb == 0 ? 2 : 0); }

// Tensor map of [B][H][N][cols] with the view's strides, boxes of 64 columns x
// 128 rows.  Columns and rows past the tensor read as zeros and are not written.
bool map_of(CUtensorMap *m, const la_view &v, int cols, const DecayLaunch &l) {
    auto fn = encode_fn();
    if (!fn) return false;
    const int H = v.sh == 0 ? 1 : l.H, B = v.sb == 0 ? 1 : l.B;
    auto bytes = [](long long stride, int n) { return (cuuint64_t)(n > 1 ? stride * 2 : 16); };
    cuuint64_t dims[4] = {(cuuint64_t)cols, (cuuint64_t)l.N, (cuuint64_t)H, (cuuint64_t)B};
    cuuint64_t strides[3] = {bytes(v.sn, l.N), bytes(v.sh, H), bytes(v.sb, B)};
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
        for (const la_view *v : {&s.x, &s.y, &s.z})
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
        if (s.out.data && !map_of(&t.x, s.x, s.D, l)) return cudaErrorInvalidValue;
        t.rows = s.out, t.start = s.start, t.end = s.end, t.D = s.D, t.M = s.M, t.blocks = (s.M + kMB - 1) / kMB;
        t.transposed = s.transposed, t.backwards = s.backwards, t.has_out = s.out.data != nullptr;
        t.shared = shared_by(s.x) | shared_by(s.y) << 2 | shared_by(s.z) << 4;
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
