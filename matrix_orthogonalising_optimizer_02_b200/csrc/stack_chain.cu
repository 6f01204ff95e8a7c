// Grouped, persistent, warp-specialised fp16 GEMM on the 5th-generation tensor cores (tcgen05 +
// TMEM + TMA) for the products of Newton-Schulz orthogonalisation of stacks of blocks and of its
// reverse pass:
//   A = X X^T,  B = bA + cA^2,  X' = aX + BX;   S = sym(D X^T),  P = bS + c(SA + AS),
//   D' = aD + BD + 2PX   (for tall blocks with the factors exchanged).
//
// Why fp16 and not bf16: the iterates are bounded (singular values below the schedule's bound, 1.2
// for the usual ones), so with power-of-two scales that the host derives from the schedule every
// operand sits inside fp16's range and carries 11 bits instead of 8 at the same tensor rate.  And
// the term a * X, which alone carries the small singular directions, takes X as a sum of two fp16
// planes: the second is never multiplied, only added in the epilogue.  On a gradient-like 768 x 768
// block five iterations are then 1e-3 off 64 bits (bf16 operands: 1.5e-2), on a rank-32 gradient
// with 1% noise 5e-4 (1.6e-1).  Every product and every combination is held in fp32; a plane is
// rounded once, when it is stored.
//
// One launch for the whole chain.  Pairs of CTAs stay and draw tiles from a counter in the order of the
// operations; a tile waits until its block's earlier operations are done (a counter per block that every
// finished epilogue warp raises).  A tile depends on tiles drawn earlier alone, and whoever has drawn one
// is running, so the chain ends whatever else holds SMs.  Against a launch per operation this saves the
// launch and its prologue (about 8 of the 12 us of a small product) and, with several blocks, the last
// wave of every operation: 24 blocks of 509 x 1021 are 72 + 72 + 192 tiles an iteration on 74 pairs, 1 + 1 + 3
// waves with gaps between them before, 4.5 without now.
//
// Two CTAs of a cluster compute one tile of 256 x 256 (128 or 64 columns where that many tiles would leave
// pairs idle) with tcgen05.mma.cta_group::2 (K = 16 a step):
// each stages its 128 rows of A and half the columns of B, so an SM reads half the B bytes that a
// one-SM tile would.  Roles per CTA (384 threads): warp 0 lane 0 TMA producer, warp 1 lane 0 of the
// leader MMA issuer, warp 2 TMEM, warp 3 lane 0 of the leader draws tiles (one ahead), warps 4..11
// epilogue (TMEM double buffered, so the epilogue of one tile overlaps the products of the next).
// Global accesses of the epilogue are turned through shared memory into 8 rows x 64 bytes per
// instruction, E arrives there a chunk ahead.  Every wait is bounded (ptx_sm100.cuh); no load uses
// cluster multicast.
//
// Bound: power and the tensor pipe for large blocks (16 of 2048 x 1408, five iterations: 1.28 ms at 1.57 GHz with
// the tensor pipe 61% busy when run alone, 1.6 ms at what the 1 kW cap leaves under load); below about 1024 x 1024
// the latency of one operation after the other (one block of 1000 x 1000: 31 us an iteration, three operations).
// Fetching E two chunks ahead, or releasing finished tiles from a warp of its own (it adds 1 us to every
// operation), gained nothing.
#include <atomic>

#include "ptx_stacks.cuh"
#include "stacks.cuh"

namespace muon {
namespace {

constexpr int BM = 256, BN = 256, BK = 64, STAGES = 5;
constexpr int HM = BM / 2, HN = BN / 2;   // per CTA: rows of A, columns of B of the widest tile
constexpr int A_BYTES = HM * BK * 2, B_BYTES = HN * BK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int BOX_BYTES = 64 * BK * 2;    // 64 x 64 fp16, whichever way it lies
constexpr int TMEM_COLS = 512, ACC_COLS = 256;
constexpr int BAR_BYTES = 256;
constexpr int THREADS = 384, EPI_THREADS = 256;
// Per epilogue warp four 32 x 32 fp16 chunks (64-byte rows): the two planes of the output (or the output and
// its transposed mirror) and the two of E, which is fetched again as soon as it is in registers.
constexpr int STG_BYTES = 32 * 64;
constexpr int STG_WARP_BYTES = 4 * STG_BYTES;
constexpr int SMEM_TOTAL = STAGES * STAGE_BYTES + BAR_BYTES + (EPI_THREADS / 32) * STG_WARP_BYTES + 1024;
static_assert(SMEM_TOTAL <= 232448, "dynamic shared memory above the 227 KB per-CTA limit");

template <int NC, int NO>
struct ChainParams {
    ChainClass cls[NC];
    ChainOp op[NO];
    int n, tiles;
    int* ticket;
    unsigned* status;
};

// A drawn tile, as the drawer hands it to the readers.
struct alignas(16) Draw {
    int op;                // operation, | kUnready; negative: no more tiles
    int b, m0, n0;         // block and place
};
constexpr int kUnready = 1 << 20;   // the block's earlier operations were not done when the tile was drawn

struct Shape {
    int M, N, K, w;        // of the operation; w: columns of a tile
    // Columns of the tile at column n0: the last ones of a row take as many 64s as are left.
    __device__ __forceinline__ int width(int n0) const { return min(w, (N - n0 + 63) & ~63); }
};
__device__ __forceinline__ Shape shape_of(const ChainClass& c, const ChainOp& o) {
    return {o.kind < 2 ? c.r8 : c.rp, o.kind < 2 ? c.r8 : c.cp, o.kind == 0 ? max(c.rp, c.cp) : c.r8, 64 * o.bn};
}
// Moves `op` on to the operation of tile t (tiles come in rising order) and gives the tile's place
// (symmetric operations list the tiles with mb <= nb, column by column).
template <class P>
__device__ __forceinline__ Draw draw_of(const P& g, int t, int& op) {
    while (op + 1 < g.n && g.op[op + 1].tile0 <= t) ++op;
    const ChainOp& o = g.op[op];
    const ChainClass& c = g.cls[o.cls];
    const Shape z = shape_of(c, o);
    const int mbs = (z.M + BM - 1) / BM, nbs = (z.N + z.w - 1) / z.w;
    const int per = chain_tiles(c, o), i = t - o.tile0;
    Draw d;
    d.op = op;
    d.b = i / per;
    int l = i - d.b * per, mb, nb;
    if (o.flags & kStackSym) {
        // column groups of 256: group g has 4 / bn columns of g + 1 tiles
        const int cols = 4 / o.bn, u = l / cols;
        int gcol = static_cast<int>((sqrtf(8.f * u + 1.f) - 1.f) * 0.5f);
        while (cols * (gcol * (gcol + 1) / 2) > l) --gcol;
        while (cols * ((gcol + 1) * (gcol + 2) / 2) <= l) ++gcol;
        l -= cols * (gcol * (gcol + 1) / 2);
        const int k = l / (gcol + 1);
        mb = l - k * (gcol + 1);
        nb = gcol * cols + k;
    } else if (o.flags & kStackRowMajor) {
        mb = l / nbs;
        nb = l - mb * nbs;
    } else {
        nb = l / mbs;
        mb = l - nb * mbs;
    }
    d.m0 = mb * BM;
    d.n0 = nb * z.w;
    return d;
}

__device__ __forceinline__ int load_done(const int* p) {
    int v;
    asm volatile("ld.acquire.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// Bounded wait until *p >= need; what the counted warps wrote is visible afterwards.
__device__ __forceinline__ bool wait_done(const int* p, int need, volatile int* abort, unsigned* status) {
    const unsigned long long t0 = global_ns();
    while (true) {
        if (load_done(p) >= need) return true;
        if (*abort) return false;
        if (global_ns() - t0 > kWaitLimitNs) {
            *abort = 1;
            atomicOr(status, kDevErrTimeout);
            return false;
        }
        __nanosleep(64);
    }
}
__device__ __forceinline__ void add_done(int* p) {
    asm volatile("red.release.gpu.global.add.s32 [%0], 1;" ::"l"(p) : "memory");
}
// Global data written by ordinary stores and read by TMA (on either side of a signal).
__device__ __forceinline__ void fence_proxy_global() { asm volatile("fence.proxy.async.global;" ::: "memory"); }

// Tiles from the leader's drawer to both CTAs: a ring of two slots.  A tile that was not ready when it was drawn
// is waited for by the CTA's producer alone (many more pollers would hold up the counter that they watch: 2048^2
// took 25% longer), which tells the epilogue through a barrier of the slot.
struct Draws {
    const Draw* slot;      // this CTA's two slots
    uint64_t* full;        // this CTA's: a tile is there
    uint64_t* ready;       // this CTA's: and its producer has seen it ready
    uint32_t empty_leader; // the leader's: all readers of both CTAs have taken it
    int i = 0;
    uint32_t waited = 0;   // phases of `ready`, as bits

    // The next tile; a negative op at the end.  By one thread per reader, which calls taken() when the slot may be
    // filled again.
    __device__ __forceinline__ Draw next(volatile int* abort, unsigned* status) {
        const int k = i & 1;
        Draw d;
        d.op = -1;
        if (!mbar_wait_cluster(&full[k], (i >> 1) & 1, abort, status)) return d;
        asm volatile("ld.shared.v4.s32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(d.op), "=r"(d.b), "=r"(d.m0), "=r"(d.n0)
                     : "r"(smem_u32(&slot[k]))
                     : "memory");
        return d;
    }
    __device__ __forceinline__ void taken() {
        mbar_arrive_cluster(empty_leader + 8u * (i & 1));
        ++i;
    }
    // For the epilogue, before taken(): the producer's word that an unready tile is ready.
    __device__ __forceinline__ bool wait_ready(volatile int* abort, unsigned* status) {
        const int k = i & 1;
        const bool ok = mbar_wait(&ready[k], (waited >> k) & 1u, abort, status);
        waited ^= 1u << k;
        return ok;
    }
    __device__ __forceinline__ void tell_ready() const { mbar_arrive(&ready[i & 1]); }
};
__device__ __forceinline__ void put_draw(uint32_t cluster_addr, const Draw& d) {
    asm volatile("st.shared::cluster.v4.s32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_addr), "r"(d.op), "r"(d.b), "r"(d.m0), "r"(d.n0)
                 : "memory");
}
constexpr int kReaders = 1 + 1 + 8 + 1 + 8;   // producer, issuer, epilogue warps; producer, epilogue warps

__device__ __forceinline__ int stg_off64(int row, int seg) { return row * 64 + 16 * (seg ^ ((row >> 1) & 3)); }

__device__ __forceinline__ void cp_async16_zfill(void* smem_dst, const void* gmem_src, int src_bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(smem_dst)), "l"(gmem_src),
                 "r"(src_bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait_group() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Transposes a 32 x 32 chunk of 16-bit elements in staging layout into `dst` (same layout).
__device__ __forceinline__ void stg_transpose32(const uint8_t* src, uint8_t* dst, int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t r0, r1, r2, r3;
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                     : "r"(smem_u32(src + stg_off64(lane, j)))
                     : "memory");
        asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};"
                     ::"r"(smem_u32(dst + stg_off64(8 * j + (lane & 7), lane >> 3))), "r"(r0), "r"(r1), "r"(r2), "r"(r3)
                     : "memory");
    }
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack_half2(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// RESCALE: operations with kStackRescale are among the launch's (the reverse pass); the others' tiles took 0.1 us longer
// with the code for them.
template <int NC, int NO, bool RESCALE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
stack_chain_kernel(const __grid_constant__ ChainParams<NC, NO> g) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
    uint64_t* full_bar = bars;                      // leader: TMA bytes of both CTAs landed
    uint64_t* empty_bar = bars + STAGES;            // both: MMAs reading the stage are done
    uint64_t* tfull_bar = bars + 2 * STAGES;        // both: accumulator ready
    uint64_t* tempty_bar = bars + 2 * STAGES + 2;   // leader: both epilogues drained it
    uint64_t* dfull_bar = bars + 2 * STAGES + 4;    // both: a tile has been drawn
    uint64_t* dempty_bar = bars + 2 * STAGES + 6;   // leader: every reader has it
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 8);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    uint64_t* ready_bar = bars + 2 * STAGES + 10;   // both: the producer has seen a tile ready
    Draw* draw_slot = reinterpret_cast<Draw*>(bars + 2 * STAGES + 12);      // 16-byte aligned
    static_assert((2 * STAGES + 12) * 8 % 16 == 0 && (2 * STAGES + 12) * 8 + 2 * sizeof(Draw) <= BAR_BYTES, "draws' slots");
    unsigned* dev_status = g.status;

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull_bar[a], 1);
            mbar_init(&tempty_bar[a], 2 * EPI_THREADS);
            mbar_init(&dfull_bar[a], 1);
            mbar_init(&dempty_bar[a], kReaders);
            mbar_init(&ready_bar[a], 1);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 2) {
        tmem_alloc_pair(tmem_slot, TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t full_leader = mapa_shared(smem_u32(full_bar), 0);
    const uint32_t tempty_leader = mapa_shared(smem_u32(tempty_bar), 0);
    Draws draws = {draw_slot, dfull_bar, ready_bar, mapa_shared(smem_u32(dempty_bar), 0)};

    if (warp == 3 && lane == 0 && rank == 0) {
        // ------------------------------------------------------------ draws tiles
        uint32_t slot_at[2], full_at[2];
        for (uint32_t r = 0; r < 2; ++r) {
            slot_at[r] = mapa_shared(smem_u32(draw_slot), r);
            full_at[r] = mapa_shared(smem_u32(dfull_bar), r);
        }
        int op = 0;
        for (int i = 0;; ++i) {
            const int k = i & 1;
            const int t = atomicAdd(g.ticket, 1);
            Draw d;
            d.op = -1;
            if (t < g.tiles) d = draw_of(g, t, op);
            if (!mbar_wait_cluster(&dempty_bar[k], ((i >> 1) & 1) ^ 1u, abort_flag, dev_status)) break;
            if (d.op >= 0) {
                // What the earlier operations wrote becomes visible to the readers with the tile.  They wait
                // themselves only where it is not ready now: a tile ahead, it mostly is.
                if (load_done(g.cls[g.op[op].cls].done + d.b) < g.op[op].need) d.op |= kUnready;
                else fence_proxy_global();
            }
            for (int r = 0; r < 2; ++r) {
                put_draw(slot_at[r] + k * static_cast<uint32_t>(sizeof(Draw)), d);
                mbar_arrive_cluster(full_at[r] + 8u * k);
            }
            if (d.op < 0) break;
            // A pair that waits draws no further tiles: they would be others' to start when they all are ready.
            if ((d.op & kUnready) && !mbar_wait_cluster(&dempty_bar[k], (i >> 1) & 1, abort_flag, dev_status)) break;
        }
    } else if (warp == 0 && lane == 0) {
        // ------------------------------------------------------------ TMA producer
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        int issued_parity[STAGES];
#pragma unroll
        for (int s = 0; s < STAGES; ++s) issued_parity[s] = -1;
        for (Draw ti; ok && (ti = draws.next(abort_flag, dev_status)).op >= 0;) {
            const ChainOp& P = g.op[ti.op & (kUnready - 1)];
            const ChainClass& c = g.cls[P.cls];
            if (ti.op & kUnready) {
                if (!wait_done(c.done + ti.b, P.need, abort_flag, dev_status)) { ok = false; break; }
                draws.tell_ready();
                fence_proxy_global();
            }
            draws.taken();
            const Shape z = shape_of(c, P);
            const bool a_mn = (P.flags & kStackAMn) != 0;
            const bool b_mn = (P.flags & kStackBMn) != 0;
            const int am0 = ti.m0 + HM * static_cast<int>(rank);
            const int hn = z.width(ti.n0) / 2;           // columns of B that this CTA uses: 128, 96, 64 or 32
            const int bn0 = ti.n0 + hn * static_cast<int>(rank);
            const int b_chunks = (hn + 63) / 64;          // boxes of 64 (rows or columns) x 64
            const int kblocks = (z.K + BK - 1) / BK;
            for (int seg = 0; seg < P.nseg && ok; ++seg) {
                const CUtensorMap* ta = &c.map[P.ma[seg]];
                const CUtensorMap* tb = &c.map[P.mb[seg]];
                const int za = P.sa[seg] * c.count + ti.b, zb = P.sb[seg] * c.count + ti.b;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, dev_status)) { ok = false; break; }
                    uint8_t* sa = smem + stage * STAGE_BYTES;
                    uint8_t* sb = sa + A_BYTES;
                    const int k0 = kb * BK;
                    const uint32_t fb = full_leader + stage * 8u;
                    if (rank == 0) {
                        mbar_arrive_expect_tx(&full_bar[stage], 2u * static_cast<uint32_t>(A_BYTES + b_chunks * BOX_BYTES));
                        issued_parity[stage] = static_cast<int>(phase);
                    }
#pragma unroll
                    for (int h = 0; h < HM / 64; ++h)
                        tma_load_3d_pair(sa + h * BOX_BYTES, ta, fb, a_mn ? am0 + 64 * h : k0, a_mn ? k0 : am0 + 64 * h, za);
                    for (int h = 0; h < b_chunks; ++h)
                        tma_load_3d_pair(sb + h * BOX_BYTES, tb, fb, b_mn ? bn0 + 64 * h : k0, b_mn ? k0 : bn0 + 64 * h, zb);
                    if (++stage == STAGES) { stage = 0; phase ^= 1u; }
                }
            }
        }
        if (!ok && rank == 0) {
            // Let copies already issued land before the pair exits (bounded).
            for (int s = 0; s < STAGES; ++s) {
                if (issued_parity[s] < 0) continue;
                const unsigned long long t0 = global_ns();
                bool landed = false;
                while (!(landed = mbar_try_wait(&full_bar[s], static_cast<uint32_t>(issued_parity[s]))) &&
                       global_ns() - t0 < 100000000ull) {
                }
                if (!landed) atomicOr(dev_status, kDevErrUndrained);
            }
        }
    } else if (warp == 1 && lane == 0 && rank == 0) {
        // ------------------------------------------------------------ MMA issuer (leader)
        uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
        bool ok = true;
        for (Draw ti; ok && (ti = draws.next(abort_flag, dev_status)).op >= 0;) {
            draws.taken();
            const ChainOp& P = g.op[ti.op & (kUnready - 1)];
            const Shape z = shape_of(g.cls[P.cls], P);
            const bool a_mn = (P.flags & kStackAMn) != 0;
            const bool b_mn = (P.flags & kStackBMn) != 0;
            const uint32_t idesc = idesc_f16_f32(BM, z.width(ti.n0), a_mn, b_mn);
            const int kblocks = (z.K + BK - 1) / BK * P.nseg;
            if (!mbar_wait(&tempty_bar[acc], acc_phase ^ 1u, abort_flag, dev_status)) { ok = false; break; }
            tc_fence_after();
            const uint32_t d_tmem = tmem_base + acc * ACC_COLS;
            uint32_t accumulate = 0;
            for (int kb = 0; kb < kblocks; ++kb) {
                if (!mbar_wait(&full_bar[stage], phase, abort_flag, dev_status)) { ok = false; break; }
                tc_fence_after();
                const uint32_t base_a = smem_u32(smem + stage * STAGE_BYTES);
                const uint32_t base_b = base_a + A_BYTES;
#pragma unroll
                for (int k = 0; k < BK / 16; ++k) {
                    const uint64_t ad = a_mn ? smem_desc_sw128(base_a + k * 2048, BOX_BYTES, 1024)
                                             : smem_desc_sw128(base_a + k * 32, 16, 1024);
                    const uint64_t bd = b_mn ? smem_desc_sw128(base_b + k * 2048, BOX_BYTES, 1024)
                                             : smem_desc_sw128(base_b + k * 32, 16, 1024);
                    tc_mma_bf16_pair(d_tmem, ad, bd, idesc, accumulate);   // kind::f16, types from idesc
                    accumulate = 1;
                }
                tc_commit_pair(&empty_bar[stage], 0x3);
                if (++stage == STAGES) { stage = 0; phase ^= 1u; }
            }
            if (!ok) break;
            tc_commit_pair(&tfull_bar[acc], 0x3);
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
        if (!ok) {
            // Drain: wait (bounded) until every MMA issued so far has finished.
            tc_commit_pair(&tfull_bar[acc], 0x3);
            const unsigned long long t0 = global_ns();
            bool done = false;
            while (!(done = mbar_try_wait(&tfull_bar[acc], acc_phase)) && global_ns() - t0 < 100000000ull) {
            }
            if (!done) atomicOr(dev_status, kDevErrUndrained);
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ epilogue
        // warp & 3 selects the TMEM lane quarter (rows), (warp - 4) >> 2 the half of the columns.
        const int q = warp & 3;
        uint8_t* stg = smem + STAGES * STAGE_BYTES + BAR_BYTES + (warp - 4) * STG_WARP_BYTES;
        uint8_t* stg_t = stg + STG_BYTES;
        uint8_t* stg_e = stg + 2 * STG_BYTES;          // the planes of E
        const int crow = lane >> 2, cseg = lane & 3;   // coalesced layout: rows crow + 8i, segment cseg
        uint32_t acc = 0, acc_phase = 0;
        while (true) {
            Draw ti;
            ti.op = -1;
            if (lane == 0) {
                ti = draws.next(abort_flag, dev_status);
                if (ti.op >= 0) {
                    if (ti.op & kUnready) ti.op = draws.wait_ready(abort_flag, dev_status) ? ti.op & (kUnready - 1) : -1;
                    draws.taken();
                }
            }
            ti.op = __shfl_sync(0xffffffffu, ti.op, 0);
            if (ti.op < 0) break;
            ti.b = __shfl_sync(0xffffffffu, ti.b, 0);
            ti.m0 = __shfl_sync(0xffffffffu, ti.m0, 0);
            ti.n0 = __shfl_sync(0xffffffffu, ti.n0, 0);
            __syncwarp();     // what lane 0 has acquired with the tile (E, the block's info) is every lane's: a shuffle orders nothing
            const ChainOp& P = g.op[ti.op];
            const ChainClass& cl = g.cls[P.cls];
            const Shape z = shape_of(cl, P);
            float f = 1.0f;
            if (P.pow != 0) {
                const float x = cl.info[static_cast<size_t>(ti.b) * kStackInfo];
                f = P.pow == 1 ? x : x * x;
            }
            const bool rescale = RESCALE && (P.flags & kStackRescale) != 0;
            GradScale* scale = rescale ? cl.scale + static_cast<size_t>(ti.b) * cl.scales + P.t : nullptr;
            unsigned long long read_sum = 0;     // of the planes that are read: on its way while the products run
            int read_e = 0;
            if (rescale) {
                read_sum = __ldcg(&scale[1].sum);
                read_e = __ldcg(&scale[1].e);
            }
            float alpha = P.alpha * f, beta = P.beta * f, squares = 0.f;
            const int chunks = z.width(ti.n0) / 64;
            const int c_beg = ((warp - 4) >> 2) * chunks, c_end = c_beg + chunks;   // this warp's chunks of 32 columns
            const bool sym = (P.flags & kStackSym) != 0;
            const bool bf = (P.flags & kStackOutBf16) != 0;
            const int row0 = ti.m0 + HM * static_cast<int>(rank) + q * 32;
            auto plane_of = [&](int pl, int slot) {
                return pl == kPlaneNone ? nullptr
                                        : cl.plane[pl].p + (static_cast<size_t>(slot) * cl.count + ti.b) * cl.plane[pl].block;
            };
            const __half* e0 = plane_of(P.e[0], P.es[0]);
            const __half* e1 = plane_of(P.e[1], P.es[1]);
            __half* o_plane[2] = {plane_of(P.o[0], P.os[0]), plane_of(P.o[1], P.os[1])};
            const int planes = o_plane[1] != nullptr ? 2 : 1;
            const int e_ld = z.N, o_ld = cl.plane[P.o[0]].ld;
            const int m_out = P.o[0] == kPlaneOut ? cl.rows : z.M;
            const uint32_t t_row = tmem_base + acc * ACC_COLS + (static_cast<uint32_t>(q * 32) << 16);

            // E of chunk c goes into staging by cp.async while the chunk before is packed and stored.
            auto prefetch_e = [&](int c) {
                const int col0 = ti.n0 + c * 32;
                if (e0 != nullptr && col0 < z.N && !(sym && col0 + 31 < row0)) {
                    const int cc = col0 + 8 * cseg;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = row0 + crow + 8 * i;
                        const bool in = rr < z.M && cc < z.N;
                        const size_t at = in ? static_cast<size_t>(rr) * e_ld + cc : 0;
                        cp_async16_zfill(stg_e + stg_off64(crow + 8 * i, cseg), e0 + at, in ? 16 : 0);
                        if (e1 != nullptr)
                            cp_async16_zfill(stg_e + STG_BYTES + stg_off64(crow + 8 * i, cseg), e1 + at, in ? 16 : 0);
                    }
                }
                cp_async_commit();
            };
            prefetch_e(c_beg);
            if (rescale) {
                // The scale of the planes that are written, from the norm of those that were read: `room` is that of the
                // planes over the most that the operation can grow them, so nothing leaves fp16's range, and they lie at
                // most one operation's slack below it.
                const float n = sqrtf(__ull2float_rn(read_sum)) * 3.0517578125e-05f;      // 2^-15
                const int e = read_sum != 0 ? max(-60, min(60, ilogbf(P.room / n))) : 0;
                alpha *= __int_as_float((e + 127) << 23);
                beta *= __int_as_float((e + 127) << 23);
                if (ti.m0 + ti.n0 == 0 && rank == 0 && warp == 4 && lane == 0) scale->e = read_e + e;
            }
            if (!__all_sync(0xffffffffu, mbar_wait(&tfull_bar[acc], acc_phase, abort_flag, dev_status))) {
                cp_async_wait_all();
                break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = c_beg; c < c_end; ++c) {
                const int col0 = ti.n0 + c * 32;
                if (col0 >= z.N) break;  // uniform across the warp
                const bool below = sym && col0 < row0;    // its mirror image is stored instead
                const bool mirror = sym && col0 > row0;   // a chunk on the diagonal holds both halves
                uint32_t r[32];
                tmem_ld_32x32b_x32(t_row + c * 32, r);
                cp_async_wait_group<0>();   // this lane's copies of chunk c have landed
                tmem_ld_wait();
                __syncwarp();               // ... and every lane's
                float v[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = alpha * __uint_as_float(r[j]);
                if (col0 == row0 && P.diag != 0.f) {
#pragma unroll
                    for (int j = 0; j < 32; ++j)
                        if (j == lane) v[j] -= P.diag;
                }
                if (e0 != nullptr && !below) {
                    for (int pl = 0; pl < (e1 != nullptr ? 2 : 1); ++pl) {
                        const uint8_t* src = stg_e + pl * STG_BYTES;
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const uint4 w = *reinterpret_cast<const uint4*>(src + stg_off64(lane, s));
                            const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const float2 e = unpack_half2(x[h]);
                                v[8 * s + 2 * h] = fmaf(beta, e.x, v[8 * s + 2 * h]);
                                v[8 * s + 2 * h + 1] = fmaf(beta, e.y, v[8 * s + 2 * h + 1]);
                            }
                        }
                    }
                }
                if (rescale) {
#pragma unroll
                    for (int j = 0; j < 32; ++j) squares = fmaf(v[j], v[j], squares);   // zeros outside the block
                }
                __syncwarp();               // E's staging is free, and the output's of the chunk before
                if (c + 1 < c_end) prefetch_e(c + 1);
                if (!below) {
                    // rows -> staging -> 8 rows x 64 bytes per instruction; plane 1 (what plane 0 has lost) beside it
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        uint32_t w[4], l[4];
#pragma unroll
                        for (int h = 0; h < 4; ++h) {
                            const float x = v[8 * s + 2 * h], y = v[8 * s + 2 * h + 1];
                            w[h] = bf ? pack_bf16x2(x, y) : pack_half2(x, y);
                            const float2 e = unpack_half2(w[h]);
                            l[h] = pack_half2(x - e.x, y - e.y);
                        }
                        *reinterpret_cast<uint4*>(stg + stg_off64(lane, s)) = make_uint4(w[0], w[1], w[2], w[3]);
                        if (planes == 2) *reinterpret_cast<uint4*>(stg_t + stg_off64(lane, s)) = make_uint4(l[0], l[1], l[2], l[3]);
                    }
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = row0 + crow + 8 * i, cc = col0 + 8 * cseg;
                        if (rr < m_out && cc < z.N) {
                            const size_t at = static_cast<size_t>(rr) * o_ld + cc;
                            *reinterpret_cast<uint4*>(o_plane[0] + at) =     // bf16: the same 2 bytes
                                *reinterpret_cast<const uint4*>(stg + stg_off64(crow + 8 * i, cseg));
                            if (planes == 2)
                                *reinterpret_cast<uint4*>(o_plane[1] + at) =
                                    *reinterpret_cast<const uint4*>(stg_t + stg_off64(crow + 8 * i, cseg));
                        }
                    }
                    if (mirror) {      // symmetric outputs have one plane
                        stg_transpose32(stg, stg_t, lane);
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int rr = col0 + crow + 8 * i, cc = row0 + 8 * cseg;
                            if (rr < z.N && cc < z.M)
                                *reinterpret_cast<uint4*>(o_plane[0] + static_cast<size_t>(rr) * o_ld + cc) =
                                    *reinterpret_cast<const uint4*>(stg_t + stg_off64(crow + 8 * i, cseg));
                        }
                    }
                    __syncwarp();
                }
            }
            cp_async_wait_all();
            tc_fence_before();
            mbar_arrive_cluster(tempty_leader + acc * 8u);
            if (rescale) {
                // whole numbers add up to the same sum in any order; rounded up, so that the norm is never too small
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) squares += __shfl_xor_sync(0xffffffffu, squares, o);
                if (lane == 0) atomicAdd(&scale->sum, __float2ull_ru(squares * 1073741824.f));
            }
            // the block's next operation may read what this warp stored, by TMA among other ways
            fence_proxy_global();
            __syncwarp();                       // the release below covers every lane's stores
            if (lane == 0) add_done(cl.done + ti.b);
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
    }
    tc_fence_before();
    cluster_sync();     // no CTA leaves while its pair may still touch its memory
    tc_fence_after();
    if (warp == 2) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// The launch of one instantiation; its attributes and occupancy are looked up once per device.
template <int NC, int NO, bool RESCALE>
cudaError_t launch(const ChainClass* classes, int nc, const ChainOp* ops, int n, int tiles, int* ticket, unsigned* d_status,
                   int num_sms, cudaStream_t stream) {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> max_pairs_of[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(THREADS, 1, 1);
    cfg.dynamicSmemBytes = SMEM_TOTAL;
    int max_pairs = max_pairs_of[dev].load();
    if (max_pairs == 0) {
        e = cudaFuncSetAttribute(stack_chain_kernel<NC, NO, RESCALE>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_TOTAL);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(2 * (num_sms / 2), 1, 1);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&max_pairs, stack_chain_kernel<NC, NO, RESCALE>, &cfg);
        if (e != cudaSuccess || max_pairs <= 0) {
            cudaGetLastError();
            max_pairs = num_sms / 2;
        }
        max_pairs_of[dev].store(max_pairs);
    }
    ChainParams<NC, NO> g;
    for (int i = 0; i < nc; ++i) g.cls[i] = classes[i];
    for (int i = 0; i < n; ++i) g.op[i] = ops[i];
    g.n = n;
    g.tiles = tiles;
    g.ticket = ticket;
    g.status = d_status;
    cfg.gridDim = dim3(2 * static_cast<unsigned>(tiles < max_pairs ? tiles : max_pairs), 1, 1);
    cfg.stream = stream;
    cfg.attrs = nullptr;
    cfg.numAttrs = 0;
    e = cudaLaunchKernelEx(&cfg, stack_chain_kernel<NC, NO, RESCALE>, g);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t stack_chain_launch(const ChainClass* classes, int nc, ChainOp* ops, int n, int* ticket, unsigned* d_status,
                               int num_sms, cudaStream_t stream) {
    long long tiles = 0;
    for (int i = 0; i < n; ++i) {
        ops[i].tile0 = static_cast<int>(tiles);
        const ChainClass& c = classes[ops[i].cls];
        tiles += static_cast<long long>(chain_tiles(c, ops[i])) * c.count;
        if (tiles > INT32_MAX / 2) return cudaErrorInvalidValue;
    }
    if (tiles == 0) return cudaSuccess;
    if (nc > kChainMaxClasses || n > kChainMaxOps) return cudaErrorInvalidValue;
    // Parameters of up to 4 KB launch in 4 us, larger ones in 30 to 40 (10 KB): short chains take the small form.
    static_assert(sizeof(ChainParams<2, 30>) <= 4000, "the small form's parameters stay below 4 KB");
    static_assert(sizeof(ChainParams<kChainMaxClasses, kChainMaxOps>) <= 32700, "the limit of a launch's parameters");
    bool rescale = false;
    for (int i = 0; i < n; ++i) rescale = rescale || (ops[i].flags & kStackRescale) != 0;
    const bool few = nc <= 2 && n <= 30;
    const auto run = few ? (rescale ? launch<2, 30, true> : launch<2, 30, false>)
                         : (rescale ? launch<kChainMaxClasses, kChainMaxOps, true> : launch<kChainMaxClasses, kChainMaxOps, false>);
    return run(classes, nc, ops, n, static_cast<int>(tiles), ticket, d_status, num_sms, stream);
}

}  // namespace muon
