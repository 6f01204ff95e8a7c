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
// Two CTAs of a cluster compute one 256 x 256 tile with tcgen05.mma.cta_group::2 (K = 16 a step):
// each stages its 128 rows of A and 128 columns of B, so an SM reads half the B bytes that a
// one-SM tile would.  Roles per CTA (384 threads): warp 0 lane 0 TMA producer, warp 1 lane 0 of the
// leader MMA issuer, warp 2 TMEM, warps 4..11 epilogue (TMEM double buffered, so the epilogue of
// one tile overlaps the products of the next).  Global accesses of the epilogue are turned through
// shared memory into 8 rows x 64 bytes per instruction.  The tiles of all problems form one list,
// computed from the parameters; pair p takes tiles p, p + pairs, ...  Every wait is bounded
// (ptx_sm100.cuh); no load uses cluster multicast.
//
// Bound: the tensor pipe for large blocks; launch and pipeline latency below about 1024 x 1024.
#include <atomic>

#include "ptx_sm100.cuh"
#include "stacks.cuh"

namespace muon {
namespace {

constexpr int BM = 256, BN = 256, BK = 64, STAGES = 4;
constexpr int HM = BM / 2, HN = BN / 2;
constexpr int A_BYTES = HM * BK * 2, B_BYTES = HN * BK * 2;
constexpr int STAGE_BYTES = A_BYTES + B_BYTES;
constexpr int PAIR_STAGE_BYTES = 2 * STAGE_BYTES;
constexpr int MN_CHUNK_BYTES = 64 * BK * 2;
constexpr int TMEM_COLS = 512, ACC_COLS = 256;
constexpr int BAR_BYTES = 256;
constexpr int THREADS = 384, EPI_THREADS = 256;
// Per epilogue warp four 32 x 32 fp16 chunks (64-byte rows): direct store, transposed mirror, and
// two of E (the one in use and the one being fetched).
constexpr int STG_BYTES = 32 * 64;
constexpr int STG_WARP_BYTES = 4 * STG_BYTES;
constexpr int SMEM_TOTAL = STAGES * STAGE_BYTES + BAR_BYTES + (EPI_THREADS / 32) * STG_WARP_BYTES + 1024;
static_assert(SMEM_TOTAL <= 232448, "dynamic shared memory above the 227 KB per-CTA limit");

template <int N>
struct alignas(64) GemmParams {
    StackProb p[N];
    int n, tiles;
};

constexpr int kFewProbs = 5;

struct Tile {
    int p, b, m0, n0;
};
// Tile t of the launch: problem, block, and position (symmetric problems list the tiles with
// mb <= nb, column by column).
template <int N>
__device__ __forceinline__ Tile tile_at(const GemmParams<N>& g, int t) {
    Tile r;
    r.p = 0;
    if (N > 1) {
        while (r.p + 1 < g.n && g.p[r.p + 1].tile0 <= t) ++r.p;
    }
    const StackProb& P = g.p[r.p];
    const int i = t - P.tile0;
    r.b = i / P.block_tiles;
    const int l = i - r.b * P.block_tiles;
    int mb, nb;
    if (P.flags & kStackSym) {
        nb = static_cast<int>((sqrtf(8.f * l + 1.f) - 1.f) * 0.5f);
        while (nb * (nb + 1) / 2 > l) --nb;
        while ((nb + 1) * (nb + 2) / 2 <= l) ++nb;
        mb = l - nb * (nb + 1) / 2;
    } else if (P.flags & kStackRowMajor) {
        mb = l / P.nbs;
        nb = l - mb * P.nbs;
    } else {
        nb = l / P.mbs;
        mb = l - nb * P.mbs;
    }
    r.m0 = mb * BM;
    r.n0 = nb * BN;
    return r;
}

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

template <int N>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
stack_gemm_kernel(const __grid_constant__ GemmParams<N> g, unsigned* dev_status) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * STAGE_BYTES);
    uint64_t* full_bar = bars;                      // leader: TMA bytes of both CTAs landed
    uint64_t* empty_bar = bars + STAGES;            // both: MMAs reading the stage are done
    uint64_t* tfull_bar = bars + 2 * STAGES;        // both: accumulator ready
    uint64_t* tempty_bar = bars + 2 * STAGES + 2;   // leader: both epilogues drained it
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * STAGES + 4);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    griddep_launch_dependents();   // the next launch waits for this grid before it touches memory
    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full_bar[s], 1);
            mbar_init(&empty_bar[s], 1);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(&tfull_bar[a], 1);
            mbar_init(&tempty_bar[a], 2 * EPI_THREADS);
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

    if (warp == 0 && lane == 0) {
        // ------------------------------------------------------------ TMA producer
        griddep_wait();
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        int issued_parity[STAGES];
#pragma unroll
        for (int s = 0; s < STAGES; ++s) issued_parity[s] = -1;
        for (int t = pair; t < g.tiles && ok; t += npairs) {
            const Tile ti = tile_at(g, t);
            const StackProb& P = g.p[ti.p];
            const bool a_mn = (P.flags & kStackAMn) != 0;
            const bool b_mn = (P.flags & kStackBMn) != 0;
            const int am0 = ti.m0 + HM * static_cast<int>(rank);
            const int bn0 = ti.n0 + HN * static_cast<int>(rank);
            const int kblocks = (P.K + BK - 1) / BK;
            for (int seg = 0; seg < P.nseg && ok; ++seg) {
                const CUtensorMap* ta = &P.tmA[seg];
                const CUtensorMap* tb = &P.tmB[seg];
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait(&empty_bar[stage], phase ^ 1u, abort_flag, dev_status)) { ok = false; break; }
                    uint8_t* sa = smem + stage * STAGE_BYTES;
                    uint8_t* sb = sa + A_BYTES;
                    const int k0 = kb * BK;
                    const uint32_t fb = full_leader + stage * 8u;
                    if (rank == 0) {
                        mbar_arrive_expect_tx(&full_bar[stage], PAIR_STAGE_BYTES);
                        issued_parity[stage] = static_cast<int>(phase);
                    }
                    if (!a_mn) {
                        tma_load_3d_pair(sa, ta, fb, k0, am0, ti.b);
                    } else {
#pragma unroll
                        for (int c = 0; c < HM / 64; ++c)
                            tma_load_3d_pair(sa + c * MN_CHUNK_BYTES, ta, fb, am0 + 64 * c, k0, ti.b);
                    }
                    if (!b_mn) {
                        tma_load_3d_pair(sb, tb, fb, k0, bn0, ti.b);
                    } else {
#pragma unroll
                        for (int c = 0; c < HN / 64; ++c)
                            tma_load_3d_pair(sb + c * MN_CHUNK_BYTES, tb, fb, bn0 + 64 * c, k0, ti.b);
                    }
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
        for (int t = pair; t < g.tiles && ok; t += npairs) {
            const Tile ti = tile_at(g, t);
            const StackProb& P = g.p[ti.p];
            const bool a_mn = (P.flags & kStackAMn) != 0;
            const bool b_mn = (P.flags & kStackBMn) != 0;
            const uint32_t idesc = idesc_f16_f32(BM, BN, a_mn, b_mn);
            const int kblocks = (P.K + BK - 1) / BK * P.nseg;
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
                    const uint64_t ad = a_mn ? smem_desc_sw128(base_a + k * 2048, MN_CHUNK_BYTES, 1024)
                                             : smem_desc_sw128(base_a + k * 32, 16, 1024);
                    const uint64_t bd = b_mn ? smem_desc_sw128(base_b + k * 2048, MN_CHUNK_BYTES, 1024)
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
        const int c_beg = ((warp - 4) >> 2) * (BN / 64);
        const int c_end = c_beg + BN / 64;
        uint8_t* stg = smem + STAGES * STAGE_BYTES + BAR_BYTES + (warp - 4) * STG_WARP_BYTES;
        uint8_t* stg_t = stg + STG_BYTES;
        uint8_t* stg_e = stg + 2 * STG_BYTES;
        const int crow = lane >> 2, cseg = lane & 3;   // coalesced layout: rows crow + 8i, segment cseg
        griddep_wait();
        uint32_t acc = 0, acc_phase = 0;
        for (int t = pair; t < g.tiles; t += npairs) {
            const Tile ti = tile_at(g, t);
            const StackProb& P = g.p[ti.p];
            float f = 1.0f;
            if (P.dscale != nullptr) {
                const float s = __ldg(P.dscale + static_cast<size_t>(ti.b) * kStackInfo);
                f = (P.scale_pow == 1) ? s : s * s;
            }
            const float alpha = P.alpha * f, beta = P.beta * f;
            const bool sym = (P.flags & kStackSym) != 0;
            const bool bf = (P.flags & kStackOutBf16) != 0;
            const int row0 = ti.m0 + HM * static_cast<int>(rank) + q * 32;
            const __half* e0 = P.E[0] != nullptr ? P.E[0] + static_cast<size_t>(ti.b) * P.e_stride : nullptr;
            const __half* e1 = P.E[1] != nullptr ? P.E[1] + static_cast<size_t>(ti.b) * P.e_stride : nullptr;
            const int planes = P.out[1] != nullptr ? 2 : 1;
            const size_t o_base = static_cast<size_t>(ti.b) * P.o_stride;
            const uint32_t t_row = tmem_base + acc * ACC_COLS + (static_cast<uint32_t>(q * 32) << 16);

            // Plane 0 of E for chunk c goes by cp.async into staging slot c & 1, one commit group
            // per chunk, so it is in flight while the previous chunk is processed.
            auto prefetch_e = [&](int c) {
                const int col0 = ti.n0 + c * 32;
                if (e0 != nullptr && col0 < P.N && !(sym && col0 + 31 < row0)) {
                    uint8_t* dst = stg_e + (c & 1) * STG_BYTES;
                    const int cc = col0 + 8 * cseg;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = row0 + crow + 8 * i;
                        const bool in = rr < P.M && cc < P.N;
                        cp_async16_zfill(dst + stg_off64(crow + 8 * i, cseg),
                                         in ? e0 + static_cast<size_t>(rr) * P.e_ld + cc : e0, in ? 16 : 0);
                    }
                }
                cp_async_commit();
            };
            prefetch_e(c_beg);
            if (!__all_sync(0xffffffffu, mbar_wait(&tfull_bar[acc], acc_phase, abort_flag, dev_status))) {
                cp_async_wait_all();
                break;
            }
            tc_fence_after();
#pragma unroll 1
            for (int c = c_beg; c < c_end; ++c) {
                const int col0 = ti.n0 + c * 32;
                if (col0 >= P.N) break;  // uniform across the warp
                const bool below = sym && col0 < row0;    // its mirror image is stored instead
                const bool mirror = sym && col0 > row0;   // a chunk on the diagonal holds both halves
                // plane 1 of E of this chunk: read directly, in the coalesced layout
                uint4 el[4];
                if (e1 != nullptr && !below) {
                    const int cc = col0 + 8 * cseg;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int rr = row0 + crow + 8 * i;
                        el[i] = rr < P.M && cc < P.N
                                    ? *reinterpret_cast<const uint4*>(e1 + static_cast<size_t>(rr) * P.e_ld + cc)
                                    : make_uint4(0, 0, 0, 0);
                    }
                }
                uint32_t r[32];
                tmem_ld_32x32b_x32(t_row + c * 32, r);
                if (c + 1 < c_end) prefetch_e(c + 1);
                else cp_async_commit();
                tmem_ld_wait();
                cp_async_wait_group<1>();   // this lane's copies of chunk c have landed
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
                    const uint8_t* src = stg_e + (c & 1) * STG_BYTES;
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
                    if (e1 != nullptr) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) *reinterpret_cast<uint4*>(stg + stg_off64(crow + 8 * i, cseg)) = el[i];
                        __syncwarp();
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            const uint4 w = *reinterpret_cast<const uint4*>(stg + stg_off64(lane, s));
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
                __syncwarp();               // slot c & 1 is free for chunk c + 2, stg for the store
                if (!below) {
#pragma unroll 1
                    for (int pl = 0; pl < planes; ++pl) {
#pragma unroll
                        for (int s = 0; s < 4; ++s) {
                            uint32_t w[4];
#pragma unroll
                            for (int h = 0; h < 4; ++h) {
                                const float x = v[8 * s + 2 * h], y = v[8 * s + 2 * h + 1];
                                w[h] = bf ? pack_bf16x2(x, y) : pack_half2(x, y);
                                if (planes == 2) {   // what plane 0 has lost, for plane 1
                                    const float2 e = unpack_half2(w[h]);
                                    v[8 * s + 2 * h] = x - e.x;
                                    v[8 * s + 2 * h + 1] = y - e.y;
                                }
                            }
                            *reinterpret_cast<uint4*>(stg + stg_off64(lane, s)) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                        __syncwarp();
                        __half* o = static_cast<__half*>(P.out[pl]) + o_base;   // bf16: the same 2 bytes
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int rr = row0 + crow + 8 * i, cc = col0 + 8 * cseg;
                            const uint4 val = *reinterpret_cast<const uint4*>(stg + stg_off64(crow + 8 * i, cseg));
                            if (rr < P.m_out && cc < P.N)
                                *reinterpret_cast<uint4*>(o + static_cast<size_t>(rr) * P.o_ld + cc) = val;
                        }
                        if (mirror) {
                            stg_transpose32(stg, stg_t, lane);
                            __syncwarp();
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int rr = col0 + crow + 8 * i, cc = row0 + 8 * cseg;
                                const uint4 val = *reinterpret_cast<const uint4*>(stg_t + stg_off64(crow + 8 * i, cseg));
                                if (rr < P.N && cc < P.M)
                                    *reinterpret_cast<uint4*>(o + static_cast<size_t>(rr) * P.o_ld + cc) = val;
                            }
                        }
                        __syncwarp();
                    }
                }
            }
            cp_async_wait_all();
            tc_fence_before();
            mbar_arrive_cluster(tempty_leader + acc * 8u);
            if (++acc == 2) { acc = 0; acc_phase ^= 1u; }
        }
    }
    tc_fence_before();
    cluster_sync();     // no CTA leaves while its pair may still touch its memory
    tc_fence_after();
    if (warp == 2) tmem_dealloc_pair(tmem_base, TMEM_COLS);
}

// The launch of one instantiation; its attributes and occupancy are looked up once per device.
template <int N>
cudaError_t launch(const StackProb* probs, int n, int tiles, unsigned* d_status, int num_sms, cudaStream_t stream) {
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
        e = cudaFuncSetAttribute(stack_gemm_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_TOTAL);
        if (e != cudaSuccess) return e;
        cfg.gridDim = dim3(2 * (num_sms / 2), 1, 1);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&max_pairs, stack_gemm_kernel<N>, &cfg);
        if (e != cudaSuccess || max_pairs <= 0) {
            cudaGetLastError();
            max_pairs = num_sms / 2;
        }
        max_pairs_of[dev].store(max_pairs);
    }
    GemmParams<N> g;
    for (int i = 0; i < n; ++i) g.p[i] = probs[i];
    g.n = n;
    g.tiles = tiles;
    // At most the resident capacity: every CTA runs from the start, so the CTAs of the next launch,
    // which wait for this grid, only take SMs that finished CTAs released.
    cfg.gridDim = dim3(2 * static_cast<unsigned>(tiles < max_pairs ? tiles : max_pairs), 1, 1);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, stack_gemm_kernel<N>, g, d_status);
    return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t stack_gemm_launch(StackProb* probs, const int* counts, int n, unsigned* d_status, int num_sms,
                              cudaStream_t stream) {
    long long tiles = 0;
    for (int i = 0; i < n; ++i) {
        StackProb& P = probs[i];
        P.mbs = (P.M + BM - 1) / BM;
        P.nbs = (P.N + BN - 1) / BN;
        P.block_tiles = stack_block_tiles(P.mbs, P.nbs, (P.flags & kStackSym) != 0);
        P.tile0 = static_cast<int>(tiles);
        tiles += static_cast<long long>(P.block_tiles) * counts[i];
    }
    if (tiles <= 0) return cudaSuccess;
    if (n > kStackMaxProbs || tiles > INT32_MAX) return cudaErrorInvalidValue;
    // Parameters of up to 4 KB launch in 4 us, larger ones in 30 to 40 (10 KB): few problems take the small form.
    static_assert(sizeof(GemmParams<kFewProbs>) <= 4000, "the small form's parameters stay below 4 KB");
    return n <= kFewProbs ? launch<kFewProbs>(probs, n, static_cast<int>(tiles), d_status, num_sms, stream)
                          : launch<kStackMaxProbs>(probs, n, static_cast<int>(tiles), d_status, num_sms, stream);
}

}  // namespace muon
