// Newton-Schulz orthogonalisation, or the whole Muon step, of blocks with a short side of at most 128
// (attention heads, low-rank factors, small matrices): one launch, one cluster per block, the block on
// chip from its first read to its last write.
//
// With r <= 128 an iteration is 6 r^2 s flops on a matrix that fits a cluster's shared memory; run as
// grouped GEMMs its three products would each read and write X from L2 with a launch in between (96
// heads of 128 x 4096: 1.31 ms of products and 0.24 ms of passes, against 0.11 ms for its HBM bytes).
//
// The block, turned so that X is r x s, is cut along s into slabs of w <= 512 columns, one per CTA:
//  - state Z = X * u / (a_0 ... a_{t-1}) in TMEM, fp32, 128 lanes x w columns.  In these units an
//    iteration X' = aX + BX is Z' = Z + B~ X^, the accumulation that the tensor core does anyway: the
//    state never leaves TMEM, and the term aX keeps 24 bits at no cost;
//  - X^ = fp16(X * tau) in shared memory as 64-column panels of 128 rows x 128 bytes, 128-byte swizzled.
//    The same panel is a K-major operand (Gram matrix, K = columns) and an MN-major one (apply, N =
//    columns).
// Per iteration: the slab's Gram matrix (M = N = 128, K = w); its rows go to their owner CTAs by
// asynchronous stores to distributed shared memory that count on the receiver's mbarrier, the owners sum
// them in rank order and send fp16 A to every CTA the same way; every CTA forms B~ = kappa (bA + cA^2)
// for itself; Z += B~ X^.  One cluster barrier an iteration, split around the conversion of Z to X^, says
// that a CTA's buffers are free again.  (With cluster barriers after each exchange and rows of 16 bytes
// per lane an iteration at w = 512 took 12.2 us, 5.6 of them in the exchanges.)
//
// In and out: one coalesced pass over G and M (M written, norm in fp64) puts U into TMEM as it is; once
// the norm is known it is scaled there.  Results go back through the same staging.  A step reads and
// writes each byte of HBM once.
#include <atomic>
#include <cmath>

#include "../../include/muon_b200.h"
#include "stacks.cuh"
#include "typed_io.cuh"

namespace muon {
namespace {

constexpr int THREADS = 512;
constexpr int PANEL = 128 * 128;                 // bytes: 128 rows x 64 fp16
constexpr int A_BYTES = 2 * PANEL;               // 128 x 128 fp16
constexpr int RED_BYTES = 128 * 128 * 4;         // partial rows of A from every CTA; then B~ (first half)
constexpr int FIXED_BYTES = A_BYTES + RED_BYTES;
constexpr int STG_PITCH = 65;                    // floats per staged row of 64: conflict-free down a column
constexpr int STG_FLOATS = 128 * STG_PITCH;
static_assert(2 * STG_FLOATS * 4 <= FIXED_BYTES, "two staging buffers overlay A and the partial rows");
constexpr int TMEM_COLS = 512, ACC = 384;        // Gram and A^2 accumulate in columns ACC .. ACC + 127

__host__ __device__ constexpr int smem_bytes(int w) { return (w / 64) * PANEL + FIXED_BYTES + 1024; }
static_assert(smem_bytes(kSmallStackSlab) + 512 <= 232448, "shared memory above the 227 KB per-CTA limit");

__device__ __forceinline__ void fence_async_proxy() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
// 16 bytes into a CTA of the cluster, counted on that CTA's mbarrier.
__device__ __forceinline__ void st_async_v4(uint32_t a, uint32_t bar, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(a),
                 "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void st_cluster_f64(uint32_t a, double x) {
    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(a), "d"(x) : "memory");
}
__device__ __forceinline__ void tmem_ld_x16(uint32_t t, float (&v)[16]) {
    uint32_t r[16];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(t)
        : "memory");
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_st_x16(uint32_t t, const float* v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(t),
        "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3])),
        "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])), "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])),
        "r"(__float_as_uint(v[8])), "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
        "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])), "r"(__float_as_uint(v[15]))
        : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint32_t half2_bits(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// 16 values of row `row`, columns c .. c + 15 (c a multiple of 16), times f, as fp16 into the panels.
__device__ __forceinline__ void put_panel16(uint8_t* panels, int row, int c, const float (&v)[16], float f) {
    uint8_t* p = panels + (c >> 6) * PANEL + row * 128;
    const int s = (c & 63) >> 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float* x = v + 8 * h;
        *reinterpret_cast<uint4*>(p + (((s + h) ^ (row & 7)) << 4)) =
            make_uint4(half2_bits(x[0] * f, x[1] * f), half2_bits(x[2] * f, x[3] * f), half2_bits(x[4] * f, x[5] * f),
                       half2_bits(x[6] * f, x[7] * f));
    }
}

struct Group {      // 8 consecutive elements of the caller's arrays: row, first column, valid count
    int row, col, n;
    int i, c;       // X's row and chunk column of the first one
};

struct alignas(16) SmallParamsS {
    SmallStackItem item[kSmallStackItems];
    SmallStackClass k;
    int n;
};

__global__ void __launch_bounds__(THREADS, 1) stack_small_kernel(const __grid_constant__ SmallParamsS p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t bar_gram, bar_square, bar_apply[2], bar_rows, bar_a;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ double red_norm[THREADS / 32];
    __shared__ double parts[16];

    const SmallStackClass& k = p.k;
    const int C = k.cluster, w = k.slab;
    uint8_t* panels = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* Am = panels + (w >> 6) * PANEL;
    uint8_t* red = Am + A_BYTES;
    uint8_t* Bm = red;
    float* stg = reinterpret_cast<float*>(Am);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int blk = static_cast<int>(blockIdx.x) / C;
    int lo = 0, hi = p.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.item[mid].block0 <= blk) lo = mid; else hi = mid - 1;
    }
    const SmallStackItem& it = p.item[lo];
    const long long b = blk - it.block0;
    const bool tall = k.rows > k.cols;
    const int c0 = rank * w;                       // first column of this slab
    const int q = warp & 3, cg = warp >> 2;        // TMEM lane quarter, column group
    const int row = 32 * q + lane;                 // this thread's row of X
    const int nchunk = w >> 6;
    const float gs = k.gscale != nullptr ? __ldg(k.gscale) : 1.f;
    const bool mom = it.M != nullptr;

    if (tid == 0) {
        for (uint64_t* x : {&bar_gram, &bar_square, &bar_apply[0], &bar_apply[1], &bar_rows, &bar_a}) mbar_init(x, 1);
        abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(&tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(32 * q) << 16);
    volatile int* abort = &abort_flag;
    unsigned* status = k.status;

    // Group e (0 or 1) of this thread in 64-column chunk ch.
    auto group = [&](int ch, int e) {
        Group g;
        const int i = e * THREADS + tid;
        if (!tall) {
            g.i = i >> 3;
            g.c = (i & 7) * 8;
            g.row = g.i;
            g.col = c0 + ch * 64 + g.c;
            g.n = g.row < k.rows ? max(0, min(8, k.cols - g.col)) : 0;
        } else {
            g.c = i >> 4;
            g.i = (i & 15) * 8;
            g.row = c0 + ch * 64 + g.c;
            g.col = g.i;
            g.n = g.row < k.rows ? max(0, min(8, k.cols - g.col)) : 0;
        }
        return g;
    };
    auto at = [&](const Group& g, long long stride, int ld) { return b * stride + static_cast<long long>(g.row) * ld + g.col; };

    // ---------------------------------------------------------------- momentum, norm, U -> TMEM
    // Two chunks of loads in flight.
    double ss = 0.0;
    struct Raw {
        float g[2][8], m[2][8];
    };
    auto fetch = [&](int ch, Raw& x) {
        if (ch >= nchunk) return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const Group g = group(ch, e);
            load8(it.G, it.g_dtype, at(g, it.g_stride, it.g_ld), g.n, it.vec & 1, x.g[e]);
            if (mom) load8(it.M, MUON_F32, at(g, it.m_stride, it.m_ld), g.n, it.vec & 2, x.m[e]);
        }
    };
    auto take = [&](int ch, Raw& x) {
        if (ch >= nchunk) return;
        float* s = stg + (ch & 1) * STG_FLOATS;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const Group g = group(ch, e);
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                float u = x.g[e][h] * gs;
                if (mom) {
                    x.m[e][h] = fmaf(k.beta, x.m[e][h], u);
                    u = k.nesterov ? fmaf(k.beta, x.m[e][h], u) : x.m[e][h];
                }
                if (h >= g.n) u = 0.f;     // 0 * a NaN factor is not zero
                ss = fma(static_cast<double>(u), static_cast<double>(u), ss);
                if (!tall) s[g.i * STG_PITCH + g.c + h] = u;
                else s[(g.i + h) * STG_PITCH + g.c] = u;
            }
            if (mom) store8(it.M, MUON_F32, at(g, it.m_stride, it.m_ld), g.n, it.vec & 2, x.m[e]);
        }
        __syncthreads();
        float z[16];
#pragma unroll
        for (int h = 0; h < 16; ++h) z[h] = s[row * STG_PITCH + cg * 16 + h];
        tmem_st_x16(t_lane + ch * 64 + cg * 16, z);
    };
    {
        Raw x0, x1;
        fetch(0, x0);
        fetch(1, x1);
        for (int ch = 0; ch < nchunk; ch += 2) {
            take(ch, x0);
            fetch(ch + 2, x0);
            take(ch + 1, x1);
            fetch(ch + 3, x1);
        }
    }
    tmem_st_wait();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (lane == 0) red_norm[warp] = ss;
    __syncthreads();
    cluster_arrive();      // every CTA of the cluster runs
    cluster_wait();
    if (tid < C) {
        double s = 0.0;
        for (int i = 0; i < THREADS / 32; ++i) s += red_norm[i];
        st_cluster_f64(mapa_shared(smem_u32(&parts[rank]), tid), s);
    }
    cluster_arrive();
    cluster_wait();
    double sum = 0.0;
    for (int i = 0; i < C; ++i) sum += parts[i];
    const double norm = sqrt(sum);
    const bool fin = isfinite(norm);
    if (tid == 0 && rank == 0 && !fin) atomicOr(status, kDevErrNonfinite);
    {
        // Z_0 = U * 2^e * zf, so that neither factor leaves fp32's range
        int ex = 0;
        if (fin && norm > 0.0) ex = max(-126, min(126, -(ilogb(norm) + 1)));
        const float up = __int_as_float((ex + 127) << 23);
        const float zf = !fin ? NAN
                              : norm > 0.0 ? static_cast<float>(static_cast<double>(k.unit) /
                                                                ((norm + static_cast<double>(k.eps)) * static_cast<double>(up)))
                                           : 0.f;
        const float zs = k.it[0].zs;
        for (int c = cg * 16; c < w; c += 64) {
            float z[16];
            tmem_ld_x16(t_lane + c, z);
#pragma unroll
            for (int h = 0; h < 16; ++h) z[h] = (z[h] * up) * zf;
            tmem_st_x16(t_lane + c, z);
            put_panel16(panels, row, c, z, zs);
        }
        tmem_st_wait();
    }
    fence_async_proxy();
    tc_fence_before();
    __syncthreads();
    if (C > 1) cluster_arrive();      // staging is over: peers may write into this CTA's buffers

    // ---------------------------------------------------------------- iterations
    const bool spill = w > ACC;
    const int rc = 128 / C;                        // rows of the Gram matrix that a CTA owns
    const int own = row / rc, orow = row - own * rc, rmask = min(rc, 8) - 1;
    const uint32_t idesc = idesc_f16_f32(128, 128, 0, 0);
    const uint32_t pan0 = smem_u32(panels), a0 = smem_u32(Am), b0 = smem_u32(Bm);
    const int pn = cg >> 1, ps = (cg & 1) * 4;     // panel and first 16-byte piece of columns 32 cg ...
    for (int t = 0; t < k.iters; ++t) {
        const SmallStackIter& f = k.it[t];
        const uint32_t phase = t & 1;
        float sp[32];
        if (spill) {       // the state's last columns make room for the small products
            uint32_t r[32];
            tmem_ld_32x32b_x32(t_lane + ACC + 32 * cg, r);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) sp[i] = __uint_as_float(r[i]);
            tc_fence_before();
            __syncthreads();
        }
        if (tid == 0) {
            if (C > 1) {
                mbar_arrive_expect_tx(&bar_rows, RED_BYTES);
                mbar_arrive_expect_tx(&bar_a, A_BYTES);
            }
            tc_fence_after();
            fence_async_proxy();
            for (int j = 0; j < nchunk; ++j)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint64_t d = smem_desc_sw128(pan0 + j * PANEL + s * 32, 16, 1024);
                    tc_mma_bf16(tmem + ACC, d, d, idesc, j + s > 0);   // kind::f16, types from idesc
                }
            tc_commit(&bar_gram);
        }
        mbar_wait(&bar_gram, phase, abort, status);
        __syncwarp();
        tc_fence_after();
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_lane + ACC + 32 * cg, r);
        tmem_ld_wait();
        tc_fence_before();
        if (C > 1) {
            // Partial rows to their owners, as [rank][16-byte piece][row]: a warp's store of one piece fills
            // whole sectors, and the row's place is turned by the piece so that the owner reads without
            // bank conflicts.
            cluster_wait();        // every CTA's buffers are free
            const uint32_t dst = mapa_shared(smem_u32(red), own) + static_cast<uint32_t>(rank * rc * 512);
            const uint32_t bar = mapa_shared(smem_u32(&bar_rows), own);
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int seg = 8 * cg + s;
                st_async_v4(dst + ((seg * rc + (orow ^ (seg & rmask))) << 4), bar, r[4 * s], r[4 * s + 1], r[4 * s + 2], r[4 * s + 3]);
            }
            mbar_wait(&bar_rows, phase, abort, status);
            __syncwarp();
            // rows rank * rc ... of A: the sum over the cluster in rank order, 8 columns a thread, to every CTA
            for (int g = tid; g < rc * 16; g += THREADS) {
                const int rr = g >> 4, pc = g & 15, ar = rank * rc + rr;
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int seg = 2 * pc + h;
                    const uint8_t* src = red + ((seg * rc + (rr ^ (seg & rmask))) << 4);
                    for (int i = 0; i < C; ++i) {
                        const float4 x = *reinterpret_cast<const float4*>(src + i * rc * 512);
                        v[4 * h] += x.x; v[4 * h + 1] += x.y; v[4 * h + 2] += x.z; v[4 * h + 3] += x.w;
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[e] *= f.ga;
                    if (8 * pc + e == ar) v[e] -= f.diag;
                }
                const uint4 x = pack8(MUON_F16, v);
                const uint32_t off = (pc >> 3) * PANEL + ar * 128 + (((pc & 7) ^ (ar & 7)) << 4);
                for (int i = 0; i < C; ++i) {
                    const int to = (rank + i) & (C - 1);
                    st_async_v4(mapa_shared(a0 + off, to), mapa_shared(smem_u32(&bar_a), to), x.x, x.y, x.z, x.w);
                }
            }
            mbar_wait(&bar_a, phase, abort, status);
            __syncwarp();
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[e] = __uint_as_float(r[8 * s + e]) * f.ga;
                    if (32 * cg + 8 * s + e == row) v[e] -= f.diag;
                }
                *reinterpret_cast<uint4*>(Am + pn * PANEL + row * 128 + (((ps + s) ^ (row & 7)) << 4)) = pack8(MUON_F16, v);
            }
        }
        fence_async_proxy();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const uint64_t d = smem_desc_sw128(a0 + (s >> 2) * PANEL + (s & 3) * 32, 16, 1024);
                tc_mma_bf16(tmem + ACC, d, d, idesc, s > 0);
            }
            tc_commit(&bar_square);
        }
        mbar_wait(&bar_square, phase, abort, status);
        __syncwarp();
        tc_fence_after();
        tmem_ld_32x32b_x32(t_lane + ACC + 32 * cg, r);
        tmem_ld_wait();
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const uint32_t off = pn * PANEL + row * 128 + (((ps + s) ^ (row & 7)) << 4);
            float av[8];
            unpack8(*reinterpret_cast<const uint4*>(Am + off), MUON_F16, av);
#pragma unroll
            for (int e = 0; e < 8; ++e) av[e] = fmaf(f.pb, av[e], f.pc * __uint_as_float(r[8 * s + e]));
            *reinterpret_cast<uint4*>(Bm + off) = pack8(MUON_F16, av);
        }
        if (spill) {
            tmem_st_x16(t_lane + ACC + 32 * cg, sp);
            tmem_st_x16(t_lane + ACC + 32 * cg + 16, sp + 16);
            tmem_st_wait();
        }
        fence_async_proxy();
        tc_fence_before();
        __syncthreads();
        if (tid == 0) {
            tc_fence_after();
            for (int n0 = 0; n0 < w; n0 += 256) {
                const int n = min(256, w - n0);
                const uint32_t id = idesc_f16_f32(128, n, 0, 1);
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint64_t ad = smem_desc_sw128(b0 + (s >> 2) * PANEL + (s & 3) * 32, 16, 1024);
                    const uint64_t xd = smem_desc_sw128(pan0 + (n0 >> 6) * PANEL + s * 2048, PANEL, 1024);
                    tc_mma_bf16(tmem + n0, ad, xd, id, 1);
                }
                tc_commit(&bar_apply[n0 >> 8]);
            }
        }
        // The first 256 columns are converted while the others are multiplied.
        const bool last = t + 1 == k.iters;
        const float zs = k.it[last ? t : t + 1].zs;
        for (int n0 = 0; n0 < w; n0 += 256) {
            mbar_wait(&bar_apply[n0 >> 8], phase, abort, status);
            __syncwarp();
            tc_fence_after();
            if (!last && n0 + 256 >= w && C > 1) cluster_arrive();   // this CTA's A, B~ and partial rows are done with
            const int nq = min(256, w - n0) >> 2;
            if (!last)
                for (int c = n0 + cg * nq; c < n0 + (cg + 1) * nq; c += 16) {
                    float z[16];
                    tmem_ld_x16(t_lane + c, z);
                    put_panel16(panels, row, c, z, zs);
                }
        }
        if (!last) {
            fence_async_proxy();
            tc_fence_before();
            __syncthreads();
        }
    }

    // ---------------------------------------------------------------- result
    // Peers' last stores into this CTA are the last rows of A, which it has waited for.
    const float out = k.out;
    const bool update = it.decay != 0.f;
    auto fetch_w = [&](int ch, float (&x)[2][8]) {
        if (!update || ch >= nchunk) return;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const Group g = group(ch, e);
            load8(it.W, it.w_dtype, at(g, it.w_stride, it.w_ld), g.n, it.vec & 4, x[e]);
        }
    };
    auto give = [&](int ch, float (&x)[2][8]) {
        if (ch >= nchunk) return;
        float* s = stg + (ch & 1) * STG_FLOATS;
        float z[16];
        tmem_ld_x16(t_lane + ch * 64 + cg * 16, z);
#pragma unroll
        for (int h = 0; h < 16; ++h) s[row * STG_PITCH + cg * 16 + h] = z[h] * out;
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const Group g = group(ch, e);
            if (g.n == 0) continue;
            float o[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) {
                const float v = !tall ? s[g.i * STG_PITCH + g.c + h] : s[(g.i + h) * STG_PITCH + g.c];
                o[h] = update ? fmaf(it.step, v, it.decay * x[e][h]) : it.step * v;
            }
            store8(it.W, it.w_dtype, at(g, it.w_stride, it.w_ld), g.n, it.vec & 4, o);
        }
    };
    {
        float x0[2][8], x1[2][8];
        fetch_w(0, x0);
        fetch_w(1, x1);
        __syncthreads();       // every warp is past the last reads of A and B~
        for (int ch = 0; ch < nchunk; ch += 2) {
            give(ch, x0);
            fetch_w(ch + 2, x0);
            give(ch + 1, x1);
            fetch_w(ch + 3, x1);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

}  // namespace

cudaError_t stack_small_launch(const SmallStackItem* items, int n, const SmallStackClass& k, cudaStream_t stream) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!ready[dev].load()) {
        e = cudaFuncSetAttribute(stack_small_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kSmallStackSlab));
        if (e != cudaSuccess) return e;
        ready[dev].store(true);
    }
    for (int i0 = 0; i0 < n; i0 += kSmallStackItems) {
        SmallParamsS p;
        p.n = n - i0 < kSmallStackItems ? n - i0 : kSmallStackItems;
        p.k = k;
        int blocks = 0;
        for (int i = 0; i < p.n; ++i) {
            p.item[i] = items[i0 + i];
            p.item[i].block0 = blocks;
            blocks += items[i0 + i].count;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(k.cluster) * blocks, 1, 1);
        cfg.blockDim = dim3(THREADS, 1, 1);
        cfg.dynamicSmemBytes = smem_bytes(k.slab);
        cfg.stream = stream;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = k.cluster;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, stack_small_kernel, p);
        if (e == cudaSuccess) e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace muon
