// Newton-Schulz orthogonalisation, or the whole Muon step, of blocks with a short side of at most 128
// (attention heads, low-rank factors, small matrices): one launch, one cluster per block, the block on
// chip from its first read to its last write.
//
// With r <= 128 an iteration is 6 r^2 s flops on a matrix that fits a cluster's shared memory; run as
// grouped GEMMs its three products would each read and write X from L2 with a launch in between (96
// heads of 128 x 4096: 1.31 ms of products and 0.24 ms of passes, against 0.11 ms for its HBM bytes).
//
// The block, turned so that X is r x s, is cut along s into chunks of 64 columns that the cluster's CTAs take
// in turn (so that together they walk along whole rows of the caller's arrays: pieces of 128 bytes a row would
// halve what HBM gives); a CTA's slab has w <= 512 columns:
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
// In and out: one pass over G and M (M written, norm in fp64) puts U into TMEM as it is; once the norm is
// known it is scaled there.  A step reads and writes each byte of HBM once.  Chunks come and go as TMA
// boxes, several in flight, 128-byte swizzled so that a thread finds its own row of X without bank
// conflicts, zero-filled and clipped at the block's edges.  (Loads through registers took twice as long,
// 26 us for a slab of 128 x 512: a quarter of the stalls were instruction fetches of the code for every
// type and edge, another the loads' latency.  Row by row, bulk copies took 42 us: about 20 ns each.)
// Arrays whose rows TMA cannot address go element by element through shared memory.  (TMA clips a store at
// 16 bytes, no finer, so rows of a broken number of 16-byte pieces are among them.)
//
// Where the reverse pass is to follow, the panels of X^_t and the matrices A_t and B~_t leave by TMA as they lie in
// shared memory, behind the products that read them (16 blocks of 96 x 641: 55 us without, 65 with).
//
// Bound: latency of the chain Gram, exchange, A^2, apply (12 blocks of 64 x 768: 50 us for five iterations, the
// tensor pipe 12% busy).  A cluster of 8 leaves 36 SMs idle (14 run at once); 96 steps of 128 x 4096 are 7 rounds
// of them, 549 us against 109 for their bytes.
#include <atomic>
#include <cmath>

#include "../../include/muon_b200.h"
#include "ptx_stacks.cuh"
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
static_assert(2 * STG_FLOATS * 4 <= FIXED_BYTES, "two staging buffers fit the smallest slab's shared memory");
static_assert(4 * PANEL <= FIXED_BYTES + PANEL, "one chunk of fp32 G and M fits the smallest slab's shared memory");
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

__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}

// ---------------------------------------------------------------- giving up
// What thread 0 has armed on the CTA's mbarriers (copies of its own, peers' stores): a bit per barrier that was armed at
// least once, and the parity of the phase armed last.  It waits for every phase before it arms the next.  After a wait has
// run out (kWaitLimitNs) nothing more is armed, copied in or multiplied, the cluster barriers are still met, and before
// the CTA leaves it waits (with a limit) for what is under way: a late copy or a peer's store must not find its memory
// given to another CTA.
struct Flight {
    uint32_t used = 0, parity = ~0u;
    bool ok = true;                // none of this thread's waits has run out
    __device__ __forceinline__ void arm(int bar) {
        used |= 1u << bar;
        parity ^= 1u << bar;
    }
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t phase, volatile int* abort, unsigned* status) {
        ok = mbar_wait(bar, phase, abort, status) && ok;
    }
};
__device__ __forceinline__ bool lands(uint64_t* bar, uint32_t parity) {
    const unsigned long long t0 = global_ns();
    bool landed = false;
    while (!(landed = mbar_try_wait(bar, parity)) && global_ns() - t0 < 100000000ull) {
    }
    return landed;
}
// Thread 0 at the end of a CTA that has given up: `bars` as counted by `fly`, `drain` a barrier without a phase so far.
// The products, and the signals that wait for them, end before `drain`'s.
__device__ __noinline__ void drain_flight(uint64_t* bars, int n, uint64_t* drain, const Flight fly, unsigned* status) {
    tc_commit(drain);
    bool landed = lands(drain, 0);
    for (int i = 0; i < n; ++i)
        if (fly.used >> i & 1u) landed = lands(&bars[i], fly.parity >> i & 1u) && landed;
    bulk_wait_read<0>();       // stores' reads of this CTA's memory
    // stores of peers that came after this CTA had armed its last: no barrier counts them, a millisecond is a thousand times theirs
    const unsigned long long t0 = global_ns();
    while (global_ns() - t0 < 1000000ull) __nanosleep(1000);
    if (!landed) atomicOr(status, kDevErrUndrained);
}

// ---------------------------------------------------------------- a slab in and out
struct Slab {
    int rows, cols, rank, cluster, nchunk;
    bool tall, two;        // two: a packed cluster has a second block
    uint8_t* buf;          // all of the shared memory that the iterations use, 1024-byte aligned
    int bytes;
    uint32_t t_lane;       // TMEM address of this warp's lanes
    uint64_t* bars;        // kRing mbarriers, the first of those that a Flight counts
    volatile int* abort;
    unsigned* status;
    __device__ __forceinline__ int first(int ch) const { return (ch * cluster + rank) * 64; }   // first column of a chunk
};
constexpr int kRing = 4;
constexpr int BOX = 128 * 128;   // bytes of a box: 128 rows (two times 64 for a tall block) of 128 bytes

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, uint32_t bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
        "l"(m), "r"(bar), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* m, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(m), "r"(src),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* m, int x, int y, int z) {
    asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(m), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// Packed: rows 64 .. of X are the next block's.  One array's part of a chunk: two boxes of 64 x 128 (64-column halves of a tall block's rows) or one of 128 x 64
// for 16-bit elements, twice as many for fp32.  A box's row has 128 bytes: 64 or 32 elements.
template <bool PACK>
struct Boxes {
    const CUtensorMap* map;
    int dtype, es, block;
    __device__ __forceinline__ int bytes() const { return BOX * es / 2; }
    // Calls f(byte offset in the buffer, x, y, block) for every box of the chunk at column c.
    template <class F>
    __device__ __forceinline__ void each(const Slab& s, int c, F f) const {
        const int per = 128 / es;
        if (!s.tall) {
            for (int h = 0; h < es / 2; ++h) {
                f(h * BOX, c + h * per, 0, block);
                if (PACK) f(h * BOX + BOX / 2, c + h * per, 0, block + 1);
            }
        } else {
            for (int h = 0; h < es; ++h) {
                const int i = h * per;
                f(h * (BOX / 2), PACK ? i & 63 : i, c, PACK ? block + (i >> 6) : block);
            }
        }
    }
    __device__ __forceinline__ bool there(const Slab& s, int x, int y, int z) const {
        return x < s.cols && y < s.rows && (!PACK || z == block || s.two);
    }
    __device__ __forceinline__ void load(const Slab& s, int c, uint32_t buf, uint32_t bar) const {
        each(s, c, [&](int o, int x, int y, int z) { tma_load_3d(buf + o, map, bar, x, y, z); });   // zeros where none
    }
    __device__ __forceinline__ void prefetch(const Slab& s, int c) const {
        each(s, c, [&](int, int x, int y, int z) { if (there(s, x, y, z)) tma_prefetch_3d(map, x, y, z); });
    }
    __device__ __forceinline__ void store(const Slab& s, int c, uint32_t buf) const {
        each(s, c, [&](int o, int x, int y, int z) { if (there(s, x, y, z)) tma_store_3d(map, buf + o, x, y, z); });
    }
    // This thread's 16 elements (X's row `row`, columns 16 cg ...) in a buffer: piece h (0, 1) of 8 for wide
    // blocks, element h (0..15) for tall ones.
    __device__ __forceinline__ uint8_t* piece(uint8_t* buf, int row, int cg, int h, int half) const {
        const int e = cg * 16 + 8 * h;                                   // column
        if (es == 2) return buf + row * 128 + (((e >> 3) ^ (row & 7)) << 4);
        return buf + (e >> 5) * BOX + row * 128 + (((((e & 31) >> 2) + half) ^ (row & 7)) << 4);
    }
    __device__ __forceinline__ uint8_t* elem(uint8_t* buf, int row, int c) const {
        if (es == 2) return buf + (row >> 6) * (BOX / 2) + c * 128 + ((((row & 63) >> 3) ^ (c & 7)) << 4) + (row & 7) * 2;
        return buf + (row >> 5) * (BOX / 2) + c * 128 + ((((row & 31) >> 2) ^ (c & 7)) << 4) + (row & 3) * 4;
    }
    __device__ __forceinline__ void get(const Slab& s, uint8_t* buf, int row, int cg, float (&v)[16]) const {
        if (!s.tall) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[8];
                if (es == 2) {
                    unpack8(*reinterpret_cast<const uint4*>(piece(buf, row, cg, h, 0)), dtype, x);
                } else {
                    const float4 a = *reinterpret_cast<const float4*>(piece(buf, row, cg, h, 0));
                    const float4 b = *reinterpret_cast<const float4*>(piece(buf, row, cg, h, 1));
                    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[8 * h + e] = x[e];
            }
        } else {
#pragma unroll
            for (int h = 0; h < 16; ++h) v[h] = load_elem(elem(buf, row, cg * 16 + h), dtype, 0);
        }
    }
    __device__ __forceinline__ void put(const Slab& s, uint8_t* buf, int row, int cg, const float (&v)[16]) const {
        if (!s.tall) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = v[8 * h + e];
                if (es == 2) {
                    *reinterpret_cast<uint4*>(piece(buf, row, cg, h, 0)) = pack8(dtype, x);
                } else {
                    *reinterpret_cast<float4*>(piece(buf, row, cg, h, 0)) = make_float4(x[0], x[1], x[2], x[3]);
                    *reinterpret_cast<float4*>(piece(buf, row, cg, h, 1)) = make_float4(x[4], x[5], x[6], x[7]);
                }
            }
        } else {
#pragma unroll
            for (int h = 0; h < 16; ++h) store_elem(elem(buf, row, cg * 16 + h), dtype, 0, v[h]);
        }
    }
};

// Chunk buffers that TMA fills in turn; thread 0 issues.  `turns`: the phases of the mbarriers, as bits.
template <int N, bool PACK>
struct Ring {
    Boxes<PACK> a[N];
    int n, size, bufs;
    __device__ __forceinline__ void shape(const Slab& s) {
        size = 0;
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) size += a[i].bytes();
        bufs = min(min(kRing, s.bytes / size), s.nchunk);
    }
    __device__ __forceinline__ uint8_t* buf(const Slab& s, int ch) const { return s.buf + (ch % bufs) * size; }
    __device__ __forceinline__ void fill(const Slab& s, int ch, Flight& fly) const {
        if (!fly.ok) return;
        const uint32_t bar = smem_u32(s.bars + ch % bufs);
        fly.arm(ch % bufs);
        mbar_arrive_expect_tx(s.bars + ch % bufs, size);
        uint32_t dst = smem_u32(buf(s, ch));
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i >= n) break;
            a[i].load(s, s.first(ch), dst, bar);
            dst += a[i].bytes();
        }
    }
    __device__ __forceinline__ void wait(const Slab& s, int ch, uint32_t& turns, Flight& fly) const {
        const int b = ch % bufs;
        fly.wait(s.bars + b, (turns >> b) & 1u, s.abort, s.status);
        turns ^= 1u << b;
        __syncwarp();
    }
    // After the barrier that ends chunk ch, with its store (if any) committed: fills a buffer whose chunk is done.
    // With several buffers that is the one before, whose store has had a chunk's time.
    __device__ __forceinline__ void refill(const Slab& s, int ch, Flight& fly) const {
        const int back = bufs > 1 ? ch - 1 : ch;
        if (back < 0 || back + bufs >= s.nchunk) return;
        if (bufs > 1) bulk_wait_read<1>();
        else bulk_wait_read<0>();
        fill(s, back + bufs, fly);
    }
};

struct Momentum {
    float gs, beta;
    bool on, nesterov;
    // The input of the iterations from gradient elements (in u); m is updated.  Zeros stay zeros, unless
    // the factor is not finite, and then the block is not.
    __device__ __forceinline__ void operator()(float (&u)[16], float (&m)[16]) const {
#pragma unroll
        for (int h = 0; h < 16; ++h) u[h] *= gs;
        if (on) {
#pragma unroll
            for (int h = 0; h < 16; ++h) m[h] = fmaf(beta, m[h], u[h]);
#pragma unroll
            for (int h = 0; h < 16; ++h) u[h] = nesterov ? fmaf(beta, m[h], u[h]) : m[h];
        }
    }
};
__device__ __forceinline__ float sum_squares(const float (&u)[16]) {
    float s = 0.f;
#pragma unroll
    for (int h = 0; h < 16; ++h) s = fmaf(u[h], u[h], s);
    return s;
}

// The element-wise walk of a chunk: element (a, h) of a thread, A x H = 16 of them, a warp along the caller's
// rows.  Offsets are a base and two steps.
template <bool TALL, bool PACK>
struct Walk {
    static constexpr int A = TALL ? 4 : 8, H = 16 / A;
    int row, col;              // the caller's, of element (0, 0)
    int rows, cols;
    bool two;
    long long at;              // its place in an array with row pitch ld
    int staged;                // its place in the staging buffer
    __device__ __forceinline__ Walk(const Slab& s, int ch, int ld) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        row = warp + (TALL ? s.first(ch) : 0);
        col = lane + (TALL ? 0 : s.first(ch));
        rows = s.rows;
        cols = s.cols;
        two = s.two;
        at = static_cast<long long>(row) * ld + col;
        staged = TALL ? lane * STG_PITCH + warp : warp * STG_PITCH + lane;
    }
    // Whether element (a, h) is the second block's, and its place from that of (0, 0).
    static __device__ __forceinline__ constexpr bool second(int a, int h) { return PACK && (TALL ? h >= 2 : a >= 4); }
    static __device__ __forceinline__ long long step(int a, int h, long long ld16, long long stride) {
        if (!PACK) return a * ld16 + 32 * h;
        return (TALL ? a * ld16 + 32 * (h & 1) : (a & 3) * ld16 + 32 * h) + (second(a, h) ? stride : 0ll);
    }
    __device__ __forceinline__ bool ok(int a, int h) const {
        return row + 16 * (PACK && !TALL ? a & 3 : a) < rows && col + 32 * (PACK && TALL ? h & 1 : h) < cols && (!second(a, h) || two);
    }
    __device__ __forceinline__ int place(int a, int h) const {
        return staged + (TALL ? 32 * h * STG_PITCH + 16 * a : 16 * a * STG_PITCH + 32 * h);
    }
};

// Out of line: their registers and code are not the iterations'.
template <bool TALL, bool PACK>
__device__ __noinline__ double slab_in_any(const Slab s, const SmallStackItem& item, long long b, const Momentum mo) {
    using W = Walk<TALL, PACK>;
    const int g_dtype = item.g_dtype, warp = threadIdx.x >> 5, row = 32 * (warp & 3) + (threadIdx.x & 31), cg = warp >> 2;
    const uint8_t* g0 = static_cast<const uint8_t*>(item.G) + b * item.g_stride * (g_dtype == MUON_F32 ? 4 : 2);
    float* m0 = item.M + b * item.m_stride;
    const int g_ld = item.g_ld, m_ld = item.m_ld;
    const long long g16 = 16ll * g_ld, m16 = 16ll * m_ld;
    double ss = 0.0;
    float u[16], m[16];
    auto fetch = [&](int ch) {
        const W g(s, ch, g_ld), k(s, ch, m_ld);
        by_type(g_dtype, [&](auto t) {
            const decltype(t)* p = reinterpret_cast<const decltype(t)*>(g0) + g.at;
#pragma unroll
            for (int a = 0; a < W::A; ++a)
#pragma unroll
                for (int h = 0; h < W::H; ++h) u[a * W::H + h] = g.ok(a, h) ? widen(p[W::step(a, h, g16, item.g_stride)]) : 0.f;
        });
        if (mo.on) {
#pragma unroll
            for (int a = 0; a < W::A; ++a)
#pragma unroll
                for (int h = 0; h < W::H; ++h) m[a * W::H + h] = k.ok(a, h) ? m0[k.at + W::step(a, h, m16, item.m_stride)] : 0.f;
        }
    };
    fetch(0);
#pragma unroll 1
    for (int ch = 0; ch < s.nchunk; ++ch) {
        float* buf = reinterpret_cast<float*>(s.buf) + (ch & 1) * STG_FLOATS;
        mo(u, m);
        ss += static_cast<double>(sum_squares(u));
        const W k(s, ch, m_ld);
#pragma unroll
        for (int a = 0; a < W::A; ++a)
#pragma unroll
            for (int h = 0; h < W::H; ++h) {
                buf[k.place(a, h)] = u[a * W::H + h];
                if (mo.on && k.ok(a, h)) m0[k.at + W::step(a, h, m16, item.m_stride)] = m[a * W::H + h];
            }
        if (ch + 1 < s.nchunk) fetch(ch + 1);      // on its way while this chunk goes to TMEM
        __syncthreads();
        float z[16];
#pragma unroll
        for (int h = 0; h < 16; ++h) z[h] = buf[row * STG_PITCH + cg * 16 + h];
        tmem_st_x16(s.t_lane + ch * 64 + cg * 16, z);
    }
    return ss;
}
template <bool TALL, bool PACK>
__device__ __noinline__ void slab_out_any(const Slab s, const SmallStackItem& item, long long b, float out) {
    using W = Walk<TALL, PACK>;
    const int w_dtype = item.w_dtype, warp = threadIdx.x >> 5, row = 32 * (warp & 3) + (threadIdx.x & 31), cg = warp >> 2;
    uint8_t* w0 = static_cast<uint8_t*>(item.W) + b * item.w_stride * (w_dtype == MUON_F32 ? 4 : 2);
    const int w_ld = item.w_ld;
    const long long w16 = 16ll * w_ld;
    const float decay = item.decay, step = item.step * out;
    const bool update = item.M != nullptr;     // a step, also with a decay of zero: what is not finite in W stays so
    by_type(w_dtype, [&](auto t) {
        using E = decltype(t);
        E x[16];
        auto fetch = [&](int ch) {
            if (!update) return;
            const W k(s, ch, w_ld);
            const E* p = reinterpret_cast<const E*>(w0) + k.at;
#pragma unroll
            for (int a = 0; a < W::A; ++a)
#pragma unroll
                for (int h = 0; h < W::H; ++h)
                    if (k.ok(a, h)) x[a * W::H + h] = p[W::step(a, h, w16, item.w_stride)];
        };
        fetch(0);
#pragma unroll 1
        for (int ch = 0; ch < s.nchunk; ++ch) {
            float* buf = reinterpret_cast<float*>(s.buf) + (ch & 1) * STG_FLOATS;
            float z[16];
            tmem_ld_x16(s.t_lane + ch * 64 + cg * 16, z);
#pragma unroll
            for (int h = 0; h < 16; ++h) buf[row * STG_PITCH + cg * 16 + h] = z[h];
            __syncthreads();
            const W k(s, ch, w_ld);
            E* p = reinterpret_cast<E*>(w0) + k.at;
#pragma unroll
            for (int a = 0; a < W::A; ++a)
#pragma unroll
                for (int h = 0; h < W::H; ++h) {
                    const float v = buf[k.place(a, h)];
                    if (k.ok(a, h))
                        narrow(p[W::step(a, h, w16, item.w_stride)], update ? fmaf(step, v, decay * widen(x[a * W::H + h])) : step * v);
                }
            if (ch + 1 < s.nchunk) fetch(ch + 1);
        }
    });
}

template <int N>
struct SmallParams {
    SmallStackItem item[N];
    SmallStackClass k;
    int n;
};
constexpr int kFewItems = 5;
static_assert(sizeof(SmallParams<kFewItems>) <= 4096, "the small form's parameters launch faster");

// PACK: two blocks with a short side of at most 64 share a cluster.  Their Gram matrices are the diagonal quarters of
// the 128 x 128 product; the others are set to zero, and with them those of B~, so that neither block sees the other
// (192 steps of 64 x 1024: 2 rounds of clusters instead of 3, 230 and 169 us).
template <int N, bool PACK>
__global__ void __launch_bounds__(THREADS, 1) stack_small_kernel(const __grid_constant__ SmallParams<N> p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t bar_fly[kRing + 2], bar_gram, bar_square, bar_apply[2], bar_drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ double red_norm[THREADS / 32];
    __shared__ double parts[PACK ? 2 : 1][16];

    constexpr int kRows = kRing, kA = kRing + 1;   // places in bar_fly, after the ring
    uint64_t &bar_rows = bar_fly[kRows], &bar_a = bar_fly[kA];
    Flight fly;
    const SmallStackClass& k = p.k;
    const int C = k.cluster, w = k.slab;
    uint8_t* panels = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* Am = panels + (w >> 6) * PANEL;
    uint8_t* red = Am + A_BYTES;
    uint8_t* Bm = red;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int blk = static_cast<int>(blockIdx.x) / C;
    int lo = 0, hi = p.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.item[mid].block0 <= blk) lo = mid; else hi = mid - 1;
    }
    const SmallStackItem& it = p.item[lo];
    const long long b = (PACK ? 2 : 1) * static_cast<long long>(blk - it.block0);
    const bool tall = k.rows > k.cols;
    const int q = warp & 3, cg = warp >> 2;        // TMEM lane quarter, column group
    const int row = 32 * q + lane;                 // this thread's row of X
    const int half = PACK ? q >> 1 : 0;            // its block of the two
    const int nchunk = w >> 6;
    const float gs = k.gscale != nullptr ? __ldg(k.gscale) : 1.f;
    const bool mom = it.M != nullptr;

    if (tid == 0) {
        for (uint64_t* x : {&bar_gram, &bar_square, &bar_apply[0], &bar_apply[1], &bar_drain}) mbar_init(x, 1);
        for (uint64_t& x : bar_fly) mbar_init(&x, 1);
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

    const bool two = PACK && b + 1 < it.count;
    const Slab slab = {k.rows, k.cols, rank, C, nchunk, tall, two, panels, (w >> 6) * PANEL + FIXED_BYTES, t_lane, bar_fly, abort, status};
    const Momentum mo = {gs, k.beta, mom, k.nesterov != 0};
    const bool tma_in = (it.vec & 1) && (!mom || (it.vec & 2)), tma_out = (it.vec & 4) != 0, update = mom;   // a step
    const Boxes<PACK> boxes_w = {&it.map_w, it.w_dtype, it.w_dtype == MUON_F32 ? 4 : 2, static_cast<int>(b)};
    uint32_t turns = 0;

    // ---------------------------------------------------------------- momentum, norm, U -> TMEM
    double ss = 0.0;
    if (tma_in) {
        Ring<2, PACK> ring;
        ring.a[0] = {&it.map_g, it.g_dtype, it.g_dtype == MUON_F32 ? 4 : 2, static_cast<int>(b)};
        ring.a[1] = {&it.map_m, MUON_F32, 4, static_cast<int>(b)};
        ring.n = mom ? 2 : 1;
        ring.shape(slab);
        if (tid == 0) {
            for (int ch = 0; ch < ring.bufs; ++ch) ring.fill(slab, ch, fly);
            if (tma_out && update)      // on its way to L2 while the block iterates
                for (int ch = 0; ch < nchunk; ++ch) boxes_w.prefetch(slab, slab.first(ch));
        }
#pragma unroll 1
        for (int ch = 0; ch < nchunk; ++ch) {
            ring.wait(slab, ch, turns, fly);
            uint8_t* buf = ring.buf(slab, ch);
            uint8_t* buf_m = buf + ring.a[0].bytes();
            float u[16], m[16];
            ring.a[0].get(slab, buf, row, cg, u);
            if (mom) ring.a[1].get(slab, buf_m, row, cg, m);
            mo(u, m);
            ss += static_cast<double>(sum_squares(u));   // 16 squares in fp32 at most
            tmem_st_x16(t_lane + ch * 64 + cg * 16, u);
            if (mom) {
                ring.a[1].put(slab, buf_m, row, cg, m);
                fence_async_proxy();
            }
            __syncthreads();
            if (tid == 0) {
                if (mom) {
                    ring.a[1].store(slab, slab.first(ch), smem_u32(buf_m));
                    bulk_commit();
                }
                ring.refill(slab, ch, fly);
            }
        }
        if (tid == 0) bulk_wait_read<0>();
        __syncthreads();       // the buffers are free
    } else {
        ss = tall ? slab_in_any<true, PACK>(slab, it, b, mo) : slab_in_any<false, PACK>(slab, it, b, mo);
        if (PACK) {            // a thread of that walk has elements of both blocks
            tmem_st_wait();
            tc_fence_before();
            __syncthreads();
            tc_fence_after();
            ss = 0.0;
            for (int c = cg * 16; c < w; c += 64) {
                float z[16];
                tmem_ld_x16(t_lane + c, z);
                ss += static_cast<double>(sum_squares(z));
            }
        }
    }
    tmem_st_wait();
    double sum = 0.0;
    for (int again = 0; again < 2; ++again) {
        if (again) {       // squares outside fp32's range: once more in fp64, from TMEM
            ss = 0.0;
            for (int c = cg * 16; c < w; c += 64) {
                float z[16];
                tmem_ld_x16(t_lane + c, z);
#pragma unroll
                for (int h = 0; h < 16; ++h) ss = fma(static_cast<double>(z[h]), static_cast<double>(z[h]), ss);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (lane == 0) red_norm[warp] = ss;
        __syncthreads();
        cluster_arrive();      // every CTA of the cluster runs, and is past its last read of `parts`
        cluster_wait();
        if (tid < (PACK ? 2 * C : C)) {
            const int to = tid & (C - 1), of = tid / C;
            double s = 0.0;
            for (int i = 0; i < THREADS / 32; ++i)
                if (!PACK || ((i & 3) >> 1) == of) s += red_norm[i];
            st_cluster_f64(mapa_shared(smem_u32(&parts[of][rank]), to), s);
        }
        cluster_arrive();
        cluster_wait();
        double sums[2] = {0.0, 0.0};
#pragma unroll
        for (int of = 0; of < (PACK ? 2 : 1); ++of)
            for (int i = 0; i < C; ++i) sums[of] += parts[of][i];
        sum = PACK && half ? sums[1] : sums[0];
        // the same in every thread of the cluster
        if (sums[0] > 1e-25 && sums[0] < 1e36 && (!two || (sums[1] > 1e-25 && sums[1] < 1e36))) break;
    }
    const double norm = sqrt(sum);
    const bool fin = isfinite(norm);
    if (lane == 0 && (warp == 0 || (PACK && warp == 2)) && rank == 0 && !fin) atomicOr(status, kDevErrNonfinite);
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
            for (int h = 0; h < 16; ++h) z[h] = fin ? (z[h] * up) * zf : 0.f;   // nothing of it into another block
            tmem_st_x16(t_lane + c, z);
            put_panel16(panels, row, c, z, zs);
        }
        tmem_st_wait();
    }
    fence_async_proxy();
    tc_fence_before();
    __syncthreads();
    if (C > 1) cluster_arrive();      // staging is over: peers may write into this CTA's buffers

    // What the reverse pass reads, kept as it lies in shared memory (thread 0): X^_t from every CTA, A_t and
    // B~_t from the first.
    const bool keep = k.saved != 0;
    const int keep_z = keep ? it.at + static_cast<int>(b) : 0, r_true = min(k.rows, k.cols), s_true = max(k.rows, k.cols);
    auto keep_x = [&](int t) {
        for (int j = 0; j < nchunk; ++j) {
            const int x = slab.first(j);
            if (x >= s_true) break;
            for (int y = 0; y < (PACK ? two ? 128 : 64 : r_true); y += 64)
                tma_store_3d(&k.x, smem_u32(panels) + j * PANEL + y * 128, x, PACK ? 0 : y, t * k.saved + keep_z + (PACK ? y >> 6 : 0));
        }
        bulk_commit();
    };
    auto keep_square = [&](const CUtensorMap* m, const uint8_t* src, int t) {
        if (rank != 0) return;
        if (PACK) {
            for (int of = 0; of < (two ? 2 : 1); ++of)
                tma_store_3d(m, smem_u32(src) + of * (PANEL + 64 * 128), 0, 0, t * k.saved + keep_z + of);
        } else
        for (int x = 0; x < r_true; x += 64)
            for (int y = 0; y < r_true; y += 64)
                tma_store_3d(m, smem_u32(src) + (x >> 6) * PANEL + y * 128, x, y, t * k.saved + keep_z);
        bulk_commit();
    };
    if (keep && tid == 0) keep_x(0);
    if (keep && lane == 0) {
        if (rank == 0 && (warp == 0 || (two && warp == 2))) {
            float* info = k.info + static_cast<size_t>(keep_z + half) * kStackInfo;
            info[0] = !fin ? NAN : norm > 0.0 ? k.f0 : 0.f;
            info[1] = 1.f;
            info[2] = static_cast<float>(1.0 / (norm + static_cast<double>(k.eps)));
            info[3] = static_cast<float>(norm);
        }
    }

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
        if (tid == 0 && fly.ok) {
            if (C > 1) {
                fly.arm(kRows);
                fly.arm(kA);
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
        fly.wait(&bar_gram, phase, abort, status);
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
            fly.wait(&bar_rows, phase, abort, status);
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
                    v[e] = PACK && (pc >> 3) != (ar >> 6) ? 0.f : v[e] * f.ga;
                    if (8 * pc + e == ar) v[e] -= f.diag;
                }
                const uint4 x = pack8(MUON_F16, v);
                const uint32_t off = (pc >> 3) * PANEL + ar * 128 + (((pc & 7) ^ (ar & 7)) << 4);
                for (int i = 0; i < C; ++i) {
                    const int to = (rank + i) & (C - 1);
                    st_async_v4(mapa_shared(a0 + off, to), mapa_shared(smem_u32(&bar_a), to), x.x, x.y, x.z, x.w);
                }
            }
            fly.wait(&bar_a, phase, abort, status);
            __syncwarp();
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    v[e] = PACK && (cg >> 1) != (row >> 6) ? 0.f : __uint_as_float(r[8 * s + e]) * f.ga;
                    if (32 * cg + 8 * s + e == row) v[e] -= f.diag;
                }
                *reinterpret_cast<uint4*>(Am + pn * PANEL + row * 128 + (((ps + s) ^ (row & 7)) << 4)) = pack8(MUON_F16, v);
            }
        }
        fence_async_proxy();
        __syncthreads();
        if (tid == 0 && fly.ok) {
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const uint64_t d = smem_desc_sw128(a0 + (s >> 2) * PANEL + (s & 3) * 32, 16, 1024);
                tc_mma_bf16(tmem + ACC, d, d, idesc, s > 0);
            }
            tc_commit(&bar_square);
            if (keep) keep_square(&k.a, Am, t);
        }
        fly.wait(&bar_square, phase, abort, status);
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
        if (tid == 0 && fly.ok) {
            if (keep) keep_square(&k.b, Bm, t);
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
            fly.wait(&bar_apply[n0 >> 8], phase, abort, status);
            __syncwarp();
            tc_fence_after();
            if (keep && n0 == 0) {     // nothing is overwritten before it has been kept
                if (tid == 0) bulk_wait_read<0>();
                __syncthreads();
            }
            // This CTA's A, B~ and partial rows are done with (and, after the last iteration, its stores into its peers)
            if (n0 + 256 >= w && C > 1) cluster_arrive();
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
            if (keep && tid == 0) keep_x(t + 1);
        }
    }

    // ---------------------------------------------------------------- result
    if (!fin) {
        const float nan[16] = {NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN};
        for (int c = cg * 16; c < w; c += 64) tmem_st_x16(t_lane + c, nan);
        tmem_st_wait();
    }
    tc_fence_before();
    __syncthreads();           // every warp is past the last reads of A and B~
    tc_fence_after();
    if (tma_out) {
        const float step = it.step * k.out, decay = it.decay;
        Ring<1, PACK> ring;
        ring.a[0] = boxes_w;
        ring.n = 1;
        ring.shape(slab);
        if (update && tid == 0)
            for (int ch = 0; ch < ring.bufs; ++ch) ring.fill(slab, ch, fly);
#pragma unroll 1
        for (int ch = 0; ch < nchunk; ++ch) {
            uint8_t* buf = ring.buf(slab, ch);
            float z[16];
            tmem_ld_x16(t_lane + ch * 64 + cg * 16, z);
            if (update) {
                float x[16];
                ring.wait(slab, ch, turns, fly);
                boxes_w.get(slab, buf, row, cg, x);
#pragma unroll
                for (int h = 0; h < 16; ++h) z[h] = fmaf(step, z[h], decay * x[h]);
            } else {
                if (ch >= ring.bufs) {     // the buffer's last store has been read out
                    if (tid == 0) bulk_wait_read<0>();
                    __syncthreads();
                }
#pragma unroll
                for (int h = 0; h < 16; ++h) z[h] *= step;
            }
            boxes_w.put(slab, buf, row, cg, z);
            fence_async_proxy();
            __syncthreads();
            if (tid == 0) {
                boxes_w.store(slab, slab.first(ch), smem_u32(buf));
                bulk_commit();
                if (update) ring.refill(slab, ch, fly);
            }
        }
        if (tid == 0) bulk_wait_read<0>();
    } else {
        if (tall) slab_out_any<true, PACK>(slab, it, b, k.out);
        else slab_out_any<false, PACK>(slab, it, b, k.out);
    }
    if (C > 1) cluster_wait();     // no peer sends any more: one that has given up on its waits is as far as this
    if (tid == 0 && *abort) drain_flight(bar_fly, kRing + 2, &bar_drain, fly, status);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// ---------------------------------------------------------------- reverse pass
// D <- aD + BD + 2PX with S = sym(D X^T), P = bS + c(SA + AS), from the kept X^_t, A_t and B~_t, t falling.
// The state V = 2^k D stays in TMEM in fp32 (columns 0 ..), the products go to the columns from ACC_G on; X^_t and
// D^ = fp16(d V) lie in panels as above.  S's partial rows are exchanged as the Gram matrix's are; A and B~ come in by
// TMA over the partial rows when those have been summed, P^ takes S^'s place.  Bound by latency as the forward pass is:
// 16 blocks of 96 x 641 take 68 us, 96 of 128 x 1024 219 (as chains of tiles 154 and 499).
constexpr int ACC_G = 256;
__host__ __device__ constexpr int grad_smem_bytes(int w) { return 2 * (w / 64) * PANEL + A_BYTES + RED_BYTES + 1024; }
static_assert(grad_smem_bytes(kSmallGradSlab) + 512 <= 232448, "shared memory above the 227 KB per-CTA limit");
static_assert(2 * STG_FLOATS * 4 <= PANEL + A_BYTES + RED_BYTES, "two staging buffers fit beside the X panels");
static_assert(2 * A_BYTES <= RED_BYTES, "A and B~ over the partial rows");

template <int N>
struct SmallGradParams {
    SmallStackItem item[N];
    SmallGradClass k;
    int n;
};
static_assert(sizeof(SmallGradParams<kFewItems>) <= 4096, "the small form's parameters launch faster");

template <int N, bool PACK>
__global__ void __launch_bounds__(THREADS, 1) stack_small_grad_kernel(const __grid_constant__ SmallGradParams<N> p) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    __shared__ uint64_t bar_fly[kRing + 4], bar_s, bar_p, bar_apply, bar_drain;
    __shared__ uint32_t tmem_slot;
    __shared__ int abort_flag;
    __shared__ double red_sum[THREADS / 32];
    __shared__ double parts[PACK ? 2 : 1][16];

    constexpr int kRows = kRing, kAll = kRing + 1, kAB = kRing + 2, kX = kRing + 3;   // places in bar_fly, after the ring
    uint64_t &bar_rows = bar_fly[kRows], &bar_all = bar_fly[kAll], &bar_ab = bar_fly[kAB], &bar_x = bar_fly[kX];
    Flight fly;
    const SmallGradClass& k = p.k;
    const int C = k.cluster, w = k.slab, nchunk = w >> 6;
    uint8_t* Xp = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* Dp = Xp + nchunk * PANEL;
    uint8_t* Sm = Dp + nchunk * PANEL;             // S^, then P^
    uint8_t* red = Sm + A_BYTES;                   // partial rows, then A and B~
    uint8_t* Am = red;
    uint8_t* Bm = red + A_BYTES;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = static_cast<int>(cluster_ctarank());
    const int blk = static_cast<int>(blockIdx.x) / C;
    int lo = 0, hi = p.n - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.item[mid].block0 <= blk) lo = mid; else hi = mid - 1;
    }
    const SmallStackItem& it = p.item[lo];
    const long long b = (PACK ? 2 : 1) * static_cast<long long>(blk - it.block0);
    const int kept = it.at + static_cast<int>(b);
    const int q = warp & 3, cg = warp >> 2, row = 32 * q + lane;
    const int half = PACK ? q >> 1 : 0;            // this thread's block of the two
    const bool tall = k.rows > k.cols, two = PACK && b + 1 < it.count;

    if (tid == 0) {
        for (uint64_t* x : {&bar_s, &bar_p, &bar_apply, &bar_drain}) mbar_init(x, 1);
        for (uint64_t& x : bar_fly) mbar_init(&x, 1);
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
    const Slab slab = {k.rows, k.cols, rank, C, nchunk, tall, two, Dp, nchunk * PANEL + A_BYTES + RED_BYTES, t_lane, bar_fly, abort, status};
    const bool tma_in = (it.vec & 1) != 0, tma_out = (it.vec & 4) != 0;

    auto load_x = [&](int t) {     // thread 0
        if (!fly.ok) return;
        const int ys = PACK && !two ? 64 : 128;
        fly.arm(kX);
        mbar_arrive_expect_tx(&bar_x, static_cast<uint32_t>(nchunk * ys * 128));
        for (int j = 0; j < nchunk; ++j)
            for (int y = 0; y < ys; y += 64)
                tma_load_3d(smem_u32(Xp) + j * PANEL + y * 128, &k.x, smem_u32(&bar_x), slab.first(j), PACK ? 0 : y,
                            t * k.saved + kept + (PACK ? y >> 6 : 0));
    };
    auto load_ab = [&](int t) {    // thread 0
        if (!fly.ok) return;
        fly.arm(kAB);
        mbar_arrive_expect_tx(&bar_ab, 2 * A_BYTES);
        for (int x = 0; x < 128; x += 64)
            for (int y = 0; y < 128; y += 64) {
                // packed: the blocks' matrices on the diagonal, zeros (from beyond the matrix) beside them and where
                // there is no second block
                const uint32_t at = (x >> 6) * PANEL + y * 128;
                const bool zeros = PACK && (x != y || (x > 0 && !two));
                const int mx = PACK ? zeros ? 64 : 0 : x, my = PACK ? 0 : y;
                const int z = t * k.saved + kept + (PACK && x > 0 && y > 0 && two ? 1 : 0);
                tma_load_3d(smem_u32(Am) + at, &k.a, smem_u32(&bar_ab), mx, my, z);
                tma_load_3d(smem_u32(Bm) + at, &k.b, smem_u32(&bar_ab), mx, my, z);
            }
    };
    // The cluster's sums of the two blocks (packed: by rows), in rank order, in every thread of every CTA.
    double sums[2] = {0.0, 0.0};
    auto cluster_sum = [&](double v) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (lane == 0) red_sum[warp] = v;
        __syncthreads();
        cluster_arrive();      // every CTA of the cluster runs, and is past its last read of `parts`
        cluster_wait();
        if (tid < (PACK ? 2 * C : C)) {
            const int to = tid & (C - 1), of = tid / C;
            double s = 0.0;
            for (int i = 0; i < THREADS / 32; ++i)
                if (!PACK || ((i & 3) >> 1) == of) s += red_sum[i];
            st_cluster_f64(mapa_shared(smem_u32(&parts[of][rank]), to), s);
        }
        cluster_arrive();
        cluster_wait();
#pragma unroll
        for (int of = 0; of < (PACK ? 2 : 1); ++of) {
            sums[of] = 0.0;
            for (int i = 0; i < C; ++i) sums[of] += parts[of][i];
        }
        return PACK && half ? sums[1] : sums[0];
    };

    // ---------------------------------------------------------------- gradient of the output -> TMEM, its norm
    if (PACK && !two)      // X^ of a block that is not there
        for (int i = tid; i < nchunk * 512; i += THREADS)
            *reinterpret_cast<uint4*>(Xp + (i >> 9) * PANEL + 64 * 128 + (i & 511) * 16) = make_uint4(0, 0, 0, 0);
    if (tid == 0) load_x(k.iters - 1);
    uint32_t turns = 0;
    double ss = 0.0;
    if (tma_in) {
        Ring<1, PACK> ring;
        ring.a[0] = {&it.map_g, it.g_dtype, it.g_dtype == MUON_F32 ? 4 : 2, static_cast<int>(b)};
        ring.n = 1;
        ring.shape(slab);
        if (tid == 0)
            for (int ch = 0; ch < ring.bufs; ++ch) ring.fill(slab, ch, fly);
#pragma unroll 1
        for (int ch = 0; ch < nchunk; ++ch) {
            ring.wait(slab, ch, turns, fly);
            float u[16];
            ring.a[0].get(slab, ring.buf(slab, ch), row, cg, u);
            ss += static_cast<double>(sum_squares(u));
            tmem_st_x16(t_lane + ch * 64 + cg * 16, u);
            __syncthreads();
            if (tid == 0) ring.refill(slab, ch, fly);
        }
    } else {
        const Momentum mo = {1.f, 0.f, false, false};
        ss = tall ? slab_in_any<true, PACK>(slab, it, b, mo) : slab_in_any<false, PACK>(slab, it, b, mo);
        if (PACK) {            // a thread of that walk has elements of both blocks
            tmem_st_wait();
            ss = 0.0;
            for (int c = cg * 16; c < w; c += 64) {
                float z[16];
                tmem_ld_x16(t_lane + c, z);
                ss += static_cast<double>(sum_squares(z));
            }
        }
    }
    tmem_st_wait();
    double sum = cluster_sum(ss);
    if (!(sums[0] > 1e-25 && sums[0] < 1e36 && (!two || (sums[1] > 1e-25 && sums[1] < 1e36)))) {     // squares outside fp32's range: once more in fp64 (all CTAs alike)
        ss = 0.0;
        for (int c = cg * 16; c < w; c += 64) {
            float z[16];
            tmem_ld_x16(t_lane + c, z);
#pragma unroll
            for (int h = 0; h < 16; ++h) ss = fma(static_cast<double>(z[h]), static_cast<double>(z[h]), ss);
        }
        sum = cluster_sum(ss);
    }
    const double norm = sqrt(sum);
    if (lane == 0 && (warp == 0 || (PACK && warp == 2)) && rank == 0 && !isfinite(norm)) atomicOr(status, kDevErrNonfinite);
    // The factors f0 of the blocks.  One that is not finite, or whose gradient is not, goes on with zeros, so that
    // nothing of it gets into another, and ends as NaN.
    float f0s[2] = {k.info[static_cast<size_t>(kept) * kStackInfo], 0.f};
    if (two) f0s[1] = k.info[static_cast<size_t>(kept + 1) * kStackInfo];
    const float* info = k.info + static_cast<size_t>(kept + (half && two ? 1 : 0)) * kStackInfo;
    const bool fin = isfinite(norm) && isfinite(half ? f0s[1] : f0s[0]);
#pragma unroll
    for (float& f : f0s)
        if (!isfinite(f)) f = 0.f;
    const float f0 = half ? f0s[1] : f0s[0];
    int ex = 0;
    if (fin && norm > 0.0) ex = max(-126, min(126, -(ilogb(norm) + 1)));
    const float up = __int_as_float((ex + 127) << 23);
    {
        const float d = k.it[k.iters - 1].d;
        for (int c = cg * 16; c < w; c += 64) {
            float z[16];
            tmem_ld_x16(t_lane + c, z);
#pragma unroll
            for (int h = 0; h < 16; ++h) z[h] = fin ? z[h] * up : 0.f;
            tmem_st_x16(t_lane + c, z);
            put_panel16(Dp, row, c, z, d);
        }
        tmem_st_wait();
    }
    fence_async_proxy();
    tc_fence_before();
    __syncthreads();
    if (C > 1) cluster_arrive();      // staging is over: peers may write into this CTA's buffers

    // ---------------------------------------------------------------- iterations
    const int rc = 128 / C;                        // rows of S that a CTA owns
    const int own = row / rc, orow = row - own * rc, rmask = min(rc, 8) - 1;
    const uint32_t idesc = idesc_f16_f32(128, 128, 0, 0);
    const uint32_t x0 = smem_u32(Xp), d0 = smem_u32(Dp), s0 = smem_u32(Sm), a0 = smem_u32(Am), b0 = smem_u32(Bm);
    const int pn = cg >> 1, ps = (cg & 1) * 4;     // panel and first 16-byte piece of columns 32 cg ...
    for (int i = 0; i < k.iters; ++i) {
        const int t = k.iters - 1 - i;
        const SmallGradIter& f = k.it[t];
        const uint32_t phase = i & 1;
        const float f0t = t == 0 ? f0 : 1.f;       // X_0 = f0 X^_0
        if (tid == 0 && fly.ok) {
            if (C > 1) {
                fly.arm(kRows);
                fly.arm(kAll);
                mbar_arrive_expect_tx(&bar_rows, RED_BYTES);
                mbar_arrive_expect_tx(&bar_all, A_BYTES);
            } else {
                load_ab(t);
            }
            fly.wait(&bar_x, phase, abort, status);
            tc_fence_after();
            fence_async_proxy();
            for (int j = 0; j < nchunk; ++j)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const uint64_t dd = smem_desc_sw128(d0 + j * PANEL + s * 32, 16, 1024);
                    const uint64_t xd = smem_desc_sw128(x0 + j * PANEL + s * 32, 16, 1024);
                    tc_mma_bf16(tmem + ACC_G, dd, xd, idesc, j + s > 0);   // kind::f16, types from idesc
                    tc_mma_bf16(tmem + ACC_G, xd, dd, idesc, 1);
                }
            tc_commit(&bar_s);
        }
        fly.wait(&bar_s, phase, abort, status);
        __syncwarp();
        tc_fence_after();
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_lane + ACC_G + 32 * cg, r);
        tmem_ld_wait();
        tc_fence_before();
        if (C > 1) {
            // as the Gram matrix's rows
            cluster_wait();        // every CTA's buffers are free
            const uint32_t dst = mapa_shared(smem_u32(red), own) + static_cast<uint32_t>(rank * rc * 512);
            const uint32_t bar = mapa_shared(smem_u32(&bar_rows), own);
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const int seg = 8 * cg + s;
                st_async_v4(dst + ((seg * rc + (orow ^ (seg & rmask))) << 4), bar, r[4 * s], r[4 * s + 1], r[4 * s + 2], r[4 * s + 3]);
            }
            fly.wait(&bar_rows, phase, abort, status);
            __syncwarp();
            for (int g = tid; g < rc * 16; g += THREADS) {
                const int rr = g >> 4, pc = g & 15, ar = rank * rc + rr;
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int seg = 2 * pc + h;
                    const uint8_t* src = red + ((seg * rc + (rr ^ (seg & rmask))) << 4);
                    for (int j = 0; j < C; ++j) {
                        const float4 x = *reinterpret_cast<const float4*>(src + j * rc * 512);
                        v[4 * h] += x.x; v[4 * h + 1] += x.y; v[4 * h + 2] += x.z; v[4 * h + 3] += x.w;
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = PACK && (pc >> 3) != (ar >> 6) ? 0.f : v[e] * f.s * (t == 0 ? f0s[PACK ? ar >> 6 : 0] : 1.f);
                const uint4 x = pack8(MUON_F16, v);
                const uint32_t off = (pc >> 3) * PANEL + ar * 128 + (((pc & 7) ^ (ar & 7)) << 4);
                for (int j = 0; j < C; ++j) {
                    const int to = (rank + j) & (C - 1);
                    st_async_v4(mapa_shared(s0 + off, to), mapa_shared(smem_u32(&bar_all), to), x.x, x.y, x.z, x.w);
                }
            }
            __syncthreads();       // the partial rows have been read
            if (tid == 0) {
                fence_async_proxy();
                load_ab(t);
            }
            fly.wait(&bar_all, phase, abort, status);
            __syncwarp();
        } else {
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = PACK && (cg >> 1) != (row >> 6) ? 0.f : __uint_as_float(r[8 * s + e]) * f.s * f0t;
                *reinterpret_cast<uint4*>(Sm + pn * PANEL + row * 128 + (((ps + s) ^ (row & 7)) << 4)) = pack8(MUON_F16, v);
            }
        }
        fence_async_proxy();
        __syncthreads();
        if (tid == 0 && fly.ok) {
            fly.wait(&bar_ab, phase, abort, status);
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                const uint32_t o = (s >> 2) * PANEL + (s & 3) * 32;
                const uint64_t sd = smem_desc_sw128(s0 + o, 16, 1024), ad = smem_desc_sw128(a0 + o, 16, 1024);
                tc_mma_bf16(tmem + ACC_G + 128, sd, ad, idesc, s > 0);
                tc_mma_bf16(tmem + ACC_G + 128, ad, sd, idesc, 1);
            }
            tc_commit(&bar_p);
        }
        fly.wait(&bar_p, phase, abort, status);
        __syncwarp();
        tc_fence_after();
        tmem_ld_32x32b_x32(t_lane + ACC_G + 128 + 32 * cg, r);
        tmem_ld_wait();
        const float pa = f.pa * f0t, pb = f.pb * f0t;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            uint4* at = reinterpret_cast<uint4*>(Sm + pn * PANEL + row * 128 + (((ps + s) ^ (row & 7)) << 4));
            float v[8];
            unpack8(*at, MUON_F16, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = fmaf(pb, v[e], pa * __uint_as_float(r[8 * s + e]));
            *at = pack8(MUON_F16, v);
        }
        fence_async_proxy();
        tc_fence_before();
        __syncthreads();
        if (tid == 0 && fly.ok) {
            tc_fence_after();
            const uint32_t id = idesc_f16_f32(128, w, 0, 1);
            for (int g = 0; g < 2; ++g)
#pragma unroll
                for (int s = 0; s < 8; ++s) {
                    const uint64_t ad = smem_desc_sw128((g ? s0 : b0) + (s >> 2) * PANEL + (s & 3) * 32, 16, 1024);
                    const uint64_t xd = smem_desc_sw128((g ? x0 : d0) + s * 2048, PANEL, 1024);
                    tc_mma_bf16(tmem + ACC_G, ad, xd, id, g + s > 0);
                }
            tc_commit(&bar_apply);
        }
        fly.wait(&bar_apply, phase, abort, status);
        __syncwarp();
        tc_fence_after();
        const bool last = t == 0;
        if (!last) {
            if (tid == 0) load_x(t - 1);
            if (C > 1) cluster_arrive();           // this CTA's partial rows, A, B~ and P^ are done with
        }
        const float d = last ? 0.f : k.it[t - 1].d;
        for (int c = cg * 16; c < w; c += 64) {
            float z[16], u[16];
            tmem_ld_x16(t_lane + c, z);
            tmem_ld_x16(t_lane + ACC_G + c, u);
#pragma unroll
            for (int h = 0; h < 16; ++h) z[h] = fmaf(f.va, z[h], f.vb * u[h]);
            tmem_st_x16(t_lane + c, z);
            if (!last) put_panel16(Dp, row, c, z, d);
        }
        tmem_st_wait();
        fence_async_proxy();
        tc_fence_before();
        __syncthreads();
    }

    // ---------------------------------------------------------------- gradient of the input
    // dU = [D - X_0 <D, X_0> (N + eps) / N] / (N + eps), D = V / 2^k, X_0 = f0 X^_0 (whose panels are still here)
    fly.wait(&bar_x, (k.iters - 1) & 1, abort, status);
    __syncwarp();
    auto x_at = [&](int c, float (&x)[16]) {
        const uint8_t* src = Xp + (c >> 6) * PANEL + row * 128;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8];
            unpack8(*reinterpret_cast<const uint4*>(src + (((((c & 63) >> 3) + h) ^ (row & 7)) << 4)), MUON_F16, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[8 * h + e] = v[e];
        }
    };
    double dot = 0.0;
    for (int c = cg * 16; c < w; c += 64) {
        float z[16], x[16];
        tmem_ld_x16(t_lane + c, z);
        x_at(c, x);
        float s = 0.f;
#pragma unroll
        for (int h = 0; h < 16; ++h) s = fmaf(z[h], x[h], s);     // 16 products in fp32, their sums in fp64
        dot += static_cast<double>(s);
    }
    dot = cluster_sum(dot);
    const double n = info[3], eps = static_cast<double>(k.eps), sd = 1.0 / static_cast<double>(up);
    const double corr = n > 0.0 ? dot * sd * f0 * (n + eps) / n : 0.0;
    const float od = fin ? static_cast<float>(sd / (n + eps)) : NAN, ox = static_cast<float>(-corr * f0 / (n + eps));
    for (int c = cg * 16; c < w; c += 64) {
        float z[16], x[16];
        tmem_ld_x16(t_lane + c, z);
        x_at(c, x);
#pragma unroll
        for (int h = 0; h < 16; ++h) z[h] = fmaf(od, z[h], ox * x[h]);
        tmem_st_x16(t_lane + c, z);
    }
    tmem_st_wait();
    __syncthreads();
    if (tma_out) {
        const Boxes<PACK> boxes = {&it.map_w, it.w_dtype, it.w_dtype == MUON_F32 ? 4 : 2, static_cast<int>(b)};
        const int size = boxes.bytes(), bufs = min(nchunk, slab.bytes / size);
#pragma unroll 1
        for (int ch = 0; ch < nchunk; ++ch) {
            uint8_t* buf = slab.buf + (ch % bufs) * size;
            if (ch >= bufs) {          // the buffer's last store has been read out
                if (tid == 0) bulk_wait_read<0>();
                __syncthreads();
            }
            float z[16];
            tmem_ld_x16(t_lane + ch * 64 + cg * 16, z);
            boxes.put(slab, buf, row, cg, z);
            fence_async_proxy();
            __syncthreads();
            if (tid == 0) {
                boxes.store(slab, slab.first(ch), smem_u32(buf));
                bulk_commit();
            }
        }
        if (tid == 0) bulk_wait_read<0>();
    } else {
        if (tall) slab_out_any<true, PACK>(slab, it, b, 1.f);
        else slab_out_any<false, PACK>(slab, it, b, 1.f);
    }
    // Peers' last stores into this CTA lie before the cluster barriers of the last sum, which also a CTA that has given
    // up on its waits meets.
    if (tid == 0 && *abort) drain_flight(bar_fly, kRing + 4, &bar_drain, fly, status);
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <class P, class K, int N, int PER>     // PER: blocks to a cluster
cudaError_t launch(void (*kernel)(P), int most_smem, int smem, const SmallStackItem* items, int n, const K& k, cudaStream_t stream) {
    constexpr int kMaxDevices = 64;
    static std::atomic<bool> ready[kMaxDevices];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (!ready[dev].load()) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most_smem);
        if (e != cudaSuccess) return e;
        ready[dev].store(true);
    }
    for (int i0 = 0; i0 < n; i0 += N) {
        P p;
        p.n = n - i0 < N ? n - i0 : N;
        p.k = k;
        int blocks = 0;
        for (int i = 0; i < p.n; ++i) {
            p.item[i] = items[i0 + i];
            p.item[i].block0 = blocks;
            blocks += (items[i0 + i].count + PER - 1) / PER;
        }
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(k.cluster) * blocks, 1, 1);
        cfg.blockDim = dim3(THREADS, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = k.cluster;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, kernel, p);
        if (e == cudaSuccess) e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <int N, bool PACK>
cudaError_t run_step(const SmallStackItem* items, int n, const SmallStackClass& k, cudaStream_t stream) {
    return launch<SmallParams<N>, SmallStackClass, N, PACK ? 2 : 1>(stack_small_kernel<N, PACK>, smem_bytes(kSmallStackSlab),
                                                                    smem_bytes(k.slab), items, n, k, stream);
}
template <int N, bool PACK>
cudaError_t run_grad(const SmallStackItem* items, int n, const SmallGradClass& k, cudaStream_t stream) {
    return launch<SmallGradParams<N>, SmallGradClass, N, PACK ? 2 : 1>(stack_small_grad_kernel<N, PACK>,
                                                                       grad_smem_bytes(kSmallGradSlab), grad_smem_bytes(k.slab),
                                                                       items, n, k, stream);
}

}  // namespace

int stack_small_resident(int cluster) {
    constexpr int kMaxDevices = 64;
    static std::atomic<int> of[kMaxDevices][4];
    const int k = cluster >= 8 ? 3 : cluster >= 4 ? 2 : cluster >= 2 ? 1 : 0;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return 112 / cluster;
    }
    int n = of[dev][k].load();
    if (n == 0) {
        const auto kernel = stack_small_kernel<kFewItems, false>;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(cluster) * 148, 1, 1);
        cfg.blockDim = dim3(THREADS, 1, 1);
        cfg.dynamicSmemBytes = smem_bytes(kSmallStackSlab);
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = cluster;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(kSmallStackSlab)) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n <= 0) {
            cudaGetLastError();
            n = 112 / cluster;
        }
        of[dev][k].store(n);
    }
    return n;
}

cudaError_t stack_small_launch(const SmallStackItem* items, int n, const SmallStackClass& k, cudaStream_t stream) {
    if (k.pack)
        return n <= kFewItems ? run_step<kFewItems, true>(items, n, k, stream) : run_step<kSmallStackItems, true>(items, n, k, stream);
    return n <= kFewItems ? run_step<kFewItems, false>(items, n, k, stream) : run_step<kSmallStackItems, false>(items, n, k, stream);
}

cudaError_t stack_small_grad_launch(const SmallStackItem* items, int n, const SmallGradClass& k, cudaStream_t stream) {
    if (k.pack)
        return n <= kFewItems ? run_grad<kFewItems, true>(items, n, k, stream) : run_grad<kSmallStackItems, true>(items, n, k, stream);
    return n <= kFewItems ? run_grad<kFewItems, false>(items, n, k, stream) : run_grad<kSmallStackItems, false>(items, n, k, stream);
}

}  // namespace muon
