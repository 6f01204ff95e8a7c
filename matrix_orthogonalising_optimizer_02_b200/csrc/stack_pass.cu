// Elementwise passes over stacks of blocks: what comes before and after the products of
// stack_chain.cu.  HBM-bound; one CTA takes 2048 elements of one block, 8 a thread, or four times as many.
//
// Norms.  A block's sum of squares is formed in fp64 (a gradient's elements, 1e-20 or 1e20, square
// out of fp32's range), one partial per CTA; the next pass's CTAs each add up their block's partials
// in one fixed order, so no launch is spent on it and every CTA gets the same number.
//
// Measured over 38e6 elements (a training step's matrices): norm and momentum 58 us (10 bytes an element, 1.0 of
// the measured copy rate), scaled planes 63 us (10, 0.93), update 39 us (6, 0.90).
//
// Scaling.  hi = fp16(U * 2^k) with the power of two that puts the block's rms into [1/2, 1): no
// element of up to 2^31 can leave fp16's range, a 16-bit input of ordinary spread is held exactly,
// and 1 / (N + eps) enters in the first products' epilogues as f0 = 1 / ((N + eps) 2^k).
#include <cmath>

#include "../../include/muon_b200.h"
#include "stacks.cuh"
#include "typed_io.cuh"

namespace muon {
namespace {

template <int N>
struct PassParams {
    StackItem item[N];
    StackPassArgs a;
    int n;
};

constexpr int kFewItems = 21;

__device__ __forceinline__ float pow2f(int k) {   // 2^k, |k| <= 126
    return __int_as_float((k + 127) << 23);
}

// Eight elements of a thread: side by side (VEC), or, for arrays that 16-byte accesses cannot reach, a warp's
// width apart, so that the warp's accesses lie side by side (8 single accesses of neighbours took 42 us to write
// 24 blocks of 509 x 1021 in bf16).
template <bool VEC>
struct Eight {
    int i[VEC ? 1 : 8], j[VEC ? 1 : 8];   // rows and columns in the block
    int n;                                // VEC: how many of the eight lie inside
    unsigned in;                          // otherwise: a bit for each that does
    unsigned padded;                      // and for each that lies in the padded block
    size_t plane;                         // the first one's place in the workspace planes

    __device__ __forceinline__ Eight(const StackItem& it, size_t plane0, int c, int q) {   // q: the thread's group
        const int rp = (it.rows + 7) & ~7, cp = (it.cols + 7) & ~7;
        if constexpr (VEC) {
            const int g = (c * it.per + q) * kStackThreads + static_cast<int>(threadIdx.x), cg = cp >> 3;
            i[0] = g / cg;
            j[0] = (g - i[0] * cg) * 8;
            n = i[0] < it.rows ? min(8, it.cols - j[0]) : 0;
            padded = i[0] < rp;
            plane = plane0 + static_cast<size_t>(g) * 8;
        } else {
            const int f0 = (c * it.per + q) * kStackGroup + static_cast<int>(threadIdx.x >> 5) * 256 + (threadIdx.x & 31);
            i[0] = f0 / cp;
            j[0] = f0 - i[0] * cp;
            in = padded = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (e > 0) {
                    i[e] = i[e - 1];
                    j[e] = j[e - 1] + 32;
                    if (cp >= 32) {
                        if (j[e] >= cp) { ++i[e]; j[e] -= cp; }
                    } else {
                        while (j[e] >= cp) { ++i[e]; j[e] -= cp; }
                    }
                }
                in |= (i[e] < it.rows && j[e] < it.cols) << e;
                padded |= (i[e] < rp) << e;
            }
            plane = plane0 + f0;
        }
    }
    // Where all eight are there for 16-byte accesses, fetch() only starts the loads and take() waits for them, so that
    // several groups' are under way together; otherwise take() does it all.
    struct Raw { uint4 a, b; };
    __device__ __forceinline__ bool whole() const { return VEC && n == 8; }
    __device__ __forceinline__ void fetch(const void* p, int dtype, long long base, int ld, Raw& r) const {
        if (!whole()) return;
        const size_t e = base + static_cast<long long>(i[0]) * ld + j[0];
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p) + e * (dtype == MUON_F32 ? 4 : 2));
        r.a = q[0];
        if (dtype == MUON_F32) r.b = q[1];
    }
    __device__ __forceinline__ void take(const Raw& r, const void* p, int dtype, long long base, int ld, float (&x)[8]) const {
        if (!whole()) return get(p, dtype, base, ld, x);
        if (dtype == MUON_F32) {
            const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(w[e]);
        } else {
            unpack8(r.a, dtype, x);
        }
    }
    __device__ __forceinline__ void fetch_plane(const __half* p, Raw& r) const {
        if (VEC) r.a = *reinterpret_cast<const uint4*>(p + plane);
    }
    __device__ __forceinline__ void take_plane(const Raw& r, const __half* p, float (&x)[8]) const {
        if (VEC) unpack8(r.a, MUON_F16, x);
        else get_plane(p, x);
    }
    __device__ __forceinline__ bool any() const {
        if constexpr (VEC) return n > 0;
        else return in != 0;
    }
    __device__ __forceinline__ void get(const void* p, int dtype, long long base, int ld, float (&x)[8]) const {
        if constexpr (VEC) {
            load8(p, dtype, base + static_cast<long long>(i[0]) * ld + j[0], n, true, x);
        } else {
            by_type(dtype, [&](auto t) {
                using E = decltype(t);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    x[e] = in >> e & 1 ? widen(static_cast<const E*>(p)[base + static_cast<long long>(i[e]) * ld + j[e]]) : 0.f;
            });
        }
    }
    __device__ __forceinline__ void put(void* p, int dtype, long long base, int ld, const float (&x)[8]) const {
        if constexpr (VEC) {
            store8(p, dtype, base + static_cast<long long>(i[0]) * ld + j[0], n, true, x);
        } else {
            by_type(dtype, [&](auto t) {
                using E = decltype(t);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (in >> e & 1) narrow(static_cast<E*>(p)[base + static_cast<long long>(i[e]) * ld + j[e]], x[e]);
            });
        }
    }
    __device__ __forceinline__ void get_plane(const __half* p, float (&x)[8]) const {
        if constexpr (VEC) {
            unpack8(*reinterpret_cast<const uint4*>(p + plane), MUON_F16, x);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = in >> e & 1 ? __half2float(p[plane + 32 * e]) : 0.f;
        }
    }
    // Stores x and leaves in it what fp16 has lost.
    __device__ __forceinline__ void put_plane(__half* p, float (&x)[8]) const {
        if constexpr (VEC) {
            const uint4 h = pack8(MUON_F16, x);
            *reinterpret_cast<uint4*>(p + plane) = h;
            float y[8];
            unpack8(h, MUON_F16, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] -= y[e];
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const __half h = __float2half_rn(x[e]);
                if (padded >> e & 1) p[plane + 32 * e] = h;
                x[e] -= __half2float(h);
            }
        }
    }
};

// A CTA's chunk c of block b; returns the thread's part of the sum that kNorm and kDot form.
template <StackPass PASS, bool VEC>
__device__ __forceinline__ double walk(const StackItem& it, const StackPassArgs& a, int b, int c, float gs, float up, float od,
                                       float ox) {
    const int rp = (it.rows + 7) & ~7, cp = (it.cols + 7) & ~7;
    const size_t plane0 = static_cast<size_t>(b) * rp * cp;
    const long long gb = b * it.g_stride, mb = b * it.m_stride, wb = b * it.w_stride;
    double ss = 0.0;
    constexpr int U = VEC ? 2 : 1;     // groups whose loads are under way together
    using At = Eight<VEC>;
    constexpr bool norm = PASS == StackPass::kNorm, pack = PASS == StackPass::kPack || PASS == StackPass::kPackGrad;
    // The momentum pass has updated M when the planes are made.
    const bool from_g = norm || it.M == nullptr || a.nesterov, from_m = it.M != nullptr;
    for (int q0 = 0; q0 < it.per; q0 += U) {
        const At at[2] = {At(it, plane0, c, q0), At(it, plane0, c, q0 + U - 1)};
        typename At::Raw r0[U], r1[U], r2[U];
        bool on[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            on[u] = q0 + u < it.per && at[u].any();
            if (!on[u]) continue;
            if (norm || pack) {
                if (from_g) at[u].fetch(it.G, it.g_dtype, gb, it.g_ld, r0[u]);
                if (from_m) at[u].fetch(it.M, MUON_F32, mb, it.m_ld, r1[u]);
            } else {
                at[u].fetch_plane(it.hi, r0[u]);
                if (PASS == StackPass::kUpdate) at[u].fetch(it.W, it.w_dtype, wb, it.w_ld, r1[u]);
                if (PASS == StackPass::kDot || PASS == StackPass::kGradOut) {
                    at[u].fetch_plane(it.lo, r1[u]);
                    at[u].fetch_plane(it.hi2, r2[u]);
                }
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (norm || pack) {
                if (!on[u] && (norm || q0 + u >= it.per || !at[u].padded)) continue;   // padding is written too
                float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (on[u]) {
                    if (from_g) {
                        at[u].take(r0[u], it.G, it.g_dtype, gb, it.g_ld, x);
#pragma unroll
                        for (int e = 0; e < 8; ++e) x[e] *= gs;
                    }
                    if (from_m) {
                        float m[8];
                        at[u].take(r1[u], it.M, MUON_F32, mb, it.m_ld, m);
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            if (norm) m[e] = fmaf(a.beta, m[e], x[e]);
                            x[e] = a.nesterov ? fmaf(a.beta, m[e], x[e]) : m[e];
                        }
                        if (norm) at[u].put(it.M, MUON_F32, mb, it.m_ld, m);
                    }
                }
                if (norm) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fma(static_cast<double>(x[e]), static_cast<double>(x[e]), ss);
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        x[e] *= up;
                        if (PASS == StackPass::kPackGrad) x[e] *= it.step;     // apart: their product may leave fp32's range
                    }
                    at[u].put_plane(it.hi, x);
                    at[u].put_plane(it.lo, x);
                }
                continue;
            }
            if (!on[u]) continue;
            float x[8];
            at[u].take_plane(r0[u], it.hi, x);
            if (PASS == StackPass::kOut) {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] *= it.step;
                at[u].put(it.W, it.w_dtype, wb, it.w_ld, x);
            } else if (PASS == StackPass::kUpdate) {
                float w[8];
                at[u].take(r1[u], it.W, it.w_dtype, wb, it.w_ld, w);
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = fmaf(it.step, x[e], it.decay * w[e]);
                at[u].put(it.W, it.w_dtype, wb, it.w_ld, w);
            } else {
                float y[8], z[8];
                at[u].take_plane(r1[u], it.lo, y);
                at[u].take_plane(r2[u], it.hi2, z);
                if (PASS == StackPass::kDot) {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        ss = fma(static_cast<double>(x[e]) + static_cast<double>(y[e]), static_cast<double>(z[e]), ss);
                } else {
                    // X_0 as its first plane: the radial term is at most as long as the whole, so 2^-11 of it is
                    // less than the products have left
#pragma unroll
                    for (int e = 0; e < 8; ++e) x[e] = fmaf(od, (x[e] + y[e]) * up, ox * z[e]);
                    at[u].put(it.W, it.w_dtype, wb, it.w_ld, x);
                }
            }
        }
    }
    return ss;
}

template <StackPass PASS, int N>
__global__ void __launch_bounds__(kStackThreads, 4)
stack_pass_kernel(const __grid_constant__ PassParams<N> p) {
    int lo = 0, hi = p.n - 1;
    const int chunk = static_cast<int>(blockIdx.x);
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.item[mid].chunk0 <= chunk) lo = mid; else hi = mid - 1;
    }
    const StackItem& it = p.item[lo];
    const int b = (chunk - it.chunk0) / it.chunks, c = (chunk - it.chunk0) - b * it.chunks;
    const float gs = p.a.gscale != nullptr ? __ldg(p.a.gscale) : 1.f;
    float* info = it.info != nullptr ? it.info + static_cast<size_t>(b) * kStackInfo : nullptr;
    double* partials = it.partials != nullptr ? it.partials + static_cast<size_t>(b) * it.chunks : nullptr;

    float up = 1.f;                            // kPack, kPackGrad: factor of the plane; kGradOut: 2^-e
    float od = 0.f, ox = 0.f;                  // kGradOut: out = od * up * D + ox * X
    if (PASS == StackPass::kPack || PASS == StackPass::kPackGrad || PASS == StackPass::kGradOut) {
        double s = 0.0;
        for (int i = threadIdx.x; i < it.chunks; i += kStackThreads) s += partials[i];
        s = block_sum256(s);
        const double eps = static_cast<double>(p.a.eps);
        if (PASS == StackPass::kGradOut) {
            // dU = [D_0 - X_0 <D_0, X_0> (N + eps) / N] / (N + eps), D_0 = (hi + lo) / 2^(k + e)
            const float* gi = it.ginfo + static_cast<size_t>(b) * kStackInfo;
            const double n = info[3], f0 = info[0];
            const int e = it.scale[static_cast<size_t>(b) * (p.a.iters + 1)].e, near = max(-100, min(100, e));
            up = pow2f(-near);                   // apart: with 2^-k it would leave fp32's normal range for tiny gradients
            const double sd = ldexp(1.0 / gi[1], near - e);
            const double corr = n > 0.0 ? s * up * sd * f0 * (n + eps) / n : (isnan(f0) ? f0 : 0.0);
            od = static_cast<float>(sd / (n + eps));
            ox = static_cast<float>(-corr * f0 / (n + eps));
        } else {
            const double n = sqrt(s);
            // hi's rms (kPack) or whole norm (kPackGrad) in [1/2, 1)
            const double size = PASS == StackPass::kPack ? n / sqrt(static_cast<double>(it.rows) * it.cols) : n;
            int k = 0;
            if (isfinite(n) && n > 0.0) k = max(-126, min(126, -(ilogb(size) + 1)));
            up = pow2f(k);
            if (c == 0 && threadIdx.x == 0) {
                const bool fin = isfinite(n);
                info[0] = !fin ? NAN : n > 0.0 ? static_cast<float>(1.0 / ((n + eps) * static_cast<double>(up))) : 0.f;
                info[1] = up;
                info[2] = static_cast<float>(1.0 / (n + eps));
                info[3] = static_cast<float>(n);
                if (!fin && p.a.status != nullptr) atomicOr(p.a.status, kDevErrNonfinite);
            }
            if (c == 0 && threadIdx.x == 1) it.done[b] = 0;
            if (PASS == StackPass::kPackGrad && c == 0 && static_cast<int>(threadIdx.x) <= p.a.iters) {
                // the planes' norm is step at most
                const bool last = static_cast<int>(threadIdx.x) == p.a.iters;
                it.scale[static_cast<size_t>(b) * (p.a.iters + 1) + threadIdx.x] = {
                    last ? static_cast<unsigned long long>(static_cast<double>(it.step) * it.step * 1073741824.0) : 0ull,
                    last ? ilogbf(it.step) : 0, 0};
            }
            if (blockIdx.x == 0 && threadIdx.x < kStackTickets) p.a.tickets[threadIdx.x] = 0;
        }
    }

    if (PASS == StackPass::kNorm && p.a.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *p.a.status = 0;

    constexpr int need = PASS == StackPass::kDot ? 0 : PASS == StackPass::kNorm || PASS == StackPass::kPack ? 3 : PASS == StackPass::kPackGrad ? 1 : 4;
    const int have = it.vec | (it.M == nullptr ? 2 : 0);
    const double ss = (have & need) == need ? walk<PASS, true>(it, p.a, b, c, gs, up, od, ox)
                                            : walk<PASS, false>(it, p.a, b, c, gs, up, od, ox);
    if (PASS == StackPass::kNorm || PASS == StackPass::kDot) {
        const double t = block_sum256(ss);
        if (threadIdx.x == 0) partials[c] = t;
    }
}

template <StackPass PASS, int N>
cudaError_t launch(const StackItem* items, int n, const StackPassArgs& a, long long chunks, cudaStream_t stream) {
    PassParams<N> p;
    for (int i = 0; i < n; ++i) p.item[i] = items[i];
    p.a = a;
    p.n = n;
    stack_pass_kernel<PASS, N><<<static_cast<unsigned>(chunks), kStackThreads, 0, stream>>>(p);
    return cudaGetLastError();
}

template <StackPass PASS>
cudaError_t launch_any(StackItem* items, int n, const StackPassArgs& a, cudaStream_t stream) {
    for (int i0 = 0; i0 < n; i0 += kStackMaxItems) {
        const int m = n - i0 < kStackMaxItems ? n - i0 : kStackMaxItems;
        long long chunks = 0;
        for (int i = 0; i < m; ++i) {
            items[i0 + i].chunk0 = static_cast<int>(chunks);
            chunks += static_cast<long long>(items[i0 + i].chunks) * items[i0 + i].count;
            if (chunks > INT32_MAX) return cudaErrorInvalidValue;
        }
        if (chunks == 0) continue;
        StackPassArgs b = a;
        if (PASS == StackPass::kNorm && i0 > 0) b.status = nullptr;   // cleared once
        static_assert(sizeof(PassParams<kFewItems>) <= 4000, "the small form's parameters launch faster (see stack_chain.cu)");
        const cudaError_t e = m <= kFewItems ? launch<PASS, kFewItems>(items + i0, m, b, chunks, stream)
                                             : launch<PASS, kStackMaxItems>(items + i0, m, b, chunks, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t stack_pass_launch(StackPass pass, StackItem* items, int n, const StackPassArgs& a, cudaStream_t stream) {
    switch (pass) {
        case StackPass::kNorm: return launch_any<StackPass::kNorm>(items, n, a, stream);
        case StackPass::kPack: return launch_any<StackPass::kPack>(items, n, a, stream);
        case StackPass::kPackGrad: return launch_any<StackPass::kPackGrad>(items, n, a, stream);
        case StackPass::kOut: return launch_any<StackPass::kOut>(items, n, a, stream);
        case StackPass::kUpdate: return launch_any<StackPass::kUpdate>(items, n, a, stream);
        case StackPass::kDot: return launch_any<StackPass::kDot>(items, n, a, stream);
        case StackPass::kGradOut: return launch_any<StackPass::kGradOut>(items, n, a, stream);
    }
    return cudaErrorInvalidValue;
}

}  // namespace muon
