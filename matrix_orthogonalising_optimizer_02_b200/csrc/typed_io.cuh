// Loads and stores of 8 (or fewer) consecutive elements of fp32, bf16 or fp16 arrays, held in fp32.
#pragma once
#include <cuda_fp16.h>

#include "ptx_sm100.cuh"

namespace muon {

__device__ __forceinline__ void unpack8(const uint4& w, int dtype, float (&v)[8]) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        if (dtype == MUON_F16) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&x[h]));
            v[2 * h] = f.x;
            v[2 * h + 1] = f.y;
        } else {
            v[2 * h] = bf16_lo_to_f32(x[h]);
            v[2 * h + 1] = bf16_hi_to_f32(x[h]);
        }
    }
}
__device__ __forceinline__ uint4 pack8(int dtype, const float (&v)[8]) {
    uint32_t x[4];
#pragma unroll
    for (int h = 0; h < 4; ++h) {
        if (dtype == MUON_F16) {
            const __half2 p = __floats2half2_rn(v[2 * h], v[2 * h + 1]);
            x[h] = *reinterpret_cast<const uint32_t*>(&p);
        } else {
            x[h] = pack_bf16x2(v[2 * h], v[2 * h + 1]);
        }
    }
    return make_uint4(x[0], x[1], x[2], x[3]);
}

__device__ __forceinline__ float load_elem(const void* p, int dtype, long long e) {
    if (dtype == MUON_F32) return static_cast<const float*>(p)[e];
    if (dtype == MUON_F16) return __half2float(static_cast<const __half*>(p)[e]);
    return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[e]);
}
__device__ __forceinline__ void store_elem(void* p, int dtype, long long e, float v) {
    if (dtype == MUON_F32) static_cast<float*>(p)[e] = v;
    else if (dtype == MUON_F16) static_cast<__half*>(p)[e] = __float2half_rn(v);
    else static_cast<__nv_bfloat16*>(p)[e] = __float2bfloat16_rn(v);
}

// Calls f with a value of the element type: code for several elements chooses the type once, so that their
// loads are under way together.
template <class F>
__device__ __forceinline__ void by_type(int dtype, F f) {
    if (dtype == MUON_F32) f(float());
    else if (dtype == MUON_F16) f(__half());
    else f(__nv_bfloat16());
}
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void narrow(float& d, float x) { d = x; }
__device__ __forceinline__ void narrow(__half& d, float x) { d = __float2half_rn(x); }
__device__ __forceinline__ void narrow(__nv_bfloat16& d, float x) { d = __float2bfloat16_rn(x); }

// Elements e .. e + n - 1 (n <= 8; the rest of v is zero).  vec: e is 16-byte aligned and n == 8.
__device__ __forceinline__ void load8(const void* p, int dtype, long long e, int n, bool vec, float (&v)[8]) {
    if (vec && n == 8) {
        if (dtype == MUON_F32) {
            const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + e);
            const float4 a = q[0], b = q[1];
            v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
        } else {
            unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + e), dtype, v);
        }
    } else {
        by_type(dtype, [&](auto t) {
            using E = decltype(t);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = j < n ? widen(static_cast<const E*>(p)[e + j]) : 0.f;
        });
    }
}
__device__ __forceinline__ void store8(void* p, int dtype, long long e, int n, bool vec, const float (&v)[8]) {
    if (vec && n == 8) {
        if (dtype == MUON_F32) {
            float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + e);
            q[0] = make_float4(v[0], v[1], v[2], v[3]);
            q[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + e) = pack8(dtype, v);
        }
    } else {
        by_type(dtype, [&](auto t) {
            using E = decltype(t);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < n) narrow(static_cast<E*>(p)[e + j], v[j]);
        });
    }
}

// Sum over a block of 256 threads, the same in every thread; fixed order.
__device__ __forceinline__ double block_sum256(double v) {
    __shared__ double red[8];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += red[i];
    return s;
}

}  // namespace muon
