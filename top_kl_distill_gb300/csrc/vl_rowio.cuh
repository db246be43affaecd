// Reading and writing rows of fp32 or bf16 elements at any alignment: 16-byte chunks where
// the rows allow them, single elements elsewhere.  bf16 values are widened exactly on the way
// in and rounded once (nearest even) on the way out.
#pragma once

#include "vl_device.cuh"

#include <cuda_bf16.h>

namespace vl {

template <typename T>
struct Pack;

template <>
struct Pack<float> {
    static constexpr int N = 4;          // elements of 16 bytes
    static __device__ __forceinline__ void unpack(uint4 r, float (&f)[N]) {
        f[0] = __uint_as_float(r.x);
        f[1] = __uint_as_float(r.y);
        f[2] = __uint_as_float(r.z);
        f[3] = __uint_as_float(r.w);
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[N]) {
        return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    }
};

template <>
struct Pack<__nv_bfloat16> {
    static constexpr int N = 8;
    static __device__ __forceinline__ void unpack(uint4 r, float (&f)[N]) {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float (&f)[N]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ float ld_elem(const float* p) { return *p; }
__device__ __forceinline__ float ld_elem(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void st_elem(float* p, float v) { *p = v; }
__device__ __forceinline__ void st_elem(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Elements before the first 16-byte boundary of a row of n.
template <typename T>
__device__ __forceinline__ int head_len(const T* p, int n) {
    const int h = (int)(((16u - (unsigned)(reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / sizeof(T));
    return h < n ? h : n;
}

// (max, sum of exp(x - max)) of one thread's share of a row: chunks t, t + NT, ...
template <typename T, int NT>
__device__ MaxSum row_max_sum(const T* x, int n, int t) {
    constexpr int N = Pack<T>::N;
    MaxSum ms = ms_empty();
    const int h = head_len(x, n), nb = (n - h) / N;
    const uint4* x4 = reinterpret_cast<const uint4*>(x + h);
    for (int i = t; i < nb; i += NT) {
        float v[N];
        Pack<T>::unpack(x4[i], v);
        float mx = v[0];
#pragma unroll
        for (int k = 1; k < N; ++k) mx = fmaxf(mx, v[k]);
        if (mx > ms.m) {
            ms.s *= ex2((ms.m - mx) * kLog2e);
            ms.m = mx;
        }
        float e = 0.f;
#pragma unroll
        for (int k = 0; k < N; ++k) e += ex2((v[k] - ms.m) * kLog2e);
        ms.s += e;
    }
    if (t < h) ms_add(ms, ld_elem(x + t));
    const int t0 = h + nb * N;
    if (t0 + t < n) ms_add(ms, ld_elem(x + t0 + t));
    return ms;
}

// g[j] = c ([j == a] - exp(x_j - m - lnS)); c == 0: zeros, and x is not read.
template <typename T, int NT>
__device__ void row_gradient(const T* x, T* g, int n, int t, float m, float lnS, float c, int a) {
    constexpr int N = Pack<T>::N;
    const int h = head_len(g, n), nb = (n - h) / N, t0 = h + nb * N;
    const bool wide = head_len(x, n) == h || c == 0.f;
    auto one = [&](int j) {
        float o = 0.f;
        if (c != 0.f) {
            o = -c * ex2(((ld_elem(x + j) - m) - lnS) * kLog2e);
            if (j == a) o += c;
        }
        st_elem(g + j, o);
    };
    if (!wide) {
        for (int j = t; j < n; j += NT) one(j);
        return;
    }
    for (int i = t; i < nb; i += NT) {
        float o[N];
#pragma unroll
        for (int k = 0; k < N; ++k) o[k] = 0.f;
        if (c != 0.f) {
            float v[N];
            Pack<T>::unpack(reinterpret_cast<const uint4*>(x + h)[i], v);
            const int j = h + i * N;
#pragma unroll
            for (int k = 0; k < N; ++k) {
                o[k] = -c * ex2(((v[k] - m) - lnS) * kLog2e);
                if (j + k == a) o[k] += c;
            }
        }
        reinterpret_cast<uint4*>(g + h)[i] = Pack<T>::pack(o);
    }
    if (t < h) one(t);
    if (t0 + t < n) one(t0 + t);
}

}  // namespace vl
