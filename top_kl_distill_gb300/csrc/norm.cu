// Layer norm over rows of hs elements, forward and backward (the norm in front of the head).
//
//   forward   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) rstd gamma + beta
//   backward  with t = dy gamma and xh = (x - mu) rstd:
//             dx = rstd (t - mean(t) - xh mean(t xh)), dgamma = sum dy xh, dbeta = sum dy
#include "vl_device.cuh"
#include "vl_internal.h"
#include "vl_rowio.cuh"

namespace vl {
namespace {

constexpr int NT = 256;
constexpr int kParts = 64;               // row chunks whose partial column sums are kept

__device__ __forceinline__ float2 cta_sum2(float2 v, float2* red) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float2 s = make_float2(0.f, 0.f);
    for (int i = 0; i < NT / 32; ++i) {
        s.x += red[i].x;
        s.y += red[i].y;
    }
    return s;
}

template <typename T>
__global__ void __launch_bounds__(NT) norm_fwd(const __grid_constant__ NormParams P) {
    __shared__ float2 red[NT / 32];
    pdl_wait_primary();
    pdl_launch_dependents();
    for (long long r = blockIdx.x; r < P.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(P.x) + r * P.ldx;
        T* y = static_cast<T*>(P.y) + r * P.ldy;
        float s = 0.f;
        for (int j = threadIdx.x; j < P.hs; j += NT) s += ld_elem(x + j);
        const float mu = cta_sum2(make_float2(s, 0.f), red).x / (float)P.hs;
        float v = 0.f;
        for (int j = threadIdx.x; j < P.hs; j += NT) {
            const float d = ld_elem(x + j) - mu;
            v += d * d;
        }
        const float var = cta_sum2(make_float2(v, 0.f), red).x / (float)P.hs;
        const float rstd = 1.f / sqrtf(var + P.eps);
        if (threadIdx.x == 0) {
            if (P.mu_out) P.mu_out[r] = mu;
            if (P.rstd_out) P.rstd_out[r] = rstd;
        }
        for (int j = threadIdx.x; j < P.hs; j += NT)
            st_elem(y + j, (ld_elem(x + j) - mu) * rstd * (P.gamma ? P.gamma[j] : 1.f) + (P.beta ? P.beta[j] : 0.f));
    }
}

template <typename T, typename D>
__global__ void __launch_bounds__(NT) norm_bwd_dx(const __grid_constant__ NormParams P) {
    __shared__ float2 red[NT / 32];
    pdl_wait_primary();
    pdl_launch_dependents();
    for (long long r = blockIdx.x; r < P.rows; r += gridDim.x) {
        const T* x = static_cast<const T*>(P.x) + r * P.ldx;
        const D* dy = static_cast<const D*>(P.dy) + r * P.lddy;
        T* dx = static_cast<T*>(P.y) + r * P.ldy;
        const float mu = P.mu[r], rstd = P.rstd[r];
        float2 s = make_float2(0.f, 0.f);
        for (int j = threadIdx.x; j < P.hs; j += NT) {
            const float t = ld_elem(dy + j) * (P.gamma ? P.gamma[j] : 1.f);
            s.x += t;
            s.y += t * ((ld_elem(x + j) - mu) * rstd);
        }
        s = cta_sum2(s, red);
        const float a = s.x / (float)P.hs, b = s.y / (float)P.hs;
        for (int j = threadIdx.x; j < P.hs; j += NT) {
            const float t = ld_elem(dy + j) * (P.gamma ? P.gamma[j] : 1.f);
            st_elem(dx + j, rstd * (t - a - ((ld_elem(x + j) - mu) * rstd) * b));
        }
    }
}

// Partial column sums of row chunk blockIdx.y: part[chunk][0 / 1][hs].
template <typename T, typename D>
__global__ void __launch_bounds__(NT) norm_bwd_part(const __grid_constant__ NormParams P) {
    pdl_wait_primary();
    pdl_launch_dependents();
    const int j = blockIdx.x * NT + threadIdx.x;
    if (j >= P.hs) return;
    const long long per = (P.rows + kParts - 1) / kParts;
    const long long r0 = blockIdx.y * per, r1 = min(P.rows, r0 + per);
    float g = 0.f, b = 0.f;
    for (long long r = r0; r < r1; ++r) {
        const float d = ld_elem(static_cast<const D*>(P.dy) + r * P.lddy + j);
        g += d * ((ld_elem(static_cast<const T*>(P.x) + r * P.ldx + j) - P.mu[r]) * P.rstd[r]);
        b += d;
    }
    P.part[(long long)(2 * blockIdx.y) * P.hs + j] = g;
    P.part[(long long)(2 * blockIdx.y + 1) * P.hs + j] = b;
}

__global__ void __launch_bounds__(NT) norm_bwd_join(const __grid_constant__ NormParams P) {
    pdl_wait_primary();
    pdl_launch_dependents();
    const int j = blockIdx.x * NT + threadIdx.x;
    if (j >= P.hs) return;
    float g = 0.f, b = 0.f;
    if (P.rows > 0)
        for (int k = 0; k < kParts; ++k) {
            g += P.part[(long long)(2 * k) * P.hs + j];
            b += P.part[(long long)(2 * k + 1) * P.hs + j];
        }
    if (P.dgamma) P.dgamma[j] = g;
    if (P.dbeta) P.dbeta[j] = b;
}

template <typename K>
cudaError_t launch_pdl(K kernel, dim3 grid, const NormParams& P, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(NT, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, P);
}

template <typename T, typename D>
cudaError_t bwd(const NormParams& P, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    const unsigned cols = (unsigned)((P.hs + NT - 1) / NT);
    if (P.dgamma || P.dbeta) {
        if (P.rows > 0) e = launch_pdl(norm_bwd_part<T, D>, dim3(cols, kParts), P, st);
        if (e == cudaSuccess) e = launch_pdl(norm_bwd_join, dim3(cols), P, st);
    }
    if (e == cudaSuccess && P.rows > 0)
        e = launch_pdl(norm_bwd_dx<T, D>, dim3((unsigned)(P.rows < 65536 ? P.rows : 65536)), P, st);
    return e;
}

}  // namespace

long long norm_bwd_ws_bytes(long long rows, long long hs) {
    (void)rows;
    return 2ll * kParts * hs * 4;
}

cudaError_t launch_norm_fwd(const NormParams& P, cudaStream_t st) {
    const dim3 grid((unsigned)(P.rows < 65536 ? P.rows : 65536));
    return P.dtype == kBf16 ? launch_pdl(norm_fwd<__nv_bfloat16>, grid, P, st) : launch_pdl(norm_fwd<float>, grid, P, st);
}

cudaError_t launch_norm_bwd(const NormParams& P, cudaStream_t st) {
    if (P.dtype != kBf16) return bwd<float, float>(P, st);
    return P.dy_f32 ? bwd<__nv_bfloat16, float>(P, st) : bwd<__nv_bfloat16, __nv_bfloat16>(P, st);
}

}  // namespace vl
