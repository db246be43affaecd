// Layer norm over rows of hs elements, forward and backward (the norm in front of the head).
//
//   forward   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) rstd gamma + beta
//   backward  with t = dy gamma and xh = (x - mu) rstd:
//             dx = rstd (t - mean(t) - xh mean(t xh)), dgamma = sum dy xh, dbeta = sum dy
//
// HBM bound: forward reads x and writes y, backward reads x and dy and writes dx, each once.
//
// Forward: a group of T threads holds a row, as it lies in memory, in registers (up to 128 bytes
// a thread, so that one or two warps hold a row and its two sums cost little): the mean, then the
// squared deviations from it (no cancellation for rows far from zero), then y.  Many small CTAs an
// SM overlap one another's loads, sums and stores.  Calls with few rows spread a row over more
// threads instead.
//
// Backward: a thread keeps its columns, 8 or 16 of them, over all the rows of its (persistent,
// one per SM) CTA, so that dgamma and dbeta build up in registers.  That leaves many threads a
// row and long sums, so rows are fetched ahead: each thread copies its own elements of the next
// rows into its own place in shared memory with cp.async and waits only for its own copies; no
// barrier guards the buffers.  The row is read from there twice, around the group's one sum.
// The CTAs' column sums meet in a fixed order (the workspace, then one kernel over it): the same
// bits on every call.
//
// Vectors: 16 bytes of x a load where addresses, strides and hs allow it, else 2 elements, else 1.
#include "vl_device.cuh"
#include "vl_internal.h"
#include "vl_rowio.cuh"
#include "vloss.h"

#include <atomic>

namespace vl {
namespace {

constexpr int FT = 512;                  // forward: threads of a row at most
constexpr int BT = 1024;                 // backward: threads of a CTA
constexpr int MAXG = 32;                 // rows a CTA works on at once

// V elements of type T, as they lie in memory.
template <typename T, int V>
struct Vec {
    static constexpr int BYTES = V * (int)sizeof(T);
    static constexpr int WORDS = (BYTES + 3) / 4;
    uint32_t w[WORDS];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (BYTES % 16 == 0) {
#pragma unroll
            for (int i = 0; i < BYTES / 16; ++i) {
                const uint4 r = reinterpret_cast<const uint4*>(p)[i];
                w[4 * i] = r.x;
                w[4 * i + 1] = r.y;
                w[4 * i + 2] = r.z;
                w[4 * i + 3] = r.w;
            }
        } else if constexpr (BYTES == 8) {
            const uint2 r = *reinterpret_cast<const uint2*>(p);
            w[0] = r.x;
            w[1] = r.y;
        } else if constexpr (BYTES == 4) {
            w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
            w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < WORDS; ++i) w[i] = 0u;
    }
    __device__ __forceinline__ float get(int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
    }
};

template <typename T, int V>
__device__ __forceinline__ void store_vec(T* p, const float (&f)[V]) {
    if constexpr (V * sizeof(T) == 16) {
        *reinterpret_cast<uint4*>(p) = Pack<T>::pack(f);
    } else if constexpr (sizeof(T) == 4 && V == 2) {
        *reinterpret_cast<float2*>(p) = make_float2(f[0], f[1]);
    } else if constexpr (sizeof(T) == 2 && V == 2) {
        *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(f[0], f[1]);
    } else {
        st_elem(p, f[0]);
    }
}

// Sum over a group of T threads (a multiple of 32) that use named barrier `id`; all get it.
// `red` alternates between calls, so that one barrier a sum is enough.
__device__ __forceinline__ float2 group_sum(float2 v, float2* red, int T, int id) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
    }
    if (T == 32) return v;
    const int lane = threadIdx.x & 31, w = (threadIdx.x % T) >> 5, W = T / 32;
    if (lane == 0) red[w] = v;
    named_sync((uint32_t)id, (uint32_t)T);
    if (W == 2) return make_float2(red[0].x + red[1].x, red[0].y + red[1].y);
    v = lane < W ? red[lane] : make_float2(0.f, 0.f);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
    }
    return v;
}
__device__ __forceinline__ float group_sum(float v, float2* red, int T, int id) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (T == 32) return v;
    const int lane = threadIdx.x & 31, w = (threadIdx.x % T) >> 5, W = T / 32;
    if (lane == 0) red[w].x = v;
    named_sync((uint32_t)id, (uint32_t)T);
    if (W == 2) return red[0].x + red[1].x;
    v = lane < W ? red[lane].x : 0.f;
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return __shfl_sync(0xffffffffu, v, 0);
}
static_assert(FT / 32 <= 16, "the forward sum's second step takes 16 lanes");

// n floats of an affine vector (nullptr: `none`).
template <int V>
__device__ __forceinline__ void load_affine(const float* p, int j, float none, float (&f)[V]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = none;
    } else if (V >= 4 && (reinterpret_cast<uintptr_t>(p) & 15u) == 0) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
            const float4 v = __ldg(reinterpret_cast<const float4*>(p + j) + i);
            f[4 * i] = v.x;
            f[4 * i + 1] = v.y;
            f[4 * i + 2] = v.z;
            f[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = __ldg(p + j + i);
    }
}

// One row a group of TH threads, U vectors of V elements a thread.
template <typename T, int V, int U>
__global__ void __launch_bounds__(FT) norm_fwd(const __grid_constant__ NormParams P, int TH) {
    __shared__ float2 red[MAXG][2][FT / 32];
    const int grp = threadIdx.x / TH, t = threadIdx.x % TH, groups = blockDim.x / TH, nv = P.hs / V;
    const long long r = (long long)blockIdx.x * groups + grp;
    pdl_launch_dependents();
    pdl_wait_primary();
    if (r >= P.rows) return;
    const T* x = static_cast<const T*>(P.x) + r * P.ldx + t * V;
    Vec<T, V> raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (t + u * TH < nv) raw[u].load(x + u * TH * V);
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        s[u] = 0.f;
        if (t + u * TH < nv)
#pragma unroll
            for (int i = 0; i < V; ++i) s[u] += raw[u].get(i);
    }
#pragma unroll
    for (int u = 1; u < U; ++u) s[0] += s[u];
    const float inv = 1.f / (float)P.hs;
    const float mu = group_sum(s[0], red[grp][0], TH, 1 + grp) * inv;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        s[u] = 0.f;
        if (t + u * TH < nv)
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float d = raw[u].get(i) - mu;
                s[u] = fmaf(d, d, s[u]);
            }
    }
#pragma unroll
    for (int u = 1; u < U; ++u) s[0] += s[u];
    const float var = group_sum(s[0], red[grp][1], TH, 1 + grp) * inv;
    const float rstd = 1.f / sqrtf(var + P.eps);
    if (t == 0) {
        if (P.mu_out) P.mu_out[r] = mu;
        if (P.rstd_out) P.rstd_out[r] = rstd;
    }
    T* y = static_cast<T*>(P.y) + r * P.ldy + t * V;
#pragma unroll
    for (int u = 0; u < U; ++u)
        if (t + u * TH < nv) {
            float o[V], ga[V], be[V];
            load_affine<V>(P.gamma, (t + u * TH) * V, 1.f, ga);
            load_affine<V>(P.beta, (t + u * TH) * V, 0.f, be);
#pragma unroll
            for (int i = 0; i < V; ++i) o[i] = fmaf((raw[u].get(i) - mu) * rstd, ga[i], be[i]);
            store_vec<T, V>(y + u * TH * V, o);
        }
}

// ---------------------------------------------------------------- backward

template <int BYTES>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src) {
    if constexpr (BYTES == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(dst), "l"(src) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" :: "r"(dst), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" :: "n"(N) : "memory"); }

// A thread's vector of V elements in shared memory: pieces of at most 16 bytes, piece q of thread
// t at (q blockDim + t) pieces, so that a warp's accesses are contiguous.
template <typename T, int V>
struct Slot {
    static constexpr int BYTES = V * (int)sizeof(T);
    static constexpr int PIECE = BYTES < 16 ? BYTES : 16;
    static constexpr int PIECES = BYTES / PIECE;
    static __device__ __forceinline__ void fetch(uint32_t base, const T* src) {
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
            const uint32_t dst = base + (uint32_t)((q * blockDim.x + threadIdx.x) * PIECE);
            if constexpr (PIECE >= 4) {
                cp_async<PIECE>(dst, reinterpret_cast<const char*>(src) + q * PIECE);
            } else {                               // two bytes: below what cp.async copies
                const uint16_t v = *reinterpret_cast<const uint16_t*>(src);
                asm volatile("st.shared.u16 [%0], %1;" :: "r"(dst), "h"(v) : "memory");
            }
        }
    }
    static __device__ __forceinline__ void read(uint32_t base, Vec<T, V>& v) {
#pragma unroll
        for (int q = 0; q < PIECES; ++q) {
            const uint32_t src = base + (uint32_t)((q * blockDim.x + threadIdx.x) * PIECE);
            if constexpr (PIECE == 16)
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v.w[4 * q]), "=r"(v.w[4 * q + 1]), "=r"(v.w[4 * q + 2]), "=r"(v.w[4 * q + 3]) : "r"(src) : "memory");
            else if constexpr (PIECE == 8)
                asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.w[0]), "=r"(v.w[1]) : "r"(src) : "memory");
            else if constexpr (PIECE == 4)
                asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v.w[0]) : "r"(src) : "memory");
            else {
                uint16_t h;
                asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(src) : "memory");
                v.w[0] = h;
            }
        }
    }
};

// Rows in flight: what 192 KB hold.
template <typename T, typename D, int E>
constexpr int kDepth = []() constexpr {
    const int n = 192 * 1024 / (BT * E * (int)(sizeof(T) + sizeof(D)));
    return n < 1 ? 1 : n > 6 ? 6 : n;
}();

template <typename T, typename D, int V, int E, bool SUMS>
__global__ void __launch_bounds__(BT, 1) norm_bwd(const __grid_constant__ NormParams P, int TH) {
    constexpr int U = E / V, DEPTH = kDepth<T, D, E>;
    constexpr bool REG = E <= 8;                      // gamma in registers, else from the caches
    extern __shared__ __align__(16) unsigned char dyn[];
    __shared__ float2 red[MAXG][2][BT / 32];
    __shared__ float stat[DEPTH][BT / 32][2];         // (mu, rstd) of the rows in flight, per warp
    const int grp = threadIdx.x / TH, t = threadIdx.x % TH, groups = blockDim.x / TH, nv = P.hs / V;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long stride = (long long)gridDim.x * groups;
    const long long r0 = (long long)blockIdx.x * groups + grp;
    const uint32_t sx = smem_u32(dyn), xs = blockDim.x * V * (uint32_t)sizeof(T), ds = blockDim.x * V * (uint32_t)sizeof(D);
    const uint32_t stage = U * (xs + ds);
    pdl_launch_dependents();
    pdl_wait_primary();
    auto fetch = [&](long long row, int st) {
        if (row < P.rows) {
            const T* x = static_cast<const T*>(P.x) + row * P.ldx + t * V;
            const D* dy = static_cast<const D*>(P.dy) + row * P.lddy + t * V;
            const uint32_t b = sx + st * stage;
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u * TH < nv) {
                    Slot<T, V>::fetch(b + u * xs, x + u * TH * V);
                    Slot<D, V>::fetch(b + U * xs + u * ds, dy + u * TH * V);
                }
            if (lane < 2) cp_async<4>(smem_u32(&stat[st][warp][lane]), (lane ? P.rstd : P.mu) + row);
        }
        cp_commit();
    };
    for (int d = 0; d < DEPTH; ++d) fetch(r0 + d * stride, d);
    float ga[REG ? U : 1][V], ag[U][V], ab[U][V];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (REG) {
            if (t + u * TH < nv) load_affine<V>(P.gamma, (t + u * TH) * V, 1.f, ga[REG ? u : 0]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) ag[u][i] = ab[u][i] = 0.f;
    }
    const float inv = 1.f / (float)P.hs;
    int st = 0, par = 0;
    for (long long r = r0; r < P.rows; r += stride, par ^= 1) {
        cp_wait<DEPTH - 1>();
        __syncwarp();
        const float mu = stat[st][warp][0], rs = stat[st][warp][1];
        const uint32_t b = sx + st * stage;
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u * TH < nv) {
                Vec<T, V> rx;
                Vec<D, V> rd;
                Slot<T, V>::read(b + u * xs, rx);
                Slot<D, V>::read(b + U * xs + u * ds, rd);
                if (!REG) load_affine<V>(P.gamma, (t + u * TH) * V, 1.f, ga[0]);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float d = rd.get(i), xh = (rx.get(i) - mu) * rs, g = d * ga[REG ? u : 0][i];
                    if (SUMS) {
                        ag[u][i] = fmaf(d, xh, ag[u][i]);
                        ab[u][i] += d;
                    }
                    s.x += g;
                    s.y = fmaf(g, xh, s.y);
                }
            }
        s = group_sum(s, red[grp][par], TH, 1 + grp);
        const float a = s.x * inv, c = s.y * inv;
        T* dx = static_cast<T*>(P.y) + r * P.ldy + t * V;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u * TH < nv) {
                Vec<T, V> rx;
                Vec<D, V> rd;
                Slot<T, V>::read(b + u * xs, rx);
                Slot<D, V>::read(b + U * xs + u * ds, rd);
                if (!REG) load_affine<V>(P.gamma, (t + u * TH) * V, 1.f, ga[0]);
                float o[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float xh = (rx.get(i) - mu) * rs;
                    o[i] = rs * ((rd.get(i) * ga[REG ? u : 0][i] - a) - xh * c);
                }
                store_vec<T, V>(dx + u * TH * V, o);
            }
        __syncwarp();                                // the warp has read mu and rstd
        fetch(r + DEPTH * stride, st);
        st = st + 1 == DEPTH ? 0 : st + 1;
    }
    cp_wait<0>();
    if (!SUMS) return;
    // the CTA's column sums: the groups' in order (in shared memory), then to the workspace
    float* const cols = reinterpret_cast<float*>(dyn);
    float* const out = P.part + (long long)blockIdx.x * 2 * P.hs;
    for (int g = 0; g < groups; ++g) {
        if (groups > 1) __syncthreads();
        if (grp == g)
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u * TH < nv)
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int j = (t + u * TH) * V + i;
                        if (g > 0) {
                            ag[u][i] += cols[j];
                            ab[u][i] += cols[P.hs + j];
                        }
                        float* to = g + 1 < groups ? cols : out;
                        to[j] = ag[u][i];
                        to[P.hs + j] = ab[u][i];
                    }
    }
}

// The partials of all CTAs: 32 columns a CTA, eight threads a column, each a run of the CTAs.
__global__ void __launch_bounds__(256) norm_join(const __grid_constant__ NormParams P, int parts) {
    __shared__ float red[8][32];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int lane = threadIdx.x & 31, seg = threadIdx.x >> 5;
    const int j = blockIdx.x * 32 + lane, cols = 2 * P.hs;
    const int per = (parts + 7) / 8, p0 = seg * per, p1 = min(parts, p0 + per);
    float s = 0.f;
    if (j < cols)
#pragma unroll 8
        for (int p = p0; p < p1; ++p) s += P.part[(long long)p * cols + j];
    red[seg][lane] = s;
    __syncthreads();
    if (seg == 0 && j < cols) {
        for (int k = 1; k < 8; ++k) s += red[k][lane];
        if (j < P.hs) {
            if (P.dgamma) P.dgamma[j] = s;
        } else if (P.dbeta) {
            P.dbeta[j - P.hs] = s;
        }
    }
}

// ---------------------------------------------------------------- launches

constexpr int kMaxParts = 256;           // CTAs of the backward pass, at most

int num_sms_dev() {
    static std::atomic<int> cache[64];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    sms = cache[dev].load(std::memory_order_acquire);
    if (sms > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cache[dev].store(sms, std::memory_order_release);
    return sms;
}

template <typename K, typename... Args>
cudaError_t launch_pdl(K kernel, long long grid, int threads, size_t smem, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Elements of a vector: bytes of x `vb` (16, 2 elements or 1) that every row start of every
// operand allows.
bool aligned(const void* p, long long ld, int es, int bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * es % bytes == 0;
}

template <typename T, int V, int U>
cudaError_t fwd_go(const NormParams& P, cudaStream_t st) {
    const int TH = ((P.hs + U * V - 1) / (U * V) + 31) / 32 * 32;
    const int groups = TH >= 256 ? 1 : TH == 32 ? 8 : 256 / TH;
    return launch_pdl(norm_fwd<T, V, U>, (P.rows + groups - 1) / groups, groups * TH, 0, st, P, TH);
}

template <typename T>
cudaError_t fwd(const NormParams& P, cudaStream_t st) {
    constexpr int N = Pack<T>::N, es = sizeof(T);
    auto ok = [&](int n) {
        return P.hs % n == 0 && aligned(P.x, P.ldx, es, n * es) && aligned(P.y, P.ldy, es, n * es);
    };
    if (ok(N)) {
        // few rows: one vector a thread, the shortest path through a row (while 512 threads take it)
        if (P.rows <= num_sms_dev() && P.hs <= FT * N) return fwd_go<T, N, 1>(P, st);
        return fwd_go<T, N, 8>(P, st);
    }
    if (ok(2)) return fwd_go<T, 2, 16>(P, st);
    return fwd_go<T, 1, 32>(P, st);
}

// Threads a row and rows a CTA of the backward pass, E elements a thread.
struct Shape {
    int E, TH, groups;
};

Shape shape_of(int hs) {
    Shape s;
    s.E = hs <= 8 * BT ? 8 : 16;
    s.TH = ((hs + s.E - 1) / s.E + 31) / 32 * 32;
    s.groups = BT / s.TH;
    if (s.TH > 32 && s.groups > 15) s.groups = 15;      // named barriers 1 .. 15
    return s;
}

template <typename T, typename D, int V, int E>
cudaError_t bwd_go(const NormParams& P, const Shape& s, cudaStream_t st) {
    const bool sums = P.dgamma || P.dbeta;
    const int sms = num_sms_dev(), threads = s.groups * s.TH;
    long long grid = (P.rows + s.groups - 1) / s.groups;
    if (grid > sms) grid = sms;
    if (grid > kMaxParts) grid = kMaxParts;
    const size_t ring = (size_t)kDepth<T, D, E> * threads * E * (sizeof(T) + sizeof(D));
    const size_t meet = sums && s.groups > 1 ? 8 * (size_t)P.hs : 0, smem = ring > meet ? ring : meet;
    const void* fn = sums ? (const void*)norm_bwd<T, D, V, E, true> : (const void*)norm_bwd<T, D, V, E, false>;
    cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = sums ? launch_pdl(norm_bwd<T, D, V, E, true>, grid, threads, smem, st, P, s.TH)
             : launch_pdl(norm_bwd<T, D, V, E, false>, grid, threads, smem, st, P, s.TH);
    if (e == cudaSuccess && sums) e = launch_pdl(norm_join, (2 * P.hs + 31) / 32, 256, 0, st, P, (int)grid);
    return e;
}

template <typename T, typename D, int V>
cudaError_t bwd_e(const NormParams& P, cudaStream_t st) {
    const Shape s = shape_of(P.hs);
    return s.E == 8 ? bwd_go<T, D, V, 8>(P, s, st) : bwd_go<T, D, V, 16>(P, s, st);
}

template <typename T, typename D>
cudaError_t bwd(const NormParams& P, cudaStream_t st) {
    constexpr int N = Pack<T>::N, es = sizeof(T), ds = sizeof(D);
    if (P.rows == 0) return launch_pdl(norm_join, (2 * P.hs + 31) / 32, 256, 0, st, P, 0);
    auto ok = [&](int n) {
        const int db = n * ds < 16 ? n * ds : 16;
        return P.hs % n == 0 && aligned(P.x, P.ldx, es, n * es) && aligned(P.y, P.ldy, es, n * es) &&
               aligned(P.dy, P.lddy, ds, db);
    };
    if (ok(N)) return bwd_e<T, D, N>(P, st);
    if (ok(2)) return bwd_e<T, D, 2>(P, st);
    return bwd_e<T, D, 1>(P, st);
}

}  // namespace

long long norm_bwd_ws_bytes(long long rows, long long hs) {
    const Shape s = shape_of((int)hs);
    const long long want = (rows + s.groups - 1) / s.groups;
    return (want < kMaxParts ? want : kMaxParts) * 2 * hs * 4;
}

cudaError_t launch_norm_fwd(const NormParams& P, cudaStream_t st) {
    return P.dtype == kBf16 ? fwd<__nv_bfloat16>(P, st) : fwd<float>(P, st);
}

cudaError_t launch_norm_bwd(const NormParams& P, cudaStream_t st) {
    if (P.dtype != kBf16) return bwd<float, float>(P, st);
    return P.dy_f32 ? bwd<__nv_bfloat16, float>(P, st) : bwd<__nv_bfloat16, __nv_bfloat16>(P, st);
}

}  // namespace vl
