// Layer norm over rows of hs elements, forward and backward (the norm in front of the head).
//
//   forward   mu = mean(x), rstd = 1 / sqrt(mean((x - mu)^2) + eps), y = (x - mu) rstd gamma + beta
//   backward  with t = dy gamma and xh = (x - mu) rstd:
//             dx = rstd (t - mean(t) - xh mean(t xh)), dgamma = sum dy xh, dbeta = sum dy
//
// HBM bound: forward reads x and writes y, backward reads x and dy and writes dx, each once.
//
// One persistent CTA per SM; a row belongs to a group of T threads, 16 to 64 elements a
// thread, several groups a CTA.  A group's rows are fetched ahead of it by 1-D bulk copies (TMA) into its
// ring in shared memory, a row a stage: one copy of each operand, issued by one thread.  (With a
// cp.async per 16 bytes and thread instead, issuing the copies was half of the backward pass's
// time.)  A row is read from its stage once, so the group's own sum, whose barrier every thread
// passes after reading, is what frees the stage.  Backward threads keep their columns over all
// rows: gamma stays in registers, and dgamma and dbeta build up there; forward keeps gamma and beta
// in shared memory (from the caches, which the ring leaves 30 KB, they took half of a row's time).
// Forward takes the mean, then the squared deviations from it (no cancellation for rows far from
// zero), each one sum over the group (one meeting, with deviations from each warp's own mean, took
// 49.6 us against 47.7 at 16384 x 4096 bf16); backward one sum of two values.  At that size forward
// reaches 0.83 of the copy rate, backward (fp32 dy, 85 us) 0.93.  The CTAs' column sums meet in a fixed order (the
// workspace, then one kernel over it): the same bits on every call.
//
// Alignment: a copy covers the 16-byte blocks that hold the row, so that it starts on a 16-byte
// boundary; where those blocks would leave the matrix (its first and last row at most) the group
// copies the row element by element.  Threads read 16 bytes of x (8 beside an fp32 dy of a bf16
// row) at a time where addresses, strides and hs allow it, else 2 elements, else 1.
//
// Forward calls of few rows (norm_fwd_few) instead spread a row over more threads, one to four
// vectors each, straight from global memory: the shortest path through a row.
#include "vl_api.h"
#include "vl_device.cuh"
#include "vl_internal.h"
#include "vl_launch.h"
#include "vl_pair.cuh"
#include "vl_rowio.cuh"
#include "vloss.h"

#include <atomic>

namespace vl {
namespace {

constexpr int FEW = 512;                 // threads of a row at most, calls of few rows
constexpr int FWD = 768, BWD = 512;      // threads of a CTA: up to 80 and 128 registers each
constexpr int FWD64 = 512;               // forward with 64 elements a thread
constexpr int RING_B = 192 * 1024;       // shared memory for rows in flight (forward: and gamma and beta)
constexpr int MAXD = 8;                  // rows in flight a group
constexpr int MAXG = FWD / 32;           // groups a CTA

__device__ unsigned int g_watchdog;

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
    } else if constexpr (sizeof(T) == 2 && V == 4) {
        const __nv_bfloat162 a = __floats2bfloat162_rn(f[0], f[1]), b = __floats2bfloat162_rn(f[2], f[3]);
        *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
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
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, W = T / 32;
    if (lane == 0) red[w] = v;
    named_sync((uint32_t)id, (uint32_t)T);
    if (W <= 4) {
        v = make_float2(red[0].x + red[1].x, red[0].y + red[1].y);
        if (W > 2) v = make_float2(v.x + red[2].x, v.y + red[2].y);
        return W > 3 ? make_float2(v.x + red[3].x, v.y + red[3].y) : v;
    }
    v = (lane & 15) < W ? red[lane & 15] : make_float2(0.f, 0.f);      // W <= BWD / 32
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, off);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, off);
    }
    return v;
}
__device__ __forceinline__ float group_sum(float v, float2* red, int T, int id) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if (T == 32) return v;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, W = T / 32;
    if (lane == 0) red[w].x = v;
    named_sync((uint32_t)id, (uint32_t)T);
    if (W <= 4) {
        v = red[0].x + red[1].x;
        if (W > 2) v += red[2].x;
        return W > 3 ? v + red[3].x : v;
    }
    v = lane < W ? red[lane].x : 0.f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}


// The pairs of n = U V elements a thread has of a row, element i of vector u at u V + i.
template <typename T, int V, int U>
__device__ __forceinline__ void to_pairs(const Vec<T, V> (&v)[U], uint64_t (&p)[U * V / 2]) {
#pragma unroll
    for (int k = 0; k < U * V / 2; ++k) p[k] = pack2(v[2 * k / V].get(2 * k % V), v[(2 * k + 1) / V].get((2 * k + 1) % V));
}
template <typename T, int V, int U>
__device__ __forceinline__ void from_pairs(const uint64_t (&p)[U * V / 2], int u, float (&o)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = u * V + i;
        float a, b;
        unpack2(p[e / 2], a, b);
        o[i] = e & 1 ? b : a;
    }
}

// V floats of an affine vector at column j (nullptr: `none`); wide: 4 V bytes a load.  The kernel before this one in
// the stream may have written them (an optimiser's step).
template <int V>
__device__ __forceinline__ void load_affine(const float* p, int j, bool wide, float none, float (&f)[V]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = none;
        return;
    }
    if constexpr (V == 8) {
        if (wide) {
            asm volatile("ld.global.v8.f32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                         : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3]), "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
                         : "l"(p + j) : "memory");
            return;
        }
    } else if constexpr (V == 4) {
        if (wide) {
            const float4 v = *reinterpret_cast<const float4*>(p + j);
            f[0] = v.x;
            f[1] = v.y;
            f[2] = v.z;
            f[3] = v.w;
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = p[j + i];
}
__device__ __forceinline__ bool wide_affine(const float* p, int V) {
    return (reinterpret_cast<uintptr_t>(p) & (uintptr_t)(4 * V - 1)) == 0;
}

// ---------------------------------------------------------------- rows in flight

// Bytes of a stage for rows of n elements: the 16-byte blocks of a row at any alignment.
template <typename T>
__host__ __device__ __forceinline__ int stage_bytes(int n) {
    return ((n * (int)sizeof(T) + 15) / 16 + 1) * 16;
}

// What this thread has seen written to shared memory (a row copied by hand) comes before the bulk
// copies it issues next.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

struct alignas(16) Bars {
    uint64_t full[MAXG][MAXD];
    int abort;
};

// A wait that ran out (a bug) leaves copies in flight: they land before the CTA goes.
__device__ __forceinline__ void drain(Bars& B, int grp, int depth, uint32_t used, int t) {
    if (t == 0 && *(volatile int*)&B.abort)
        for (int d = 0; d < depth; ++d) wait_parity_drain(&B.full[grp][d], (used >> d) & 1u, 200000000ll);
}

// One operand of the pass: a matrix of rows of hs elements.
template <typename T>
struct Rows {
    const unsigned char* p;
    long long pitch;                                  // bytes
    uint32_t low, lowp;                               // their low words, for offsets within a 16-byte block
    __device__ __forceinline__ Rows(const void* q, long long ld)
        : p(static_cast<const unsigned char*>(q)), pitch(ld * (long long)sizeof(T)),
          low((uint32_t)reinterpret_cast<uintptr_t>(q)), lowp((uint32_t)(ld * (long long)sizeof(T))) {}
    // where row r starts inside its stage
    __device__ __forceinline__ uint32_t offset(long long r) const { return (low + (uint32_t)r * lowp) & 15u; }
    // bytes of the 16-byte blocks that hold row r
    __device__ __forceinline__ uint32_t bytes(long long r, int hs) const {
        return (offset(r) + (uint32_t)hs * (uint32_t)sizeof(T) + 15u) & ~15u;
    }
    __device__ __forceinline__ void copy(long long r, int hs, unsigned char* stage, uint64_t* bar) const {
        bulk_g2s(stage, p + r * pitch - offset(r), bytes(r, hs), bar);
    }
    // the group's threads copy row r themselves
    __device__ __forceinline__ void copy_by_hand(long long r, int hs, unsigned char* stage, int t, int TH) const {
        T* to = reinterpret_cast<T*>(stage + offset(r));
        for (int j = t; j < hs; j += TH) to[j] = reinterpret_cast<const T*>(p + r * pitch)[j];
    }
};

// Rows [lo, hi) whose 16-byte blocks lie inside the matrices (all but a row or two at the ends).
struct Safe {
    long long lo, hi;
    __device__ __forceinline__ bool has(long long r) const { return r >= lo && r < hi; }
};

// ---------------------------------------------------------------- forward

// Few rows: a row a CTA, C vectors of V elements a thread.
template <typename T, int V, int C>
__global__ void __launch_bounds__(FEW) norm_fwd_few(const __grid_constant__ NormParams P) {
    __shared__ float2 red[2][FEW / 32];
    const int t = threadIdx.x, TH = blockDim.x, nv = P.hs / V;
    const long long r = blockIdx.x;
    const bool wg = wide_affine(P.gamma, V), wb = wide_affine(P.beta, V);
    float ga[C][V], be[C][V], x[C][V], s = 0.f;
    pdl_launch_dependents();
    pdl_wait_primary();
    Vec<T, V> raw[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int q = t + c * TH;
        raw[c].zero();
        if (q < nv) {
            raw[c].load(static_cast<const T*>(P.x) + r * P.ldx + q * V);
            load_affine<V>(P.gamma, q * V, wg, 1.f, ga[c]);
            load_affine<V>(P.beta, q * V, wb, 0.f, be[c]);
        }
    }
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < V; ++i) s += raw[c].get(i);
    const float inv = 1.f / (float)P.hs;
    const float mu = group_sum(s, red[0], TH, 1) * inv;
    s = 0.f;
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[c][i] = t + c * TH < nv ? raw[c].get(i) - mu : 0.f;
            s = fmaf(x[c][i], x[c][i], s);
        }
    const float var = group_sum(s, red[1], TH, 1) * inv;
    const float rstd = __frsqrt_rn(var + P.eps);
    if (t == 0) {
        if (P.mu_out) P.mu_out[r] = mu;
        if (P.rstd_out) P.rstd_out[r] = rstd;
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int q = t + c * TH;
        if (q >= nv) break;
#pragma unroll
        for (int i = 0; i < V; ++i) x[c][i] = fmaf(x[c][i] * rstd, ga[c][i], be[c][i]);
        store_vec<T, V>(static_cast<T*>(P.y) + r * P.ldy + q * V, x[c]);
    }
}

template <typename T, int V, int E>
__global__ void __launch_bounds__(E == 64 ? FWD64 : FWD, 1) norm_fwd(const __grid_constant__ NormParams P, int depth, Safe safe) {
    constexpr int U = E / V, E2 = E / 2;
    extern __shared__ __align__(128) unsigned char dyn[];     // the groups' rings; gamma, beta
    __shared__ Bars B;
    __shared__ float2 red[MAXG][4][FWD / 32];
    const int grp = threadIdx.y, t = threadIdx.x, TH = blockDim.x, groups = blockDim.y, hs = P.hs, nv = hs / V;
    const long long stride = (long long)gridDim.x * groups, r0 = (long long)blockIdx.x * groups + grp;
    const int sb = stage_bytes<T>(hs);
    unsigned char* const ring = dyn + (size_t)grp * depth * sb;
    const Rows<T> X(P.x, P.ldx);
    if (t == 0) {
        for (int d = 0; d < depth; ++d) mbar_init(&B.full[grp][d], 1);
        fence_mbar_init_cluster();
    }
    if (t == 0 && grp == 0) B.abort = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait_primary();
    auto fetch = [&](long long row, int st) {
        if (!safe.has(row)) return;
        fence_async();
        mbar_arrive_expect_tx(&B.full[grp][st], X.bytes(row, hs));
        X.copy(row, hs, ring + (size_t)st * sb, &B.full[grp][st]);
    };
    if (t == 0)
        for (int d = 0; d < depth; ++d) fetch(r0 + d * stride, d);
    // gamma and beta in pieces of F floats: piece q of all vectors after piece q - 1 of all, so that
    // a warp's 16-byte reads lie side by side
    constexpr int F = V < 4 ? V : 4;
    float* const aff = reinterpret_cast<float*>(dyn + (size_t)groups * depth * sb);
    for (int j = grp * TH + t; j < hs; j += groups * TH) {
        const int at = (j % V / F * nv + j / V) * F + j % F;
        aff[at] = P.gamma ? P.gamma[j] : 1.f;
        aff[hs + at] = P.beta ? P.beta[j] : 0.f;
    }
    __syncthreads();
    auto affine = [&](const float* a, int v, float (&f)[V]) {
#pragma unroll
        for (int q = 0; q < V / F; ++q) {
            const float* p = a + (q * nv + v) * F;
            if constexpr (F == 4) {
                const float4 w = *reinterpret_cast<const float4*>(p);
                f[4 * q] = w.x;
                f[4 * q + 1] = w.y;
                f[4 * q + 2] = w.z;
                f[4 * q + 3] = w.w;
            } else {
#pragma unroll
                for (int i = 0; i < F; ++i) f[i] = p[i];
            }
        }
    };
    const float inv = 1.f / (float)hs;
    const bool full = nv == U * TH;                   // no vector past the row's end
    auto tree = [](uint64_t (&s)[4]) { return sum2(add2(add2(s[0], s[1]), add2(s[2], s[3]))); };
    int st = 0, par = 0;
    uint32_t used = 0;                                // bit st: the phase of stage st to wait for
    for (long long r = r0; r < P.rows; r += stride, par ^= 2) {
        unsigned char* const stage = ring + (size_t)st * sb;
        if (safe.has(r)) {
            wait_parity<false>(&B.full[grp][st], (used >> st) & 1u, &B.abort, &g_watchdog);
            used ^= 1u << st;
        } else {
            X.copy_by_hand(r, hs, stage, t, TH);
            if (TH == 32) __syncwarp();
            else named_sync(1 + grp, TH);
        }
        const T* x = reinterpret_cast<const T*>(stage + X.offset(r)) + t * V;
        uint64_t p[E2];
        {
            Vec<T, V> raw[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                raw[u].zero();
                if (t + u * TH < nv) raw[u].load(x + u * TH * V);
            }
            to_pairs<T, V, U>(raw, p);
        }
        uint64_t s[4] = {};
#pragma unroll
        for (int k = 0; k < E2; ++k) s[k & 3] = add2(s[k & 3], p[k]);
        const float mu = group_sum(tree(s), red[grp][par], TH, 1 + grp) * inv;
        if (t == 0) fetch(r + depth * stride, st);    // past the sum: every thread has read its stage
        const uint64_t nmu = both(-mu);
#pragma unroll
        for (int k = 0; k < 4; ++k) s[k] = 0;
#pragma unroll
        for (int k = 0; k < E2; ++k) {
            p[k] = add2(p[k], nmu);
            if (!full) {
                float a, b;
                unpack2(p[k], a, b);
                if (t + 2 * k / V * TH >= nv) a = 0.f;
                if (t + (2 * k + 1) / V * TH >= nv) b = 0.f;
                p[k] = pack2(a, b);
            }
            s[k & 3] = fma2(p[k], p[k], s[k & 3]);
        }
        const float var = group_sum(tree(s), red[grp][par + 1], TH, 1 + grp) * inv;
        const float rstd = __frsqrt_rn(var + P.eps);
        if (t == 0) {
            if (P.mu_out) P.mu_out[r] = mu;
            if (P.rstd_out) P.rstd_out[r] = rstd;
        }
        const uint64_t rs2 = both(rstd);
#pragma unroll
        for (int k = 0; k < E2; ++k) p[k] = mul2(p[k], rs2);
        T* y = static_cast<T*>(P.y) + r * P.ldy + t * V;
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (t + u * TH < nv) {
                float o[V], ga[V], be[V];
                affine(aff, t + u * TH, ga);
                affine(aff + hs, t + u * TH, be);
                from_pairs<T, V, U>(p, u, o);
#pragma unroll
                for (int i = 0; i < V; ++i) o[i] = fmaf(o[i], ga[i], be[i]);
                store_vec<T, V>(y + u * TH * V, o);
            }
        st = st + 1 == depth ? 0 : st + 1;
    }
    drain(B, grp, depth, used, t);
}

// ---------------------------------------------------------------- backward

template <typename T, typename D, int V, int E, bool SUMS>
__global__ void __launch_bounds__(BWD, 1) norm_bwd(const __grid_constant__ NormParams P, int depth, Safe safe) {
    constexpr int U = E / V, E2 = E / 2;
    constexpr bool REG = E <= 16;                     // gamma and the row's values in registers; else gamma from
                                                      // the caches and the row from shared memory again
    extern __shared__ __align__(128) unsigned char dyn[];
    __shared__ Bars B;
    __shared__ float2 red[BWD / 32][2][BWD / 32];
    const int grp = threadIdx.y, t = threadIdx.x, TH = blockDim.x, groups = blockDim.y, hs = P.hs, nv = hs / V;
    const long long stride = (long long)gridDim.x * groups, r0 = (long long)blockIdx.x * groups + grp;
    const int sx = stage_bytes<T>(hs), sb = sx + stage_bytes<D>(hs);
    unsigned char* const ring = dyn + (size_t)grp * depth * sb;
    const Rows<T> X(P.x, P.ldx);
    const Rows<D> Y(P.dy, P.lddy);
    if (t == 0) {
        for (int d = 0; d < depth; ++d) mbar_init(&B.full[grp][d], 1);
        fence_mbar_init_cluster();
    }
    if (t == 0 && grp == 0) B.abort = 0;
    __syncthreads();
    pdl_launch_dependents();
    pdl_wait_primary();
    auto fetch = [&](long long row, int st) {
        if (!safe.has(row)) return;
        fence_async();
        mbar_arrive_expect_tx(&B.full[grp][st], X.bytes(row, hs) + Y.bytes(row, hs));
        X.copy(row, hs, ring + (size_t)st * sb, &B.full[grp][st]);
        Y.copy(row, hs, ring + (size_t)st * sb + sx, &B.full[grp][st]);
    };
    if (t == 0)
        for (int d = 0; d < depth; ++d) fetch(r0 + d * stride, d);
    float nmu = 0.f, nrs = 0.f;
    auto stats = [&](long long row) {
        if (row < P.rows) {
            nmu = P.mu[row];
            nrs = P.rstd[row];
        }
    };
    stats(r0);
    const bool wg = wide_affine(P.gamma, V);
    uint64_t ga[REG ? E2 : 1], ag[E2], ab[E2];
    // gamma's pairs of this thread's vectors from u0 on, as many as g takes
    auto gamma = [&](int u0, auto& g) {
        constexpr int N2 = sizeof(g) / 8;
        float f[2 * N2 / V][V];
#pragma unroll
        for (int u = 0; u < 2 * N2 / V; ++u) {
#pragma unroll
            for (int i = 0; i < V; ++i) f[u][i] = 0.f;
            if (t + (u0 + u) * TH < nv) load_affine<V>(P.gamma, (t + (u0 + u) * TH) * V, wg, 1.f, f[u]);
        }
#pragma unroll
        for (int k = 0; k < N2; ++k) g[k] = pack2(f[2 * k / V][2 * k % V], f[(2 * k + 1) / V][(2 * k + 1) % V]);
    };
    if constexpr (REG) gamma(0, ga);
#pragma unroll
    for (int k = 0; k < E2; ++k) ag[k] = ab[k] = 0;
    const float inv = 1.f / (float)hs;
    int st = 0, par = 0;
    uint32_t used = 0;                                // bit st: the phase of stage st to wait for
    for (long long r = r0; r < P.rows; r += stride, par ^= 1) {
        unsigned char* const stage = ring + (size_t)st * sb;
        const uint64_t nmu2 = both(-nmu), rs2 = both(nrs);
        stats(r + stride);
        if (safe.has(r)) {
            wait_parity<false>(&B.full[grp][st], (used >> st) & 1u, &B.abort, &g_watchdog);
            used ^= 1u << st;
        } else {
            X.copy_by_hand(r, hs, stage, t, TH);
            Y.copy_by_hand(r, hs, stage + sx, t, TH);
            if (TH == 32) __syncwarp();
            else named_sync(1 + grp, TH);
        }
        const T* x = reinterpret_cast<const T*>(stage + X.offset(r)) + t * V;
        const D* dy = reinterpret_cast<const D*>(stage + sx + Y.offset(r)) + t * V;
        // xh and dy of vectors [u0, u0 + NU) of this thread (dy 0 past the row's end)
        constexpr int NU = REG ? U : 16 / V, C2 = NU * V / 2;
        auto row = [&](int u0, uint64_t (&xh)[C2], uint64_t (&d)[C2]) {
            Vec<T, V> rx[NU];
            Vec<D, V> rd[NU];
#pragma unroll
            for (int u = 0; u < NU; ++u) {
                rx[u].zero();
                rd[u].zero();
                if (t + (u0 + u) * TH < nv) {
                    rx[u].load(x + (u0 + u) * TH * V);
                    rd[u].load(dy + (u0 + u) * TH * V);
                }
            }
            to_pairs<T, V, NU>(rx, xh);
            to_pairs<D, V, NU>(rd, d);
#pragma unroll
            for (int k = 0; k < C2; ++k) xh[k] = mul2(add2(xh[k], nmu2), rs2);
        };
        auto scale = [&](int u0, uint64_t (&g)[C2]) {
            if constexpr (REG) {
#pragma unroll
                for (int k = 0; k < C2; ++k) g[k] = mul2(g[k], ga[k]);
            } else {
                uint64_t gg[C2];
                gamma(u0, gg);
#pragma unroll
                for (int k = 0; k < C2; ++k) g[k] = mul2(g[k], gg[k]);
            }
        };
        uint64_t xh[C2], g[C2], s1[2] = {}, s2[2] = {};
#pragma unroll
        for (int u0 = 0; u0 < U; u0 += NU) {
            row(u0, xh, g);
            if (SUMS) {
#pragma unroll
                for (int k = 0; k < C2; ++k) {
                    ag[u0 * V / 2 + k] = fma2(g[k], xh[k], ag[u0 * V / 2 + k]);
                    ab[u0 * V / 2 + k] = add2(g[k], ab[u0 * V / 2 + k]);
                }
            }
            scale(u0, g);
#pragma unroll
            for (int k = 0; k < C2; ++k) {
                s1[k & 1] = add2(s1[k & 1], g[k]);
                s2[k & 1] = fma2(g[k], xh[k], s2[k & 1]);
            }
        }
        const float2 s = group_sum(make_float2(sum2(add2(s1[0], s1[1])), sum2(add2(s2[0], s2[1]))), red[grp][par], TH, 1 + grp);
        if (REG && t == 0) fetch(r + depth * stride, st);     // past the sum: every thread has read its stage
        const uint64_t na = both(-s.x * inv), nc = both(-s.y * inv);
        T* dx = static_cast<T*>(P.y) + r * P.ldy + t * V;
#pragma unroll
        for (int u0 = 0; u0 < U; u0 += NU) {
            if (!REG) {
                row(u0, xh, g);
                scale(u0, g);
            }
#pragma unroll
            for (int k = 0; k < C2; ++k) g[k] = mul2(fma2(xh[k], nc, add2(g[k], na)), rs2);
#pragma unroll
            for (int u = 0; u < NU; ++u)
                if (t + (u0 + u) * TH < nv) {
                    float o[V];
                    from_pairs<T, V, NU>(g, u, o);
                    store_vec<T, V>(dx + (u0 + u) * TH * V, o);
                }
        }
        if (!REG) {
            if (TH == 32) __syncwarp();
            else named_sync(1 + grp, TH);
            if (t == 0) fetch(r + depth * stride, st);
        }
        st = st + 1 == depth ? 0 : st + 1;
    }
    drain(B, grp, depth, used, t);
    if (!SUMS) return;
    // the CTA's column sums: the groups' in order (in shared memory), then to the workspace
    float* const cols = reinterpret_cast<float*>(dyn);
    float* const out = P.part + (long long)blockIdx.x * 2 * hs;
    for (int k = 0; k < groups; ++k) {
        if (groups > 1) __syncthreads();
        if (grp == k)
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (t + u * TH < nv) {
                    float a[V], b[V];
                    from_pairs<T, V, U>(ag, u, a);
                    from_pairs<T, V, U>(ab, u, b);
                    float* to = k + 1 < groups ? cols : out;
#pragma unroll
                    for (int i = 0; i < V; ++i) {
                        const int j = (t + u * TH) * V + i;
                        to[j] = k > 0 ? a[i] + cols[j] : a[i];
                        to[hs + j] = k > 0 ? b[i] + cols[hs + j] : b[i];
                    }
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

// Elements of a vector: bytes of x `vb` (16, 2 elements or 1) that every row start of every
// operand allows.
bool aligned(const void* p, long long ld, int es, int bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && ld * es % bytes == 0;
}

// Threads a row (E elements each) and rows a CTA of `threads` threads.
struct Shape {
    int E, TH, groups;
};

Shape shape_of(int hs, int threads, int E) {
    Shape s;
    s.E = E;
    s.TH = ((hs + E - 1) / E + 31) / 32 * 32;
    s.groups = threads / s.TH;
    if (s.TH > 32 && s.groups > 15) s.groups = 15;      // named barriers 1 .. 15
    return s;
}

// Backward: 16 elements a thread in all rows that 512 threads hold so (with 32 the column sums fill
// the registers): 2048 x 4096 bf16 23 us, with 32 35.
Shape bwd_shape(int hs) { return shape_of(hs, BWD, hs <= 16 * BWD ? 16 : 32); }

int depth_of(int groups, int stage, int ring) {
    const int d = ring / (groups * stage);
    return d < 1 ? 1 : d > MAXD ? MAXD : d;
}

// The rows of a matrix that bulk copies of whole 16-byte blocks may take.
Safe safe_rows(const void* p, long long ld, int es, long long rows, int hs) {
    const uintptr_t base = reinterpret_cast<uintptr_t>(p), end = base + (uintptr_t)(((rows - 1) * ld + hs) * es);
    Safe s{0, rows};
    while (s.lo < rows && ((base + (uintptr_t)(s.lo * ld * es)) & ~uintptr_t(15)) < base) ++s.lo;
    while (s.hi > s.lo && ((base + (uintptr_t)(((s.hi - 1) * ld + hs) * es) + 15) & ~uintptr_t(15)) > end) --s.hi;
    return s;
}

// The kernel may use smem bytes of shared memory: asked for when a call needs more than any before
// it on the device.
template <typename F>
cudaError_t opt_in(F kernel, size_t smem, std::atomic<int> (&had)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (had[dev].load(std::memory_order_acquire) >= (int)smem) return cudaSuccess;
    e = cudaFuncSetAttribute((const void*)kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024 - 24 * 1024);
    if (e == cudaSuccess) had[dev].store(227 * 1024 - 24 * 1024, std::memory_order_release);
    return e;
}

template <typename T, int V, int E>
cudaError_t fwd_go(const NormParams& P, Shape s, cudaStream_t st) {
    const int stage = stage_bytes<T>(P.hs), affine = (8 * P.hs + 15) / 16 * 16;
    while (s.groups > 1 && s.groups * stage + affine > RING_B) --s.groups;
    const int depth = depth_of(s.groups, stage, RING_B - affine);
    const size_t smem = (size_t)s.groups * depth * stage + affine;
    static std::atomic<int> had[64];
    const cudaError_t e = opt_in(norm_fwd<T, V, E>, smem, had);
    if (e != cudaSuccess) return e;
    const long long want = (P.rows + s.groups - 1) / s.groups, sms = num_sms();
    return launch_pdl(norm_fwd<T, V, E>, want < sms ? want : sms, dim3(s.TH, s.groups), smem, st, P, depth,
                      safe_rows(P.x, P.ldx, sizeof(T), P.rows, P.hs));
}

template <typename T, int V>
cudaError_t fwd_e(const NormParams& P, cudaStream_t st) {
    // Fewer threads a row meet less at its sums: 16384 x 512 bf16 12.3 us with 16 elements each and 14.1
    // with 32, 16384 x 4096 70 and 50.  64 pay in bf16 rows of 2048 to 8192 that fill their warps:
    // 16384 x 2048 26.4 us against 29.3 with 32, x 4096 47.8 and 50.3, 8192 x 8192 46.1 and 52.4 (4096 x
    // 12288 43.1 and 42.2; fp32 the same within 2%).
    if (P.hs <= 512) return fwd_go<T, V, 16>(P, shape_of(P.hs, FWD, 16), st);
    if constexpr (sizeof(T) == 2 && V == 8) {
        const Shape s = shape_of(P.hs, FWD64, 64);
        if (P.hs >= 2048 && P.hs <= 8192 && 64 * s.TH - P.hs <= P.hs / 4) return fwd_go<T, V, 64>(P, s, st);
    }
    // 24 where they need no more threads than 32: 16384 x 2304 bf16 34.1 us against 36.1, x 768 15.6 and 16.6,
    // 3001 x 2050 fp32 16.4 and 17.0.
    const Shape s = shape_of(P.hs, FWD, 24);
    if (s.TH == shape_of(P.hs, FWD, 32).TH) return fwd_go<T, V, 24>(P, s, st);
    return fwd_go<T, V, 32>(P, shape_of(P.hs, FWD, 32), st);
}

template <typename T>
cudaError_t fwd(const NormParams& P, cudaStream_t st) {
    constexpr int N = Pack<T>::N, es = sizeof(T);
    auto ok = [&](int n) {
        return P.hs % n == 0 && aligned(P.x, P.ldx, es, n * es) && aligned(P.y, P.ldy, es, n * es);
    };
    if (ok(N)) {
        // Few rows: a row a CTA (8 x 4096 bf16 2.1 us a call in a graph against 5.2 by the ring, 608 x
        // 1024 2.1 and 4.9, 608 x 4096 5.6 and 6.8, fp32 7.6 and 8.1).
        const int nv = P.hs / N;
        if (P.rows <= 4 * num_sms() && nv <= 4 * FEW) {
            const int C = nv <= FEW ? 1 : nv <= 2 * FEW ? 2 : 4;
            const dim3 threads(((nv + C - 1) / C + 31) / 32 * 32);
            if (C == 1) return launch_pdl(norm_fwd_few<T, N, 1>, P.rows, threads, 0, st, P);
            if (C == 2) return launch_pdl(norm_fwd_few<T, N, 2>, P.rows, threads, 0, st, P);
            return launch_pdl(norm_fwd_few<T, N, 4>, P.rows, threads, 0, st, P);
        }
        return fwd_e<T, N>(P, st);
    }
    if (ok(2)) return fwd_e<T, 2>(P, st);
    return fwd_e<T, 1>(P, st);
}

template <typename T, typename D, int V, int E>
cudaError_t bwd_go(const NormParams& P, const Shape& s, cudaStream_t st) {
    const bool sums = P.dgamma || P.dbeta;
    long long grid = (P.rows + s.groups - 1) / s.groups;
    const int sms = num_sms(), most = sms < kMaxParts ? sms : kMaxParts;
    if (grid > most) grid = most;
    const int stage = stage_bytes<T>(P.hs) + stage_bytes<D>(P.hs), depth = depth_of(s.groups, stage, RING_B);
    const size_t ring = (size_t)s.groups * depth * stage, meet = 8 * (size_t)P.hs, smem = ring > meet ? ring : meet;
    static std::atomic<int> had[2][64];
    cudaError_t e = sums ? opt_in(norm_bwd<T, D, V, E, true>, smem, had[1]) : opt_in(norm_bwd<T, D, V, E, false>, smem, had[0]);
    if (e != cudaSuccess) return e;
    const Safe a = safe_rows(P.x, P.ldx, sizeof(T), P.rows, P.hs), b = safe_rows(P.dy, P.lddy, sizeof(D), P.rows, P.hs);
    const Safe safe{a.lo > b.lo ? a.lo : b.lo, a.hi < b.hi ? a.hi : b.hi};
    e = sums ? launch_pdl(norm_bwd<T, D, V, E, true>, grid, dim3(s.TH, s.groups), smem, st, P, depth, safe)
             : launch_pdl(norm_bwd<T, D, V, E, false>, grid, dim3(s.TH, s.groups), smem, st, P, depth, safe);
    if (e == cudaSuccess && sums) e = launch_pdl(norm_join, (2 * P.hs + 31) / 32, dim3(256), 0, st, P, (int)grid);
    return e;
}

template <typename T, typename D, int V>
cudaError_t bwd_e(const NormParams& P, cudaStream_t st) {
    const Shape s = bwd_shape(P.hs);
    return s.E == 16 ? bwd_go<T, D, V, 16>(P, s, st) : bwd_go<T, D, V, 32>(P, s, st);
}

template <typename T, typename D>
cudaError_t bwd(const NormParams& P, cudaStream_t st) {
    constexpr int N = 16 / (sizeof(T) > sizeof(D) ? sizeof(T) : sizeof(D)), es = sizeof(T), ds = sizeof(D);
    if (P.rows == 0) return launch_pdl(norm_join, (2 * P.hs + 31) / 32, dim3(256), 0, st, P, 0);
    auto ok = [&](int n) {
        return P.hs % n == 0 && aligned(P.x, P.ldx, es, n * es) && aligned(P.y, P.ldy, es, n * es) &&
               aligned(P.dy, P.lddy, ds, n * ds);
    };
    if (ok(N)) return bwd_e<T, D, N>(P, st);
    if (ok(2)) return bwd_e<T, D, 2>(P, st);
    return bwd_e<T, D, 1>(P, st);
}

}  // namespace

long long norm_bwd_ws_bytes(long long rows, long long hs) {
    const Shape s = bwd_shape((int)hs);
    const long long want = (rows + s.groups - 1) / s.groups;
    return (want < kMaxParts ? want : kMaxParts) * 2 * hs * 4;
}

unsigned int norm_watchdog(bool clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_watchdog, sizeof(v)) != cudaSuccess) return 0xffffffffu;
    if (clear && v) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_watchdog, &z, sizeof(z)) != cudaSuccess) return 0xffffffffu;
    }
    return v;
}

cudaError_t launch_norm_fwd(const NormParams& P, cudaStream_t st) {
    return P.dtype == kBf16 ? fwd<__nv_bfloat16>(P, st) : fwd<float>(P, st);
}

cudaError_t launch_norm_bwd(const NormParams& P, cudaStream_t st) {
    if (P.dtype != kBf16) return bwd<float, float>(P, st);
    return P.dy_f32 ? bwd<__nv_bfloat16, float>(P, st) : bwd<__nv_bfloat16, __nv_bfloat16>(P, st);
}

}  // namespace vl
