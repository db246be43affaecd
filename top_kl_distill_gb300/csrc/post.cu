// Post-training losses over rows of vocabulary logits: the clipped policy loss with a KL term,
// and the preference loss over pairs of sequences, each with the gradient of the logits.
//
// Both need, of a row s with picked column a, m = max s, lnS = ln sum exp(s - m) and
// logp = (s[a] - m) - lnS, then a factor G = d loss / d logp, and write
// scale G ([j == a] - exp(s_j - m - lnS)).  In the policy loss G follows from the row alone;
// in the preference loss from every row of the row's pair, so its rows are read twice.
#include "vl_device.cuh"
#include "vl_internal.h"
#include "vl_rowio.cuh"
#include "vloss.h"

#include <cmath>

namespace vl {
namespace {

constexpr int NT = 512;                  // threads of a row's CTA
// What the first pass leaves as the factor of a row with a bad label: a zero (its gradient row
// is zero whether or not a sequence holds it) that the pair kernel can tell from the others'.
constexpr float kBadLabel = -0.f;

// What a row's G and losses are made of (policy).
struct Outcome {
    float G, loss, kl;
};

// The losses of one token.  Comparisons are arranged so that a NaN stays a NaN.
__device__ __forceinline__ Outcome policy_outcome(const PostParams& P, long long r, float w, float logp) {
    const float A = P.adv[r];
    const float ratio = expf(logp - P.old_logp[r]);
    const float f = ratio * A;
    const float h = (ratio < P.lo ? P.lo : ratio > P.hi ? P.hi : ratio) * A;
    const bool capped = f > h;
    Outcome o;
    float each = capped ? -h : -f;
    float d = capped ? 0.f : -f;
    o.kl = 0.f;
    if (P.ref_logp) {
        const float q = P.ref_logp[r] - logp;
        const float e1 = expm1f(q);
        o.kl = q > 80.f ? e1 : e1 - q;              // the same in fp32, and no inf - inf
        if (P.kl_coef != 0.f) {
            each += P.kl_coef * o.kl;
            d -= P.kl_coef * e1;
        }
    }
    o.loss = w * each;
    o.G = w * d;
    return o;
}

// One CTA a row: (max, sum) over the row, its outcome, then the gradient over a second read.
enum Mode : int { kPolicy = 0, kLogp = 1, kGrad = 2 };

template <typename T, int MODE>
__global__ void __launch_bounds__(NT) post_rows(const __grid_constant__ PostParams P) {
    __shared__ float2 part[NT / 32];
    __shared__ float3 bc;
    const int ct = threadIdx.x, n = (int)P.V;
    pdl_wait_primary();
    pdl_launch_dependents();
    for (long long r = blockIdx.x; r < P.ntok; r += gridDim.x) {
        const T* x = static_cast<const T*>(P.x) + r * P.ld;
        T* g = P.g ? static_cast<T*>(P.g) + r * P.ldg : nullptr;
        const float w = P.weight[r];
        const uint32_t a = P.label[r];
        const bool bad = (long long)a >= P.V;
        float m = 0.f, lnS = 0.f, c = 0.f;
        if (MODE != kGrad) {
            if (w == 0.f || bad) {
                if (ct == 0) {
                    const float miss = w != 0.f ? __int_as_float(0x7fc00000) : 0.f;
                    if (MODE == kPolicy) {
                        P.loss[r] = miss;
                        if (P.logp) P.logp[r] = miss;
                        if (P.kl) P.kl[r] = 0.f;
                    } else {
                        P.logp[r] = miss;
                        P.coef[r] = w != 0.f ? kBadLabel : 0.f;
                    }
                    if (w != 0.f && P.err) atomicAdd(P.err, 1);
                }
            } else {
                const float sa = ld_elem(x + a);
                MaxSum ms = row_max_sum<T, NT>(x, n, ct);
                ms = ms_warp_reduce(ms);
                if ((ct & 31) == 0) part[ct >> 5] = make_float2(ms.m, ms.s);
                __syncthreads();
                if (ct == 0) {
                    float M = part[0].x, S = 0.f;
                    for (int i = 1; i < NT / 32; ++i) M = fmaxf(M, part[i].x);
                    for (int i = 0; i < NT / 32; ++i) S += part[i].y * ex2((part[i].x - M) * kLog2e);
                    const float l = logf(S), logp = (sa - M) - l;
                    float G = 0.f;
                    if (MODE == kPolicy) {
                        const Outcome o = policy_outcome(P, r, w, logp);
                        G = P.scale * o.G;
                        P.loss[r] = o.loss;
                        if (P.logp) P.logp[r] = logp;
                        if (P.kl) P.kl[r] = o.kl;
                    } else {
                        P.logp[r] = logp;
                        P.coef[r] = 0.f;
                        P.stats[2 * r] = M;
                        P.stats[2 * r + 1] = l;
                    }
                    bc = make_float3(M, l, G);
                }
                __syncthreads();
                m = bc.x;
                lnS = bc.y;
                c = bc.z;
                __syncthreads();
            }
        } else {
            c = P.coef[r];
            if (c != 0.f) {
                m = P.stats[2 * r];
                lnS = P.stats[2 * r + 1];
            }
        }
        if (MODE != kLogp && g) row_gradient<T, NT>(x, g, n, ct, m, lnS, c, (int)a);
    }
}

// One CTA a pair: both sequences' sums in 64 bits, the pair's loss, and each row's factor.
constexpr int PT = 256;

__device__ double cta_sum(double v, double* red) {
    const int t = threadIdx.x;
    red[t] = v;
    __syncthreads();
    for (int off = PT / 2; off > 0; off >>= 1) {
        if (t < off) red[t] += red[t + off];
        __syncthreads();
    }
    const double s = red[0];
    __syncthreads();
    return s;
}

__device__ __forceinline__ float softplus(float v) {       // ln(1 + e^v)
    return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
}

__global__ void __launch_bounds__(PT) pair_kernel(const __grid_constant__ PairParams Q) {
    __shared__ double red[PT];
    pdl_wait_primary();
    pdl_launch_dependents();
    for (long long i = blockIdx.x; i < Q.npairs; i += gridDim.x) {
        long long lo[2], hi[2];
        double sum[2];
        int bad = 0;
        for (int k = 0; k < 2; ++k) {
            const long long s = i + (k ? Q.npairs : 0);
            lo[k] = min(max(Q.start[s], 0ll), Q.ntok);
            hi[k] = min(max(Q.start[s + 1], lo[k]), Q.ntok);
            double v = 0.0;
            for (long long t = lo[k] + threadIdx.x; t < hi[k]; t += PT) {
                const float w = Q.weight[t];
                if (w == 0.f) continue;
                if (signbit(Q.coef[t])) bad = 1;
                v += (double)w * (double)Q.logp[t];
            }
            sum[k] = cta_sum(v, red);
        }
        bad = __syncthreads_or(bad);
        const double gap = (sum[0] - (Q.ref ? (double)Q.ref[i] : 0.0)) - (sum[1] - (Q.ref ? (double)Q.ref[Q.npairs + i] : 0.0));
        const float h = (float)((double)Q.beta * gap);
        float loss, d;                              // d loss / d gap
        if (Q.kind == VL_PREF_SIGMOID) {
            loss = (1.f - Q.smooth) * softplus(-h) + Q.smooth * softplus(h);
            // sigmoid(h) - (1 - smooth), each tail from the side that does not cancel
            const float e = expf(-fabsf(h)), small = e / (1.f + e);
            d = Q.beta * (h >= 0.f ? Q.smooth - small : small - (1.f - Q.smooth));
        } else if (Q.kind == VL_PREF_IPO) {
            const float z = (float)(gap - 0.5 / (double)Q.beta);
            loss = z * z;
            d = 2.f * z;
        } else {
            loss = h < 1.f ? 1.f - h : h >= 1.f ? 0.f : h;    // a NaN stays one
            d = h < 1.f ? -Q.beta : h >= 1.f ? 0.f : h;
        }
        if (threadIdx.x == 0) {
            Q.loss[i] = loss;
            Q.margin[i] = h;
            if (Q.seq) {
                Q.seq[i] = (float)sum[0];
                Q.seq[Q.npairs + i] = (float)sum[1];
            }
        }
        for (int k = 0; k < 2; ++k)
            for (long long t = lo[k] + threadIdx.x; t < hi[k]; t += PT) {
                const float w = Q.weight[t];
                Q.coef[t] = bad || w == 0.f ? 0.f : Q.scale * (k ? -d : d) * w;
            }
        __syncthreads();
    }
}

// The sum of n losses, in 64 bits and a fixed order.
__global__ void __launch_bounds__(1024) total_kernel(const float* loss, long long n, float* total) {
    __shared__ double red[32];
    pdl_wait_primary();
    pdl_launch_dependents();
    double v = 0.0;
    for (long long i = threadIdx.x; i < n; i += 1024) v += (double)loss[i];
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    if (threadIdx.x < 32) {
        v = red[threadIdx.x];
        for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
        if (threadIdx.x == 0) *total = (float)v;
    }
}

template <typename K, typename... Args>
cudaError_t launch_pdl(K kernel, long long grid, int threads, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <int MODE>
cudaError_t launch_post(const PostParams& P, cudaStream_t st) {
    const long long grid = P.ntok < 65536 ? P.ntok : 65536;
    if (P.dtype == kBf16) return launch_pdl(post_rows<__nv_bfloat16, MODE>, grid, NT, st, P);
    return launch_pdl(post_rows<float, MODE>, grid, NT, st, P);
}

}  // namespace

cudaError_t launch_policy(const PostParams& P, float* total, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (P.ntok > 0) e = launch_post<kPolicy>(P, st);
    if (e == cudaSuccess && total) e = launch_pdl(total_kernel, 1, 1024, st, (const float*)P.loss, P.ntok, total);
    return e;
}

cudaError_t launch_preference(const PostParams& P, const PairParams& Q, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (P.ntok > 0) e = launch_post<kLogp>(P, st);
    if (e == cudaSuccess && Q.npairs > 0)
        e = launch_pdl(pair_kernel, Q.npairs < 65536 ? Q.npairs : 65536, PT, st, Q);
    if (e == cudaSuccess && P.ntok > 0 && P.g) e = launch_post<kGrad>(P, st);
    return e;
}

}  // namespace vl
