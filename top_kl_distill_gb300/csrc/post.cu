// Post-training losses over rows of vocabulary logits: the clipped policy loss with a KL term,
// and the preference loss over pairs of sequences, each with the gradient of the logits.
//
// Both need, of a row s with picked column a, m = max s, lnS = ln sum exp(s - m) and
// logp = (s[a] - m) - lnS, then a factor c = scale d loss / d logp, and write
// c ([j == a] - exp(s_j - m - lnS)).  In the policy loss c follows from the row alone; in the
// preference loss from every row of the row's pair, so its rows are read twice: a pass for the
// log-probabilities (kLogp), a kernel over the pairs, a pass for the gradient (kGrad).
//
// HBM bound: a row is read once and its gradient written once, 8 V bytes fp32.  The policy pass
// keeps a row on chip between the two: each thread holds the exponentials of its 64 columns,
// exp(s - mt) with mt its own running maximum at that tile, in registers while the row's
// statistics meet; the gradient is then one multiplication a column by
// -c exp(mt - m - lnS), with no second read and no second exponential.
//
//   long rows    (rows_ring) one persistent CTA per SM, consumer warps and a producer warp: a
//                ring of six 30 KB tiles of 1-D bulk copies runs ahead of the consumers, so
//                the reads go on while a row's statistics meet and its gradient is written.
//                What a row has beyond the registers (30720 columns) stays in the ring, up to
//                two tiles.  Longer rows, and rows too few for the SMs, are split over a cluster;
//                every warp sends its partial (max, sum) to every rank with st.async.
//   short rows   (rows_direct, up to 8192 columns) a CTA of 128 or 256 threads a row, loaded straight
//                into registers; several CTAs an SM overlap each other's phases.  A short row in the
//                ring kernel would leave most of its threads idle and pay a barrier a row.
//   beyond       (rows_twice) rows of more than VL_POLICY_ONEPASS_COLS columns are read twice.
//
// The producer warp also fetches each row's token data (weight, column, its logit, ...), 32 rows
// at a time, so that no consumer waits on a chain of global loads; rows that do not count are
// not read, their gradient rows are zeroed.
#include "vl_device.cuh"
#include "vl_internal.h"
#include "vl_launch.h"
#include "vl_pair.cuh"
#include "vl_rowio.cuh"
#include "vloss.h"

#include <atomic>
#include <cmath>

namespace vl {
namespace {

constexpr int NT = 512;                  // threads of a CTA of rows_twice
// What the first pass leaves as the factor of a row with a bad label: a zero (its gradient row
// is zero whether or not a sequence holds it) that the pair kernel can tell from the others'.
constexpr float kBadLabel = -0.f;

// What a row's G and losses are made of (policy).
struct Outcome {
    float G, loss, kl;
};

// The losses of one token.  Comparisons are arranged so that a NaN stays a NaN.
__device__ __forceinline__ Outcome policy_outcome(const PostParams& P, float w, float old, float ref, float A, float logp) {
    const float e0 = expf(logp - old);
    const float ratio = A == 0.f && isinf(e0) ? 1.f : e0;      // no advantage: 0 however far the ratio went, not 0 inf
    const float f = ratio * A;
    const float h = (ratio < P.lo ? P.lo : ratio > P.hi ? P.hi : ratio) * A;
    const bool capped = f > h;
    Outcome o;
    float each = capped ? -h : -f;
    float d = capped ? 0.f : -f;
    o.kl = 0.f;
    if (P.ref_logp) {
        const float q = ref - logp;
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

enum Mode : int { kPolicy = 0, kLogp = 1, kGrad = 2 };

// What one thread of a row writes besides the gradient; returns the gradient's factor c.
template <int MODE>
__device__ __forceinline__ float settle_row(const PostParams& P, long long r, float w, float old, float ref, float adv,
                                            float xa, float m, float lnS, bool writer) {
    const float logp = (xa - m) - lnS;
    if (MODE == kLogp) {
        if (writer) {
            P.logp[r] = logp;
            P.coef[r] = 0.f;
            P.stats[2 * r] = m;
            P.stats[2 * r + 1] = lnS;
        }
        return 0.f;
    }
    const Outcome o = policy_outcome(P, w, old, ref, adv, logp);
    if (writer) {
        P.loss[r] = o.loss;
        if (P.logp) P.logp[r] = logp;
        if (P.kl) P.kl[r] = o.kl;
    }
    return P.scale * o.G;
}

// A row that does not count (weight 0), or whose column is out of range.
template <int MODE>
__device__ __forceinline__ void skip_row(const PostParams& P, long long r, float w) {
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

// (max, sum) of n <= 256 partials, by one warp: every lane gets the same bits.
__device__ __forceinline__ MaxSum combine_parts(const float2* part, int n, int lane) {
    float M = -FLT_MAX;
    for (int j = lane; j < n; j += 32) M = fmaxf(M, part[j].x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float T = 0.f;
    for (int j = lane; j < n; j += 32) T += part[j].y * ex2((part[j].x - M) * kLog2e);
    return MaxSum{M, warp_sum(T)};
}

// ---------------------------------------------------------------- rows read twice

template <typename T>
__global__ void __launch_bounds__(NT) rows_twice(const __grid_constant__ PostParams P) {
    __shared__ float2 part[NT / 32];
    const int ct = threadIdx.x, n = (int)P.V;
    pdl_launch_dependents();
    pdl_wait_primary();
    for (long long r = blockIdx.x; r < P.ntok; r += gridDim.x) {
        const T* x = static_cast<const T*>(P.x) + r * P.ld;
        T* g = P.g ? static_cast<T*>(P.g) + r * P.ldg : nullptr;
        const float w = P.weight[r];
        const uint32_t a = P.label[r];
        float m = 0.f, lnS = 0.f, c = 0.f;
        if (w == 0.f || (long long)a >= P.V) {
            if (ct == 0) skip_row<kPolicy>(P, r, w);
        } else {
            const float xa = ld_elem(x + a);
            const MaxSum ms = ms_warp_reduce(row_max_sum<T, NT>(x, n, ct));
            if ((ct & 31) == 0) part[ct >> 5] = make_float2(ms.m, ms.s);
            __syncthreads();
            const MaxSum tot = combine_parts(part, NT / 32, ct & 31);
            m = tot.m;
            lnS = logf(tot.s);
            c = settle_row<kPolicy>(P, r, w, P.old_logp[r], P.ref_logp ? P.ref_logp[r] : 0.f, P.adv[r], xa, m, lnS, ct == 0);
        }
        if (g) row_gradient<T, NT>(x, g, n, ct, m, lnS, c, (int)a);
        __syncthreads();
    }
}

// ---------------------------------------------------------------- short rows

// DT threads, CH 16-byte chunks a thread: rows of up to DT * CH chunks.
template <typename T, int MODE, int DT, int CH>
__global__ void __launch_bounds__(DT) rows_direct(const __grid_constant__ PostParams P) {
    constexpr int N = Pack<T>::N;
    __shared__ float2 part[2][DT / 32];
    const int ct = threadIdx.x, lane = ct & 31, n = (int)P.V;
    uint32_t li = 0;
    pdl_launch_dependents();
    pdl_wait_primary();
    for (long long i = blockIdx.x; i < P.ntok; i += gridDim.x) {
        const long long r = MODE == kGrad ? P.ntok - 1 - i : i;       // the last rows read are still in L2
        const T* x = static_cast<const T*>(P.x) + r * P.ld;
        T* g = P.g ? static_cast<T*>(P.g) + r * P.ldg : nullptr;
        const uint32_t a = P.label[r];
        const float w = MODE == kGrad ? P.coef[r] : P.weight[r];
        const bool live = w != 0.f && (MODE == kGrad || (long long)a < P.V);
        const int h = head_len(x, n), nb = (n - h) / N, t0 = h + nb * N;
        // head and tail columns: one a thread (head columns first)
        const int jht = ct < h ? ct : ct >= N && t0 + ct - N < n ? t0 + ct - N : -1;
        float v[CH][N], ht = 0.f, m = 0.f, lnS = 0.f, c = w;
        MaxSum ms = ms_empty();
        if (live) {
            const uint4* x4 = reinterpret_cast<const uint4*>(x + h);
            uint4 raw[CH];
#pragma unroll
            for (int u = 0; u < CH; ++u)
                if (u * DT + ct < nb) raw[u] = x4[u * DT + ct];
            ht = jht >= 0 ? ld_elem(x + jht) : 0.f;
            if (MODE == kGrad) {
                m = P.stats[2 * r];
                lnS = P.stats[2 * r + 1];
#pragma unroll
                for (int u = 0; u < CH; ++u)
                    if (u * DT + ct < nb) {
                        Pack<T>::unpack(raw[u], v[u]);
#pragma unroll
                        for (int k = 0; k < N; ++k) v[u][k] = ex2(((v[u][k] - m) - lnS) * kLog2e);
                    }
            } else {
                const float xa = ld_elem(x + a);
                const float old = MODE == kPolicy ? P.old_logp[r] : 0.f, adv = MODE == kPolicy ? P.adv[r] : 0.f;
                const float ref = MODE == kPolicy && P.ref_logp ? P.ref_logp[r] : 0.f;
#pragma unroll
                for (int u = 0; u < CH; ++u)
                    if (u * DT + ct < nb) {
                        Pack<T>::unpack(raw[u], v[u]);
#pragma unroll
                        for (int k = 0; k < N; ++k) ms.m = fmaxf(ms.m, v[u][k]);
                    }
                if (jht >= 0) ms.m = fmaxf(ms.m, ht);
#pragma unroll
                for (int u = 0; u < CH; ++u)
                    if (u * DT + ct < nb) {
                        float e = 0.f;
#pragma unroll
                        for (int k = 0; k < N; ++k) {
                            v[u][k] = ex2((v[u][k] - ms.m) * kLog2e);
                            e += v[u][k];
                        }
                        ms.s += e;
                    }
                if (jht >= 0) ms.s += ex2((ht - ms.m) * kLog2e);
                const MaxSum wm = ms_warp_reduce(ms);
                if (lane == 0) part[li & 1][ct >> 5] = make_float2(wm.m, wm.s);
                __syncthreads();
                const MaxSum tot = combine_parts(part[li & 1], DT / 32, lane);
                ++li;
                m = tot.m;
                lnS = logf(tot.s);
                c = settle_row<MODE>(P, r, w, old, ref, adv, xa, m, lnS, ct == 0);
            }
        } else {
            if (MODE != kGrad && ct == 0) skip_row<MODE>(P, r, w);
            c = 0.f;
        }
        if (MODE == kLogp || !g) continue;
        const float f = c == 0.f ? 0.f : MODE == kGrad ? -c : -c * ex2(((ms.m - m) - lnS) * kLog2e);
        const bool wide = ((reinterpret_cast<uintptr_t>(g + h)) & 15u) == 0;
#pragma unroll
        for (int u = 0; u < CH; ++u)
            if (u * DT + ct < nb) {
                const int j = h + (u * DT + ct) * N;
                float o[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    o[k] = c == 0.f ? 0.f : f * v[u][k];
                    if (j + k == (int)a) o[k] += c;
                }
                if (wide) {
                    *reinterpret_cast<uint4*>(g + j) = Pack<T>::pack(o);
                } else {
#pragma unroll
                    for (int k = 0; k < N; ++k) st_elem(g + j + k, o[k]);
                }
            }
        if (jht >= 0) {
            float o = c == 0.f ? 0.f : -c * ex2(((ht - m) - lnS) * kLog2e);
            if (jht == (int)a) o += c;
            st_elem(g + jht, o);
        }
    }
}

// ---------------------------------------------------------------- long rows

constexpr int CW = 15;                   // consumer warps (with the producer 16: up to 128 registers a thread)
constexpr int CT = CW * 32;
constexpr int RT = CT + 32;              // + the producer warp
constexpr int CHT = 4;                   // 16-byte chunks of a tile per consumer thread
constexpr int TILE_B = CT * CHT * 16;    // 30 KB
constexpr int SLOTS = 6;
constexpr int REGV = 64;                 // exponentials a thread holds in registers
constexpr int HOLD = 2;                  // tiles of a row that stay in the ring until its gradient is written
constexpr int MAXC = 8;                  // CTAs a row
constexpr long long kKeepBytes = 64ll << 20;   // 0: 105.6 us at 8 pairs of 32000 columns, 40 MB 105.6, 64 MB 103.2, 90 MB 103.0
constexpr int BATCH = 32;                // rows whose token data the producer fetches at once
constexpr int kWindow = 96;              // rows a cluster takes of one window of the rows
static_assert(kWindow * 256 <= 64 * RT - RT, "deal(): a lane's flags of a window of 256 clusters");
// Buffers of the warps' partials.  Warp 0 settles a row while the others go on; they get no
// further than the ring lets them (a slot is refilled only when warp 0 too has read it), so at
// most SLOTS rows of one tile, and over a cluster one row more.
constexpr int NB = 8;
static_assert(NB > SLOTS + 1, "a partial is read before its buffer comes round again");

__device__ unsigned int g_watchdog;

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float warp_max(float a) {
    float d;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(a));
    return d;
}
__device__ __forceinline__ MaxSum warp_max_sum(MaxSum a) {
    const float M = warp_max(a.m);
    return MaxSum{M, warp_sum(a.s * ex2((a.m - M) * kLog2e))};
}

// The elements of a 16-byte chunk, two to a word.
template <typename T>
__device__ __forceinline__ void unpack_pairs(uint4 r, uint64_t (&v)[Pack<T>::N / 2]) {
    if constexpr (sizeof(T) == 4) {
        v[0] = pack2(__uint_as_float(r.x), __uint_as_float(r.y));
        v[1] = pack2(__uint_as_float(r.z), __uint_as_float(r.w));
    } else {
        const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = pack2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
}

// 16 bytes of shared memory where `p`, else 4 words `fill`; 16 bytes to global memory where `p`.
// Predicated instructions: a branch around each chunk would keep the chunks' latencies apart.
__device__ __forceinline__ uint4 ld_shared_if(uint32_t addr, bool p, uint32_t fill) {
    uint4 r = make_uint4(fill, fill, fill, fill);
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t@q ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
                 : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w) : "r"(addr), "r"((uint32_t)p));
    return r;
}
__device__ __forceinline__ void st_global_if(void* at, uint4 v, bool p, uint64_t policy) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t@q st.global.L2::cache_hint.v4.u32 [%0], {%1, %2, %3, %4}, %6;\n\t}"
                 :: "l"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"((uint32_t)p), "l"(policy) : "memory");
}
__device__ __forceinline__ void st_global_if(void* at, uint4 v, bool p) {
    asm volatile("{\n\t.reg .pred q;\n\tsetp.ne.u32 q, %5, 0;\n\t@q st.global.v4.u32 [%0], {%1, %2, %3, %4};\n\t}"
                 :: "l"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"((uint32_t)p) : "memory");
}

// exp(v - m) of both lanes, nm = -m twice: the difference is exact where it matters (near 0).
__device__ __forceinline__ uint64_t exp_pair(uint64_t v, uint64_t nm, uint64_t l2e) {
    float a, b;
    unpack2(mul2(add2(v, nm), l2e), a, b);
    return pack2(ex2(a), ex2(b));
}

struct Meta {
    float w;                             // weight (kGrad: the factor)
    uint32_t a;
    float xa;                            // the picked logit (kGrad: m)
    float old;                           // (kGrad: lnS)
    float ref, adv;                      // (kGrad: ref holds the picked logit)
    int live;
};

struct alignas(128) RSmem {
    alignas(16) unsigned char ring[SLOTS][TILE_B];
    uint64_t full[SLOTS], empty[SLOTS];
    uint64_t mfull[2], mempty[2];
    uint64_t pbar[NB];                   // every warp's partial of a row is in
    float2 part[NB][MAXC * CW];          // over a cluster: from every rank
    float4 row[2];                       // (m, lnS, c, the picked column's gradient), from the warp that settles the row
    int picked[2];                       // the picked column, -1 where the gradient row is zero
    Meta meta[2][BATCH];
    int list[kWindow + 1];                      // this cluster's rows of the window (from its start): the counting ones first
    int wlive[32];
    int abort;
};
static_assert(sizeof(RSmem) <= 227 * 1024, "shared memory of one CTA");
// Columns of a row part that the policy pass keeps on chip (less a chunk for the split's rounding).
template <typename T>
constexpr int kPartCols = CT * REGV + HOLD * TILE_B / (int)sizeof(T) - 16;
static_assert((long long)kPartCols<float> * MAXC >= VL_POLICY_ONEPASS_COLS, "the header's one-pass limit");
static_assert(HOLD + 2 <= SLOTS, "a held row leaves room for the next one's tiles");

// Columns of a row that CTA `rank` of c takes: a share of the 16-byte-aligned body; rank 0
// also the head before it, the last rank the tail.
struct Part {
    int b0, bn;      // body
    int hn;          // head columns [0, hn)
    int t0, tn;      // tail columns
};

template <typename T>
__device__ __forceinline__ Part part_of(const T* x, int n, int rank, int c, int per) {
    constexpr int N = Pack<T>::N;
    const int h = head_len(x, n), nb = (n - h) / N;
    const int s = min(rank * per, nb), e = min(s + per, nb);      // per: chunks a CTA
    Part p;
    p.b0 = h + s * N;
    p.bn = (e - s) * N;
    p.hn = rank == 0 ? h : 0;
    p.t0 = h + nb * N;
    p.tn = rank == c - 1 ? n - p.t0 : 0;
    return p;
}

// The rows of a window, dealt out: the rows that count first, then the others, round robin over
// the clusters.  Dealt by row number instead, the prompts (runs of rows that cost half as much,
// or nothing) left some CTAs 12% more work than the mean.  Every CTA makes its own list, with
// all threads: it reads the window's weights, which L2 holds.  kGrad goes backwards, as the last
// rows read are still in L2.
struct Window {
    long long w0;        // first row
    int n, live;         // rows of this cluster's list, of which the first `live` count
};

template <int MODE>
__device__ __forceinline__ long long window_row(const PostParams& P, const Window& W, int k) {
    return MODE == kGrad ? P.ntok - 1 - (W.w0 + k) : W.w0 + k;
}

template <int MODE>
__device__ Window deal(const PostParams& P, RSmem& S, long long w0, long long cid, long long ncl) {
    const float* wt = MODE == kGrad ? P.coef : P.weight;
    Window W{w0, 0, 0};
    if (P.ntok <= ncl) {                 // one row a cluster
        if (threadIdx.x == 0) S.list[0] = (int)cid;
        __syncthreads();
        W.n = 1;
        W.live = wt[window_row<MODE>(P, W, (int)cid)] != 0.f;
        return W;
    }
    const int n = (int)min(P.ntok - w0, ncl * kWindow);
    const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const int per = (n + RT - 1) / RT * 32, lo = wp * per, hi = min(n, lo + per);
    auto counts = [&](int k) { return k < hi && wt[window_row<MODE>(P, W, k)] != 0.f; };
    int mine = 0;
    uint64_t flags = 0;                  // this lane's rows lo + 32 q + lane, bit q (a window is cut to fit)
#pragma unroll 8
    for (int q = 0; q < per / 32; ++q) {
        const bool f = counts(lo + 32 * q + lane);
        flags |= (uint64_t)f << q;
        mine += __popc(__ballot_sync(0xffffffffu, f));
    }
    __syncthreads();                     // everybody is done with the list before
    if (lane == 0) S.wlive[wp] = mine;
    __syncthreads();
    int before = 0, all = 0;
    for (int i = 0; i < RT / 32; ++i) {
        before += i < wp ? S.wlive[i] : 0;
        all += S.wlive[i];
    }
    for (int k = lo; k < hi; k += 32) {
        const bool c = (flags >> ((k - lo) >> 5)) & 1u;
        const unsigned live = __ballot_sync(0xffffffffu, c), under = (1u << lane) - 1u;
        if (k + lane < hi) {
            const unsigned lb = (unsigned)before + __popc(live & under);
            const unsigned j = c ? lb : (unsigned)all + (unsigned)(k + lane) - lb;     // place among all rows
            const unsigned q = j / (unsigned)ncl;
            if (j - q * (unsigned)ncl == (unsigned)cid) S.list[q] = k + lane;
        }
        before += __popc(live);
    }
    __syncthreads();
    W.n = (int)((n - cid + ncl - 1) / ncl);
    W.live = (int)((all - cid + ncl - 1) / ncl);
    return W;
}

template <typename T, int MODE>
__device__ bool ring_producer(const PostParams& P, RSmem& S, int rank, int c, const Window& W, uint32_t& g, uint32_t& b) {
    constexpr int TE = TILE_B / (int)sizeof(T);
    const int lane = threadIdx.x & 31, n = (int)P.V;
    const int per = (n / Pack<T>::N + c - 1) / c;
    bool ok = true;
    // The preference loss reads its logits twice; what the gradient pass reads first, the last
    // kKeepBytes, is kept in L2 over the rest of the traffic.
    const uint64_t gone = l2_evict_first(), keep = l2_evict_last();
    const long long kept = MODE == kLogp ? P.ntok - kKeepBytes / (P.V * (long long)sizeof(T)) : 0;
    // tiles [t0, t1) of list entry k
    auto issue = [&](int k, int t0, int t1) {
        const long long r = window_row<MODE>(P, W, S.list[k]);
        const T* x = static_cast<const T*>(P.x) + r * P.ld;
        const Part pt = part_of(x, n, rank, c, per);
        const uint64_t policy = MODE == kLogp && P.g && r >= kept ? keep : gone;
        for (int t = t0; t < t1 && t * TE < pt.bn; ++t) {
            const uint32_t slot = g % SLOTS, use = g / SLOTS;
            if (use > 0 && !wait_parity<false>(&S.empty[slot], (use - 1) & 1u, &S.abort, &g_watchdog)) return false;
            const uint32_t bytes = (uint32_t)min(TE, pt.bn - t * TE) * (uint32_t)sizeof(T);
            mbar_arrive_expect_tx(&S.full[slot], bytes);
            if (MODE == kPolicy) bulk_g2s(S.ring[slot], x + pt.b0 + t * TE, bytes, &S.full[slot]);
            else bulk_g2s_hint(S.ring[slot], x + pt.b0 + t * TE, bytes, &S.full[slot], policy);
            ++g;
        }
        return true;
    };
    // The first row's tiles go out before its token data is fetched, as many as the ring takes
    // without a consumer's help: of a window's first tiles each slot's last use is over.
    if (lane == 0 && W.live > 0) ok = issue(0, 0, SLOTS);
    ok = __all_sync(0xffffffffu, ok);
    for (int k0 = 0; k0 < W.n && ok; k0 += BATCH, ++b) {
        const int k = k0 + lane;
        Meta m;
        m.live = 0;
        if (k < W.n) {
            const long long r = window_row<MODE>(P, W, S.list[k]);
            m.a = P.label[r];
            if (MODE == kGrad) {
                m.w = P.coef[r];
                m.live = k < W.live && m.w != 0.f;
                if (m.live) {
                    m.xa = P.stats[2 * r];
                    m.old = P.stats[2 * r + 1];
                    if ((long long)m.a < P.V) m.ref = ld_elem(static_cast<const T*>(P.x) + r * P.ld + m.a);
                }
            } else {
                m.w = P.weight[r];
                if (MODE == kPolicy) {
                    m.old = P.old_logp[r];
                    m.ref = P.ref_logp ? P.ref_logp[r] : 0.f;
                    m.adv = P.adv[r];
                }
                m.live = k < W.live && m.w != 0.f && (long long)m.a < P.V;
                if (m.live) m.xa = ld_elem(static_cast<const T*>(P.x) + r * P.ld + m.a);
            }
        }
        if (b >= 2) ok = wait_parity<false>(&S.mempty[b & 1], ((b >> 1) - 1) & 1u, &S.abort, &g_watchdog);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        S.meta[b & 1][lane] = m;
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&S.mfull[b & 1]);
            for (int j = k0; j < min(k0 + BATCH, W.live) && ok; ++j) ok = issue(j, j == 0 ? SLOTS : 0, 0x7fffffff);
        }
        ok = __all_sync(0xffffffffu, ok);
    }
    return ok;
}

template <typename T, int MODE>
__device__ void ring_consumer(const PostParams& P, RSmem& S, int rank, int c, const Window& W, uint32_t& g,
                              uint32_t& batch, uint32_t& nx) {
    constexpr int N = Pack<T>::N, H = N / 2;
    constexpr int TE = TILE_B / (int)sizeof(T);
    constexpr int RTILES = REGV / (CHT * N);         // policy: tiles a thread's registers hold (4 fp32, 2 bf16)
    const int ct = (int)threadIdx.x, lane = ct & 31, cw = ct >> 5, n = (int)P.V;
    const int per = (n / N + c - 1) / c;
    const uint64_t l2e = pack2(kLog2e, kLog2e), first = MODE == kGrad ? l2_evict_first() : 0;
    const bool reads_meta = MODE == kGrad || cw == 0;
    // rows of one alignment are all cut alike
    const bool uniform = ((P.ld * (long long)sizeof(T)) & 15) == 0;
    Part pt = part_of(static_cast<const T*>(P.x), n, rank, c, per);
    // chunk u of the tile in `slot`, where the row has it; -inf elsewhere
    constexpr uint32_t kNegInf = sizeof(T) == 4 ? 0xff800000u : 0xff80ff80u;
    auto chunk = [&](uint32_t slot, int u, bool here) {
        return ld_shared_if(smem_u32(&S.ring[slot][16 * (u * CT + ct)]), here, kNegInf);
    };
    auto await = [&](uint32_t gt) {
        wait_parity<false>(&S.full[gt % SLOTS], (gt / SLOTS) & 1u, &S.abort, &g_watchdog);
        return gt % SLOTS;
    };
    auto release = [&](uint32_t slot) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.empty[slot]);
    };
    int next = S.list[0];
    for (int k = 0; k < W.n; ++k) {
        if (reads_meta && k % BATCH == 0 && k > 0) { // this warp is done with the batch before
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.mempty[batch & 1]);
            ++batch;
        }
        const Meta& mt = S.meta[batch & 1][k % BATCH];
        auto meta_ready = [&] {
            if (k % BATCH == 0) wait_parity<false>(&S.mfull[batch & 1], (batch >> 1) & 1u, &S.abort, &g_watchdog);
        };
        const long long r = window_row<MODE>(P, W, next);
        next = S.list[min(k + 1, W.n - 1)];
        const T* x = static_cast<const T*>(P.x) + r * P.ld;
        T* gr = P.g ? static_cast<T*>(P.g) + r * P.ldg : nullptr;
        if (!uniform) pt = part_of(x, n, rank, c, per);
        const int nt = (pt.bn + TE - 1) / TE, n16 = pt.bn / N;
        const bool wide = ((reinterpret_cast<uintptr_t>(gr + pt.b0)) & 15u) == 0;
        const int jht = ct < pt.hn ? ct : ct >= N && ct - N < pt.tn ? pt.t0 + ct - N : -1;
        // chunk q of the part's body (this thread's, where the row has it): its gradient but for the
        // picked column
        auto store = [&](int q, uint64_t (&o)[H]) {
            T* at = gr + pt.b0 + N * q;
            float v[N];
#pragma unroll
            for (int e = 0; e < H; ++e) unpack2(o[e], v[2 * e], v[2 * e + 1]);
            if (MODE == kGrad) st_global_if(at, Pack<T>::pack(v), wide && q < n16, first);
            else st_global_if(at, Pack<T>::pack(v), wide && q < n16);
            if (!wide && q < n16) {
#pragma unroll
                for (int e = 0; e < N; ++e) st_elem(at + e, v[e]);
            }
        };
        // the head or tail column of this thread, then the picked column a, which the thread that
        // stored its chunk rewrites with `pick`
        auto store_rest = [&](float ht, float m, float lnS, float f0, int a, float pick) {
            if (jht >= 0) st_elem(gr + jht, -f0 * ex2(((ht - m) - lnS) * kLog2e));
            const int d = a - pt.b0;
            if (a >= 0 && ((unsigned)d < (unsigned)pt.bn ? (d / N) % CT == ct : a == jht)) st_elem(gr + a, pick);
        };
        auto store_zeros = [&] {
            uint64_t z[H] = {};
            for (int q = ct; q < n16; q += CT) store(q, z);
            if (jht >= 0) st_elem(gr + jht, 0.f);
        };
        if (k >= W.live) {
            if (reads_meta) meta_ready();
            if (MODE != kGrad && rank == 0 && ct == 0) skip_row<MODE>(P, r, mt.w);
            if (MODE != kLogp && gr) store_zeros();
            continue;
        }
        const float ht = jht >= 0 ? ld_elem(x + jht) : 0.f;
        if (MODE == kGrad) {
            // the row's statistics are known: each tile turned into gradient as it lands
            meta_ready();
            const float m = mt.xa, lnS = mt.old, f0 = mt.w;
            const uint64_t nm = pack2(-m, -m), nl = pack2(-lnS, -lnS), f2 = pack2(-f0, -f0);
            for (int t = 0; t < nt; ++t, ++g) {
                const uint32_t slot = await(g);
                const int q0 = t * CHT * CT + ct;
                uint64_t v[CHT][H];
#pragma unroll
                for (int u = 0; u < CHT; ++u) unpack_pairs<T>(chunk(slot, u, q0 + u * CT < n16), v[u]);
                release(slot);
#pragma unroll
                for (int u = 0; u < CHT; ++u) {
#pragma unroll
                    for (int e = 0; e < H; ++e) v[u][e] = mul2(exp_pair(add2(v[u][e], nm), nl, l2e), f2);
                    store(q0 + u * CT, v[u]);
                }
            }
            store_rest(ht, m, lnS, f0, (int)mt.a, f0 - f0 * ex2(((mt.ref - m) - lnS) * kLog2e));
            continue;
        }
        MaxSum ms = ms_empty();
        // tile t's exponentials against the running maximum into v, their sum into ms; absent
        // chunks of a row's last tile are skipped
        auto tile = [&](int t, uint64_t (&v)[CHT][H]) {
            const uint32_t slot = await(g + (uint32_t)t);
            const int q0 = t * CHT * CT + ct;
            float M = ms.m;
            float mu[CHT];
#pragma unroll
            for (int u = 0; u < CHT; ++u) {
                unpack_pairs<T>(chunk(slot, u, q0 + u * CT < n16), v[u]);
                mu[u] = -FLT_MAX;
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    float a, b;
                    unpack2(v[u][e], a, b);
                    mu[u] = max3(mu[u], a, b);
                }
            }
            release(slot);
#pragma unroll
            for (int u = 0; u < CHT; u += 2) M = max3(M, mu[u], mu[u + 1]);
            ms.s *= ex2((ms.m - M) * kLog2e);
            ms.m = M;
            const uint64_t nm = pack2(-M, -M);
            uint64_t s[CHT];
#pragma unroll
            for (int u = 0; u < CHT; ++u) {
#pragma unroll
                for (int e = 0; e < H; ++e) {
                    v[u][e] = exp_pair(v[u][e], nm, l2e);
                    s[u] = e == 0 ? v[u][e] : add2(s[u], v[u][e]);
                }
            }
#pragma unroll
            for (int u = 1; u < CHT; ++u) s[0] = add2(s[0], s[u]);
            float a, b;
            unpack2(s[0], a, b);
            ms.s += a + b;
        };
        uint64_t E[MODE == kPolicy ? RTILES : 1][CHT][H];
        float mx[RTILES];
        if (MODE == kPolicy) {
#pragma unroll
            for (int t = 0; t < RTILES; ++t)
                if (t < nt) {
                    tile(t, E[t]);
                    mx[t] = ms.m;
                }
            // what the registers do not hold stays in the ring for the gradient
            for (int t = RTILES; t < nt; ++t) {
                const uint32_t slot = await(g + (uint32_t)t);
                const int q0 = t * CHT * CT + ct;
#pragma unroll 1
                for (int u = 0; u < CHT && q0 + u * CT < n16; ++u) {
                    uint64_t v[H];
                    unpack_pairs<T>(chunk(slot, u, true), v);
                    float M = ms.m;
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        float a, b;
                        unpack2(v[e], a, b);
                        M = max3(M, a, b);
                    }
                    ms.s *= ex2((ms.m - M) * kLog2e);
                    ms.m = M;
                    uint64_t s = 0;
#pragma unroll
                    for (int e = 0; e < H; ++e) s = add2(s, exp_pair(v[e], pack2(-M, -M), l2e));
                    float a, b;
                    unpack2(s, a, b);
                    ms.s += a + b;
                }
            }
        } else {
            for (int t = 0; t < nt; ++t) tile(t, E[0]);
        }
        const uint32_t g0 = g;
        g += (uint32_t)nt;
        if (jht >= 0) ms_add(ms, ht);
        const MaxSum wm = warp_max_sum(ms);
        // every warp's partial (of every rank) meets in warp 0, which settles the row
        const uint32_t pb = nx % NB, ppar = (nx / NB) & 1u, rb = nx & 1u;
        ++nx;
        if (c > 1) {
            // Once every partial is in, a peer may write its part of the row, in place over the picked
            // logit: this rank's must have been fetched by then.
            if (MODE == kPolicy && cw == 0) meta_ready();
            if (ct == 0) mbar_arrive_expect_tx(&S.pbar[pb], 8u * (uint32_t)(c * CW));
            if (lane < c)
                st_async_f32x2(map_to_rank(&S.part[pb][rank * CW + cw], (uint32_t)lane), wm.m, wm.s,
                               map_to_rank(&S.pbar[pb], (uint32_t)lane));
        } else if (lane == 0) {
            S.part[pb][cw] = make_float2(wm.m, wm.s);
            mbar_arrive(&S.pbar[pb]);
        }
        if (cw == 0) {
            meta_ready();
            const bool bad = !mt.live;               // a column past the row
            MaxSum tot;
            if (c > 1) {
                wait_parity<true>(&S.pbar[pb], ppar, &S.abort, &g_watchdog);
                tot = combine_parts(S.part[pb], c * CW, lane);
            } else {
                wait_parity<false>(&S.pbar[pb], ppar, &S.abort, &g_watchdog);
                const float2 q = lane < CW ? S.part[pb][lane] : make_float2(-FLT_MAX, 0.f);
                tot = warp_max_sum(MaxSum{q.x, q.y});
            }
            const float l = logf(tot.s);
            float f = 0.f;
            if (!bad) f = settle_row<MODE>(P, r, mt.w, mt.old, mt.ref, mt.adv, mt.xa, tot.m, l, rank == 0 && lane == 0);
            else if (rank == 0 && lane == 0) skip_row<MODE>(P, r, mt.w);
            if (MODE == kPolicy && lane == 0) {
                S.row[rb] = make_float4(tot.m, l, f, f - f * ex2(((mt.xa - tot.m) - l) * kLog2e));
                S.picked[rb] = f != 0.f ? (int)mt.a : -1;
            }
        }
        if (MODE == kLogp) continue;
        named_sync(1, CT);
        const float m = S.row[rb].x, lnS = S.row[rb].y, f0 = S.row[rb].z;
        if (f0 == 0.f) {                             // no gradient (whatever the logits hold)
            for (int t = RTILES; t < nt; ++t) release((g0 + (uint32_t)t) % SLOTS);
            if (gr) store_zeros();
            continue;
        }
        for (int t = RTILES; t < nt; ++t) {
            const uint32_t slot = (g0 + (uint32_t)t) % SLOTS;
            if (gr) {
                const uint64_t nm = pack2(-m, -m), nl = pack2(-lnS, -lnS), f2 = pack2(-f0, -f0);
                const int q0 = t * CHT * CT + ct;
#pragma unroll 1
                for (int u = 0; u < CHT && q0 + u * CT < n16; ++u) {
                    uint64_t v[H];
                    unpack_pairs<T>(chunk(slot, u, true), v);
#pragma unroll
                    for (int e = 0; e < H; ++e) v[e] = mul2(exp_pair(add2(v[e], nm), nl, l2e), f2);
                    store(q0 + u * CT, v);
                }
            }
            release(slot);
        }
        if (!gr) continue;
#pragma unroll
        for (int t = 0; t < RTILES; ++t)
            if (t < nt) {
                const float f = -f0 * ex2(((mx[t] - m) - lnS) * kLog2e);
                const uint64_t f2 = pack2(f, f);
                const int q0 = t * CHT * CT + ct;
#pragma unroll
                for (int u = 0; u < CHT; ++u) {
#pragma unroll
                    for (int e = 0; e < H; ++e) E[MODE == kPolicy ? t : 0][u][e] = mul2(E[MODE == kPolicy ? t : 0][u][e], f2);
                    store(q0 + u * CT, E[MODE == kPolicy ? t : 0][u]);
                }
            }
        store_rest(ht, m, lnS, f0, S.picked[rb], S.row[rb].w);
    }
    if (reads_meta) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.mempty[batch & 1]);
        ++batch;
    }
}

template <typename T, int MODE>
__global__ void __launch_bounds__(RT, 1) rows_ring(const __grid_constant__ PostParams P, int c) {
    extern __shared__ __align__(128) unsigned char ring_raw[];
    RSmem& S = *reinterpret_cast<RSmem*>(ring_raw);
    const int rank = c > 1 ? (int)cluster_ctarank() : 0;
    const long long cid = blockIdx.x / c, ncl = gridDim.x / c;
    if (threadIdx.x == 0) {
        for (int s = 0; s < SLOTS; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], CW);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.mfull[b], 1);
            mbar_init(&S.mempty[b], MODE == kGrad ? CW : 1);
        }
        for (int b = 0; b < NB; ++b) mbar_init(&S.pbar[b], c > 1 ? 1 : CW);
        S.abort = 0;
        fence_mbar_init_cluster();
    }
    if (c > 1) cluster_sync_all();
    else __syncthreads();
    pdl_launch_dependents();
    pdl_wait_primary();
    uint32_t g = 0, batch = 0, nx = 0;
    bool ok = true;
    for (long long w0 = 0; w0 < P.ntok; w0 += ncl * kWindow) {
        const Window W = deal<MODE>(P, S, w0, cid, ncl);
        if (W.n == 0) continue;
        if (threadIdx.x < CT) ring_consumer<T, MODE>(P, S, rank, c, W, g, batch, nx);
        else if (ok) ok = ring_producer<T, MODE>(P, S, rank, c, W, g, batch);
    }
    if (threadIdx.x == CT)            // every copy issued has landed before the CTA leaves
        for (uint32_t gt = g > (uint32_t)SLOTS ? g - SLOTS : 0u; gt < g; ++gt)
            wait_parity_drain(&S.full[gt % SLOTS], (gt / SLOTS) & 1u);
    __syncwarp();
    if (c > 1) cluster_sync_all();       // no CTA may leave while a peer can still write to it
}

// ---------------------------------------------------------------- pairs

// Unevaluated pairs of floats (about 48 bits): the sums over a sequence and over the rows. The
// card's 64-bit rate is far below its 32-bit one (the pair kernel took 11 us with doubles).  Each
// operation rounds by itself: a product fused into one of two_sum's additions would leave its low
// part counted twice.
struct FF {
    float hi, lo;
};
__device__ __forceinline__ FF two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
    return FF{s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}
__device__ __forceinline__ FF ff_add(FF a, FF b) {
    const FF s = two_sum(a.hi, b.hi);
    // an infinite or NaN sum has no error term (inf - inf would make one)
    const float e = isfinite(s.hi) ? __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)) : 0.f;
    const float h = __fadd_rn(s.hi, e);
    return FF{h, isfinite(h) ? __fsub_rn(e, __fsub_rn(h, s.hi)) : 0.f};
}
__device__ __forceinline__ FF ff_mul(float a, float b) {
    const float p = __fmul_rn(a, b);
    return FF{p, isfinite(p) ? __fmaf_rn(a, b, -p) : 0.f};
}

__device__ __forceinline__ FF warp_sum_ff(FF v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        v = ff_add(v, FF{__shfl_xor_sync(0xffffffffu, v.hi, off), __shfl_xor_sync(0xffffffffu, v.lo, off)});
    return v;
}

// The sum over the CTA's 1024 threads, in a fixed order; every thread gets it.
__device__ FF cta_sum(FF v, FF* red) {
    v = warp_sum_ff(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    return warp_sum_ff(red[threadIdx.x & 31]);
}

__device__ __forceinline__ float softplus(float v) {       // ln(1 + e^v)
    return fmaxf(v, 0.f) + log1pf(expf(-fabsf(v)));
}

// The pairs, in one launch of one cluster, so that the mean needs no other: each group of 128
// threads takes pairs group, group + 64, ...: both sequences' sums, the pair's loss and each row's
// factor.  After the cluster's barrier one CTA sums the losses.
constexpr int kPairCtas = 8, kPairGroups = 8, GTH = 1024 / kPairGroups;

__global__ void __cluster_dims__(kPairCtas, 1, 1) __launch_bounds__(1024) pair_kernel(const __grid_constant__ PairParams Q) {
    __shared__ FF red[32];
    __shared__ FF part[kPairGroups][2][GTH / 32];
    __shared__ int flag[kPairGroups][GTH / 32];
    const int grp = threadIdx.x / GTH, gt = threadIdx.x % GTH, lane = threadIdx.x & 31, gw = gt >> 5;
    pdl_launch_dependents();
    pdl_wait_primary();
    for (long long i = blockIdx.x * kPairGroups + grp; i < Q.npairs; i += kPairCtas * kPairGroups) {
        long long lo[2], hi[2];
        int bad = 0;
        for (int k = 0; k < 2; ++k) {
            const long long s = i + (k ? Q.npairs : 0);
            lo[k] = min(max(Q.start[s], 0ll), Q.ntok);
            hi[k] = min(max(Q.start[s + 1], lo[k]), Q.ntok);
        }
        for (int k = 0; k < 2; ++k) {
            FF v{0.f, 0.f};
#pragma unroll 4
            for (long long t = lo[k] + gt; t < hi[k]; t += GTH) {
                const float w = Q.weight[t], c = Q.coef[t], l = Q.logp[t];
                if (w == 0.f) continue;
                if (signbit(c)) bad = 1;
                v = ff_add(v, ff_mul(w, l));
            }
            v = warp_sum_ff(v);
            if (lane == 0) part[grp][k][gw] = v;
        }
        bad = __any_sync(0xffffffffu, bad);
        if (lane == 0) flag[grp][gw] = bad;
        named_sync(1 + grp, GTH);
        FF sum[2];
        for (int k = 0; k < 2; ++k) {
            sum[k] = part[grp][k][0];
            for (int j = 1; j < GTH / 32; ++j) sum[k] = ff_add(sum[k], part[grp][k][j]);
        }
        bad = 0;
        for (int j = 0; j < GTH / 32; ++j) bad |= flag[grp][j];
        FF gap = ff_add(sum[0], FF{-sum[1].hi, -sum[1].lo});
        if (Q.ref) gap = ff_add(gap, two_sum(-Q.ref[i], Q.ref[Q.npairs + i]));
        const float h = Q.beta * gap.hi + Q.beta * gap.lo;
        float loss, d;                              // d loss / d gap
        if (Q.kind == VL_PREF_SIGMOID) {
            loss = (1.f - Q.smooth) * softplus(-h);
            if (Q.smooth != 0.f) loss += Q.smooth * softplus(h);      // (0 times infinity where h is infinite)
            // sigmoid(h) - (1 - smooth), each tail from the side that does not cancel
            const float e = expf(-fabsf(h)), small = e / (1.f + e);
            d = Q.beta * (h >= 0.f ? Q.smooth - small : small - (1.f - Q.smooth));
        } else if (Q.kind == VL_PREF_IPO) {
            const float half = 0.5f / Q.beta, rest = fmaf(-half, Q.beta, 0.5f) / Q.beta;    // 1 / (2 beta), in two parts
            const FF zz = ff_add(gap, FF{-half, -rest});
            const float z = zz.hi + zz.lo;
            loss = z * z;
            d = 2.f * z;
        } else {
            loss = h < 1.f ? 1.f - h : h >= 1.f ? 0.f : h;    // a NaN stays one
            d = h < 1.f ? -Q.beta : h >= 1.f ? 0.f : h;
        }
        if (gt == 0) {
            Q.loss[i] = loss;
            Q.margin[i] = h;
            if (Q.seq) {
                Q.seq[i] = sum[0].hi + sum[0].lo;
                Q.seq[Q.npairs + i] = sum[1].hi + sum[1].lo;
            }
        }
        for (int k = 0; k < 2; ++k)
            for (long long t = lo[k] + gt; t < hi[k]; t += GTH) {
                const float w = Q.weight[t];
                Q.coef[t] = bad || w == 0.f ? 0.f : Q.scale * (k ? -d : d) * w;
            }
        named_sync(1 + grp, GTH);                   // the partials' buffer is free again
    }
    if (!Q.mean) return;
    cluster_sync_all();                             // every loss is written, visible to the cluster
    if (blockIdx.x != 0) return;
    FF v{0.f, 0.f};
    for (long long i = threadIdx.x; i < Q.npairs; i += 1024) v = ff_add(v, FF{__ldcg(Q.loss + i), 0.f});
    v = cta_sum(v, red);
    if (threadIdx.x == 0) *Q.mean = Q.npairs > 0 ? v.hi / (float)Q.npairs + v.lo / (float)Q.npairs : 0.f;
}

// The sum of n losses.
__global__ void __launch_bounds__(1024) total_kernel(const float* loss, long long n, float* total) {
    __shared__ FF red[32];
    pdl_launch_dependents();
    pdl_wait_primary();
    FF v{0.f, 0.f};
    for (long long i = threadIdx.x; i < n; i += 1024) v = ff_add(v, FF{loss[i], 0.f});
    v = cta_sum(v, red);
    if (threadIdx.x == 0) *total = v.hi + v.lo;
}

constexpr int kMaxDev = 64;

int device() {
    int d = 0;
    return cudaGetDevice(&d) == cudaSuccess && d >= 0 && d < kMaxDev ? d : -1;
}

// Clusters of c CTAs of the ring kernel that run at once (0: none); asked once per device.
template <typename T, int MODE>
int ring_clusters(int dev, int c) {
    static std::atomic<int> cache[kMaxDev][MAXC + 1];
    int v = cache[dev][c].load(std::memory_order_acquire);
    if (v != 0) return v > 0 ? v : 0;
    const void* fn = (const void*)rows_ring<T, MODE>;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(RSmem)) != cudaSuccess) return 0;
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    v = sms;
    if (c > 1) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(c * v), 1, 1);
        cfg.blockDim = dim3(RT, 1, 1);
        cfg.dynamicSmemBytes = sizeof(RSmem);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {(unsigned)c, 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&v, fn, &cfg) != cudaSuccess) {
            (void)cudaGetLastError();
            v = 0;
        }
    }
    cache[dev][c].store(v > 0 ? v : -1, std::memory_order_release);
    return v > 0 ? v : 0;
}

template <typename T, int MODE>
cudaError_t launch_ring(const PostParams& P, cudaStream_t st) {
    const int dev = device();
    if (dev < 0) return cudaErrorInvalidDevice;
    // CTAs a row: the policy pass needs the row in its registers.  Beyond that, the fewest
    // modelled bytes a CTA: rows a cluster x (its share of a row + the exchange, as bytes).
    int cmin = 1;
    if (MODE == kPolicy)
        while (cmin < MAXC && (P.V + cmin - 1) / cmin > kPartCols<T>) ++cmin;
    int best = 0, ncl = 0;
    double cost = 0;
    for (int c = cmin; c <= (MODE == kGrad ? 1 : MAXC); ++c) {
        const int n = ring_clusters<T, MODE>(dev, c);
        if (n <= 0) continue;
        const long long k = P.ntok < n ? P.ntok : n;
        const double t = (double)((P.ntok + k - 1) / k) *
                         ((double)((P.V + c - 1) / c) * sizeof(T) * (MODE == kPolicy ? 2 : 1) + (c > 1 ? 60e3 : 30e3));
        if (best == 0 || t < 0.97 * cost) {
            best = c;
            ncl = (int)k;
            cost = t;
        }
    }
    if (best == 0) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(ncl * best), 1, 1);
    cfg.blockDim = dim3(RT, 1, 1);
    cfg.dynamicSmemBytes = sizeof(RSmem);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {(unsigned)best, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = best > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, rows_ring<T, MODE>, P, best);
}

template <typename T, int MODE>
cudaError_t launch_rows_t(const PostParams& P, cudaStream_t st) {
    constexpr int N = Pack<T>::N;
    const long long grid = P.ntok < (1 << 20) ? P.ntok : (1 << 20);
    // Policy, 4096 x 2048 fp32: 19 us with 128 threads, 42 with 256.  4096 x 8192: 60 us so, 80 by the ring;
    // beyond, with 512 threads, one CTA fits an SM: 4096 x 8200 88 us, by the ring 77.
    if (P.V <= 2048) return launch_pdl(rows_direct<T, MODE, 128, 16 / N>, grid, 128, 0, st, P);
    if (P.V <= 8192) return launch_pdl(rows_direct<T, MODE, 256, 32 / N>, grid, 256, 0, st, P);
    if (MODE == kPolicy && P.V > VL_POLICY_ONEPASS_COLS) return launch_pdl(rows_twice<T>, grid, NT, 0, st, P);
    return launch_ring<T, MODE>(P, st);
}

template <int MODE>
cudaError_t launch_post(const PostParams& P, cudaStream_t st) {
    return P.dtype == kBf16 ? launch_rows_t<__nv_bfloat16, MODE>(P, st) : launch_rows_t<float, MODE>(P, st);
}

}  // namespace

cudaError_t launch_policy(const PostParams& P, float* total, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (P.ntok > 0) e = launch_post<kPolicy>(P, st);
    if (e == cudaSuccess && total) e = launch_pdl(total_kernel, 1, 1024, 0, st, (const float*)P.loss, P.ntok, total);
    return e;
}

cudaError_t launch_preference(const PostParams& P, const PairParams& Q, cudaStream_t st) {
    cudaError_t e = cudaSuccess;
    if (P.ntok > 0) e = launch_post<kLogp>(P, st);
    if (e == cudaSuccess) e = launch_pdl(pair_kernel, kPairCtas, 1024, 0, st, Q);
    if (e == cudaSuccess && P.ntok > 0 && P.g) e = launch_post<kGrad>(P, st);
    return e;
}

unsigned int post_watchdog(bool clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_watchdog, sizeof(v)) != cudaSuccess) return 0xffffffffu;
    if (clear && v) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_watchdog, &z, sizeof(z)) != cudaSuccess) return 0xffffffffu;
    }
    return v;
}

}  // namespace vl
