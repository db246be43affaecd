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
//   long rows    (rows_ring) one persistent CTA per SM, 15 consumer warps and a producer warp:
//                a ring of six 30 KB tiles of 1-D bulk copies runs ahead of the consumers, so
//                the reads go on while a row's statistics meet and its gradient is written.
//                What a row has beyond the registers (30720 columns) stays in the ring, up to
//                two tiles.  Longer rows, and rows too few for the SMs, are split over a cluster;
//                every warp sends its partial (max, sum) to every rank with st.async.
//   short rows   (rows_direct, up to 8192 columns) a CTA of 128 or 256 threads a row, loaded straight
//                into registers; many CTAs an SM overlap each other's phases.  A short row in the
//                ring kernel would leave most of its threads idle and pay a barrier a row.
//   beyond       (rows_twice) rows of more than VL_POLICY_ONEPASS_COLS columns are read twice.
//
// The producer warp also fetches each row's token data (weight, column, its logit, ...), 32 rows
// at a time, so that no consumer waits on a chain of global loads; rows that do not count are
// not read, their gradient rows are zeroed.
#include "vl_device.cuh"
#include "vl_internal.h"
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
    const float ratio = expf(logp - old);
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

// Warp partials (max, sum) of n <= 32 q values: every lane gets the row's (max, sum), combined
// in a fixed order, the same bits in every warp.
__device__ __forceinline__ MaxSum combine_parts(const float2* part, int n, int lane) {
    float2 q[4];
    float M = -FLT_MAX;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int j = lane + 32 * i;
        q[i] = j < n ? part[j] : make_float2(-FLT_MAX, 0.f);
        M = fmaxf(M, q[i].x);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
    float T = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) T += q[i].y * ex2((q[i].x - M) * kLog2e);
    return MaxSum{M, warp_sum(T)};
}

// ---------------------------------------------------------------- rows read twice

template <typename T>
__global__ void __launch_bounds__(NT) rows_twice(const __grid_constant__ PostParams P) {
    __shared__ float2 part[NT / 32];
    const int ct = threadIdx.x, n = (int)P.V;
    pdl_wait_primary();
    pdl_launch_dependents();
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
    pdl_wait_primary();
    pdl_launch_dependents();
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

constexpr int CW = 15;                   // consumer warps (with the producer 16: 128 registers a thread)
constexpr int CT = CW * 32;
constexpr int RT = CT + 32;              // + the producer warp
constexpr int CHT = 4;                   // 16-byte chunks of a tile per consumer thread
constexpr int TILE_B = CT * CHT * 16;    // 30 KB
constexpr int SLOTS = 6;
constexpr int REGV = 64;                 // exponentials a thread holds in registers
constexpr int HOLD = 2;                  // tiles of a row that stay in the ring until its gradient is written
constexpr int MAXC = 8;                  // CTAs a row
constexpr int BATCH = 32;                // rows whose token data the producer fetches at once

__device__ unsigned int g_watchdog;

// Two fp32 lanes in one instruction.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void unpack2(uint64_t d, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(d));
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
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
    float ref, adv;
    int live;
};

struct alignas(128) RSmem {
    alignas(16) unsigned char ring[SLOTS][TILE_B];
    uint64_t full[SLOTS], empty[SLOTS];
    uint64_t mfull[2], mempty[2];
    uint64_t xbar[2];
    float2 xw[2][MAXC * CW];             // cluster: every warp's partial, from every rank
    float2 part[2][16];
    float4 row[2];                       // (m, lnS, c) of the row, from the warp that settles it
    Meta meta[2][BATCH];
    int abort;
};
static_assert(sizeof(RSmem) <= 227 * 1024, "shared memory of one CTA");
static_assert(MAXC * CW <= 128, "combine_parts takes up to 128 partials");
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

template <int MODE>
__device__ __forceinline__ long long row_of(const PostParams& P, long long i) {
    return MODE == kGrad ? P.ntok - 1 - i : i;      // backwards: the last rows read are still in L2
}

template <typename T, int MODE>
__device__ void ring_producer(const PostParams& P, RSmem& S, int rank, int c, long long cid, long long ncl) {
    constexpr int TE = TILE_B / (int)sizeof(T);
    const int lane = threadIdx.x & 31, n = (int)P.V;
    const int per = (n / Pack<T>::N + c - 1) / c;
    uint32_t g = 0;
    bool ok = true;
    // tiles [t0, t1) of item i
    auto issue = [&](long long i, int t0, int t1) {
        const T* x = static_cast<const T*>(P.x) + row_of<MODE>(P, i) * P.ld;
        const Part pt = part_of(x, n, rank, c, per);
        for (int t = t0; t < t1 && t * TE < pt.bn; ++t) {
            const uint32_t slot = g % SLOTS, use = g / SLOTS;
            if (use > 0 && !wait_parity<false>(&S.empty[slot], (use - 1) & 1u, &S.abort, &g_watchdog)) return false;
            const uint32_t bytes = (uint32_t)min(TE, pt.bn - t * TE) * (uint32_t)sizeof(T);
            mbar_arrive_expect_tx(&S.full[slot], bytes);
            bulk_g2s(S.ring[slot], x + pt.b0 + t * TE, bytes, &S.full[slot]);
            ++g;
        }
        return true;
    };
    // The first row's tiles go out before anything is known of it (it is read even if it does
    // not count); they never wait, so no consumer has to have started.
    if (lane == 0 && cid < P.ntok) issue(cid, 0, SLOTS);
    __syncwarp();
    for (long long b = 0; cid + b * BATCH * ncl < P.ntok; ++b) {
        const long long i = cid + (b * BATCH + lane) * ncl;
        Meta m;
        m.live = 0;
        if (i < P.ntok) {
            const long long r = row_of<MODE>(P, i);
            m.a = P.label[r];
            if (MODE == kGrad) {
                m.w = P.coef[r];
                m.xa = P.stats[2 * r];
                m.old = P.stats[2 * r + 1];
                m.live = m.w != 0.f;
            } else {
                m.w = P.weight[r];
                if (MODE == kPolicy) {
                    m.old = P.old_logp[r];
                    m.ref = P.ref_logp ? P.ref_logp[r] : 0.f;
                    m.adv = P.adv[r];
                }
                m.live = m.w != 0.f && (long long)m.a < P.V;
                if (m.live) m.xa = ld_elem(static_cast<const T*>(P.x) + r * P.ld + m.a);
            }
        }
        if (ok && b >= 2) ok = wait_parity<false>(&S.mempty[b & 1], (uint32_t)((b >> 1) - 1) & 1u, &S.abort, &g_watchdog);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        S.meta[b & 1][lane] = m;
        const uint32_t live = __ballot_sync(0xffffffffu, m.live != 0);
        __syncwarp();
        if (lane == 0) {
            mbar_arrive(&S.mfull[b & 1]);
            for (int k = 0; k < BATCH && ok; ++k) {
                const long long ik = cid + (b * BATCH + k) * ncl;
                if (ik >= P.ntok) break;
                const bool first = b == 0 && k == 0;
                if (first || (live >> k & 1u)) ok = issue(ik, first ? SLOTS : 0, 0x7fffffff);
            }
        }
        ok = __all_sync(0xffffffffu, ok);
    }
    if (lane == 0)
        for (uint32_t gt = g > (uint32_t)SLOTS ? g - SLOTS : 0u; gt < g; ++gt)
            wait_parity_drain(&S.full[gt % SLOTS], (gt / SLOTS) & 1u);
}

template <typename T, int MODE>
__device__ void ring_consumer(const PostParams& P, RSmem& S, int rank, int c, long long cid, long long ncl) {
    constexpr int N = Pack<T>::N, H = N / 2;
    constexpr int TE = TILE_B / (int)sizeof(T);
    constexpr int RTILES = REGV / (CHT * N);         // tiles a thread's registers hold: 4 fp32, 2 bf16
    const int ct = (int)threadIdx.x, lane = ct & 31, cw = ct >> 5, n = (int)P.V;
    const int per = (n / N + c - 1) / c;
    const uint64_t l2e = pack2(kLog2e, kLog2e);
    uint32_t g = 0, nx = 0, k = 0, batch = 0;
    // chunk u of the tile in `slot`
    auto chunk = [&](uint32_t slot, int u) { return *reinterpret_cast<const uint4*>(&S.ring[slot][16 * (u * CT + ct)]); };
    auto await = [&](uint32_t gt) {
        wait_parity<false>(&S.full[gt % SLOTS], (gt / SLOTS) & 1u, &S.abort, &g_watchdog);
        return gt % SLOTS;
    };
    auto release = [&](uint32_t slot) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.empty[slot]);
    };
    for (long long i = cid; i < P.ntok; i += ncl) {
        if (k == BATCH) {                            // this warp is done with the batch before
            __syncwarp();
            if (lane == 0) mbar_arrive(&S.mempty[batch & 1]);
            k = 0;
            ++batch;
        }
        if (k == 0) wait_parity<false>(&S.mfull[batch & 1], (batch >> 1) & 1u, &S.abort, &g_watchdog);
        const Meta& mt = S.meta[batch & 1][k++];
        const long long r = row_of<MODE>(P, i);
        const T* x = static_cast<const T*>(P.x) + r * P.ld;
        T* gr = P.g ? static_cast<T*>(P.g) + r * P.ldg : nullptr;
        const Part pt = part_of(x, n, rank, c, per);
        const int nt = (pt.bn + TE - 1) / TE, n16 = pt.bn / N;
        const bool wide = ((reinterpret_cast<uintptr_t>(gr + pt.b0)) & 15u) == 0;
        const int jht = ct < pt.hn ? ct : ct >= N && ct - N < pt.tn ? pt.t0 + ct - N : -1;
        // chunk q of the part's body is this thread's; its gradient
        auto store = [&](int q, uint64_t (&o)[H], float f0) {
            T* at = gr + pt.b0 + N * q;
            const unsigned d = mt.a - (unsigned)(pt.b0 + N * q);
            float v[N];
#pragma unroll
            for (int e = 0; e < H; ++e) unpack2(o[e], v[2 * e], v[2 * e + 1]);
            if (d < (unsigned)N) {
#pragma unroll
                for (int e = 0; e < N; ++e)
                    if ((unsigned)e == d) v[e] += f0;
            }
            if (wide) {
                *reinterpret_cast<uint4*>(at) = Pack<T>::pack(v);
            } else {
#pragma unroll
                for (int e = 0; e < N; ++e) st_elem(at + e, v[e]);
            }
        };
        auto store_ht = [&](float ht, float m, float lnS, float f0) {
            float o = f0 == 0.f ? 0.f : -f0 * ex2(((ht - m) - lnS) * kLog2e);
            if (jht == (int)mt.a) o += f0;
            st_elem(gr + jht, o);
        };
        if (!mt.live) {
            if (i == cid) {                          // its tiles were issued: let them pass
                for (int t = 0; t < nt; ++t, ++g) release(await(g));
            }
            if (MODE != kGrad && rank == 0 && ct == 0) skip_row<MODE>(P, r, mt.w);
            if (MODE != kLogp && gr) {
                uint64_t z[H] = {};
                for (int q = ct; q < n16; q += CT) store(q, z, 0.f);
                if (jht >= 0) st_elem(gr + jht, 0.f);
            }
            continue;
        }
        const float ht = jht >= 0 ? ld_elem(x + jht) : 0.f;
        // the gradient of a tile that is in the ring, from the row's statistics
        auto tile_gradient = [&](uint32_t slot, int t, float m, float lnS, float f0) {
            const uint64_t nm = pack2(-m, -m), nl = pack2(-lnS, -lnS), f2 = pack2(-f0, -f0);
            const int q0 = t * CHT * CT + ct;
            uint64_t v[CHT][H];
#pragma unroll
            for (int u = 0; u < CHT; ++u)
                if (q0 + u * CT < n16) unpack_pairs<T>(chunk(slot, u), v[u]);
            release(slot);
#pragma unroll
            for (int u = 0; u < CHT; ++u)
                if (q0 + u * CT < n16) {
#pragma unroll
                    for (int e = 0; e < H; ++e) v[u][e] = mul2(exp_pair(add2(v[u][e], nm), nl, l2e), f2);
                    store(q0 + u * CT, v[u], f0);
                }
        };
        if (MODE == kGrad) {
            const float m = mt.xa, lnS = mt.old, c0 = mt.w;
            for (int t = 0; t < nt; ++t, ++g) tile_gradient(await(g), t, m, lnS, c0);
            if (jht >= 0) store_ht(ht, m, lnS, c0);
            continue;
        }
        MaxSum ms = ms_empty();
        if (jht >= 0) ms.m = fmaxf(ms.m, ht);
        // tile t's exponentials against the running maximum into v, their sum into ms; absent
        // chunks of a row's last tile are skipped
        auto tile = [&](int t, uint64_t (&v)[CHT][H]) {
            const uint32_t slot = await(g + (uint32_t)t);
            const int q0 = t * CHT * CT + ct;
            float M = ms.m;
#pragma unroll
            for (int u = 0; u < CHT; ++u)
                if (q0 + u * CT < n16) {
                    unpack_pairs<T>(chunk(slot, u), v[u]);
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        float a, b;
                        unpack2(v[u][e], a, b);
                        M = max3(M, a, b);
                    }
                }
            release(slot);
            ms.s *= ex2((ms.m - M) * kLog2e);
            ms.m = M;
            const uint64_t nm = pack2(-M, -M);
            uint64_t s[2] = {};
#pragma unroll
            for (int u = 0; u < CHT; ++u)
                if (q0 + u * CT < n16) {
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        v[u][e] = exp_pair(v[u][e], nm, l2e);
                        s[e & 1] = add2(s[e & 1], v[u][e]);
                    }
                }
            float a, b;
            unpack2(add2(s[0], s[1]), a, b);
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
                uint64_t v[H];
                float M = ms.m;
#pragma unroll 1
                for (int u = 0; u < CHT && q0 + u * CT < n16; ++u) {
                    unpack_pairs<T>(chunk(slot, u), v);
#pragma unroll
                    for (int e = 0; e < H; ++e) {
                        float a, b;
                        unpack2(v[e], a, b);
                        M = max3(M, a, b);
                    }
                }
                ms.s *= ex2((ms.m - M) * kLog2e);
                ms.m = M;
                const uint64_t nm = pack2(-M, -M);
#pragma unroll 1
                for (int u = 0; u < CHT && q0 + u * CT < n16; ++u) {
                    unpack_pairs<T>(chunk(slot, u), v);
                    uint64_t s = 0;
#pragma unroll
                    for (int e = 0; e < H; ++e) s = add2(s, exp_pair(v[e], nm, l2e));
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
        if (jht >= 0) ms.s += ex2((ht - ms.m) * kLog2e);
        const MaxSum wm = warp_max_sum(ms);
        // The row's statistics: every warp's partial meets in warp 0, which settles the row and
        // hands (m, lnS, c) back.  Two buffers: a warp writes one again only after it has the
        // outcome of the row between, for which every warp (of every rank) has sent its partial,
        // each after it was done with this buffer.
        const uint32_t xb = nx & 1u, xpar = (nx >> 1) & 1u;
        ++nx;
        if (c > 1) {
            if (ct == 0) mbar_arrive_expect_tx(&S.xbar[xb], 8u * (uint32_t)(c * CW));
            if (lane < c)
                st_async_f32x2(map_to_rank(&S.xw[xb][rank * CW + cw], (uint32_t)lane), wm.m, wm.s,
                               map_to_rank(&S.xbar[xb], (uint32_t)lane));
        } else {
            if (lane == 0) S.part[xb][cw] = make_float2(wm.m, wm.s);
            if (cw != 0) named_arrive(2, CT);
        }
        if (cw == 0) {
            MaxSum tot;
            if (c > 1) {
                wait_parity<true>(&S.xbar[xb], xpar, &S.abort, &g_watchdog);
                tot = combine_parts(S.xw[xb], c * CW, lane);
            } else {
                named_sync(2, CT);
                const int l = lane & 15;
                const float2 q = l < CW ? S.part[xb][l] : make_float2(-FLT_MAX, 0.f);
                tot.m = warp_max(q.x);
                tot.s = q.y * ex2((q.x - tot.m) * kLog2e);
#pragma unroll
                for (int off = 8; off > 0; off >>= 1) tot.s += __shfl_xor_sync(0xffffffffu, tot.s, off);
            }
            const float l = logf(tot.s);
            const float f = settle_row<MODE>(P, r, mt.w, mt.old, mt.ref, mt.adv, mt.xa, tot.m, l, rank == 0 && lane == 0);
            if (lane == 0) S.row[xb] = make_float4(tot.m, l, f, 0.f);
        }
        named_sync(1, CT);
        if (MODE == kLogp) continue;
        const float m = S.row[xb].x, lnS = S.row[xb].y, f0 = S.row[xb].z;
        for (int t = RTILES; t < nt; ++t) {
            const uint32_t slot = (g0 + (uint32_t)t) % SLOTS;
            if (gr) {
                const uint64_t nm = pack2(-m, -m), nl = pack2(-lnS, -lnS), f2 = pack2(-f0, -f0);
                const int q0 = t * CHT * CT + ct;
#pragma unroll 1
                for (int u = 0; u < CHT && q0 + u * CT < n16; ++u) {
                    uint64_t v[H];
                    unpack_pairs<T>(chunk(slot, u), v);
#pragma unroll
                    for (int e = 0; e < H; ++e) v[e] = mul2(exp_pair(add2(v[e], nm), nl, l2e), f2);
                    store(q0 + u * CT, v, f0);
                }
            }
            release(slot);
        }
        if (!gr) continue;
#pragma unroll
        for (int t = 0; t < RTILES; ++t)
            if (t < nt) {
                const float f = f0 == 0.f ? 0.f : -f0 * ex2(((mx[t] - m) - lnS) * kLog2e);
                const uint64_t f2 = pack2(f, f);
                const int q0 = t * CHT * CT + ct;
#pragma unroll
                for (int u = 0; u < CHT; ++u)
                    if (q0 + u * CT < n16) {
#pragma unroll
                        for (int e = 0; e < H; ++e) E[MODE == kPolicy ? t : 0][u][e] = mul2(E[MODE == kPolicy ? t : 0][u][e], f2);
                        store(q0 + u * CT, E[MODE == kPolicy ? t : 0][u], f0);
                    }
            }
        if (jht >= 0) store_ht(ht, m, lnS, f0);
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
            mbar_init(&S.mempty[b], CW);
            mbar_init(&S.xbar[b], 1);
        }
        S.abort = 0;
        fence_mbar_init_cluster();
    }
    if (c > 1) cluster_sync_all();
    else __syncthreads();
    pdl_wait_primary();
    pdl_launch_dependents();
    if (threadIdx.x >= CT) ring_producer<T, MODE>(P, S, rank, c, cid, ncl);
    else ring_consumer<T, MODE>(P, S, rank, c, cid, ncl);
    __syncwarp();
    if (c > 1) cluster_sync_all();       // no CTA may leave while a peer can still write to it
}

// ---------------------------------------------------------------- pairs

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
        cfg.gridDim = dim3((unsigned)(c * sms), 1, 1);
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
    if (P.V <= 2048) return launch_pdl(rows_direct<T, MODE, 128, 16 / N>, grid, 128, st, P);
    if (P.V <= 8192) return launch_pdl(rows_direct<T, MODE, 256, 32 / N>, grid, 256, st, P);
    if (MODE == kPolicy && P.V > VL_POLICY_ONEPASS_COLS) return launch_pdl(rows_twice<T>, grid, NT, st, P);
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
