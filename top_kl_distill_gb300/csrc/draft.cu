// Verification of drafted tokens against the target's probabilities (sm_103a).
//
// A sequence brings k drafted tokens d_0 .. d_(k-1), the drafter's rows of logits they were drawn from, and k + 1 rows
// of the target's.  With p_j, q_j the softmax of row j at the sequence's temperature: d_j is accepted while
// u_j q_j(d_j) < p_j(d_j); at the first token refused the next one is drawn from max(p_j - q_j, 0), after k
// accepted ones from p_k: the first column whose running sum exceeds pick * total.  The tokens are then
// distributed as the target's own, whatever the drafter.
//
// HBM bound: a row is read once for its (max, sum of exponentials); the refused row's two rows once more, from L2.
// A cluster of CTAs takes a sequence: its warps share out the rows' segments (1024 columns or more) in pieces of 2 KB, each piece in
// registers between the maximum and the sum, with the next one's loads under way, and send each segment's (max, sum) to
// every CTA of the cluster; after one cluster barrier all CTAs hold the same partials and come to the same
// decision.  A sweep takes `per` positions at once, two to four, or eight where rows are short (see `verify_go`), so up to
// seven rows after the first refused one are read too; they never matter.  The partials are by column, not by CTA, so a row's
// statistics and its draw do not depend on the cluster's size or on the other sequences, but for the place within 16 bytes at
// which the row begins: chunks, and with them the order of the sums, are aligned where the row is.
//
// Statistics are in units of log2: m2 is the largest x sc, sc = log2(e) / temperature, rounded to fp32, and only a
// reference: with x sc - m2 in one fma (its error is half an ulp of the difference, nothing near the top) the sums are
// right relative to it whatever it was rounded by.  It would have to be off by 2^126 to lose them: x sc near 2^32.  So a
// reference is never below kLow: where a lane's columns are all masked, by -inf or by a number as low as the type has, each
// is nothing next to it.  A row without anything else has the sum 0, and no softmax.
//
// 256 sequences of 8 drafted tokens over 128256 bf16 columns: 130 us, 546 MB read (4.2 TB/s; 490 MB are the rows that count);
// 32 of 5: 27 us; one of 4 over 32000 fp32: 9.7.  A sweep's end (cluster barrier, decision) is 2 to 3 us in which its CTAs
// read nothing, the draw 5; the four CTAs of an SM hide that from one another where there are enough, and the longest sequences
// run on alone.  Tried: the next sweep's rows brought into L2 ahead (27 to 30 us, 130 to 143), its
// first pieces loaded before the barrier (27.3 to 28.4, 129 to 133: the barrier waits for them), clusters of 16 CTAs (one
// sequence 9.3 to 8.2 us, but 32 of them 31 to 39).
#include "vl_api.h"
#include "vl_device.cuh"
#include "vl_fp4.h"
#include "vl_internal.h"
#include "vl_pair.cuh"
#include "vl_rowio.cuh"
#include "vl_tc.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>

namespace vl {
namespace {

constexpr int SEG = 1024;                // columns of a segment, or a multiple where rows are long
constexpr int MAX_SEGS = 64;
constexpr int MAX_PER = 8;               // positions a sweep
constexpr int ROWS = 2 * MAX_PER + 1;
constexpr uint32_t kNone = 0xffffffffu;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLow = -2147483648.f;    // half an ulp of what is above is 64 at most
constexpr float kNever = -745.f;         // ln of a probability that is 0 in 64 bits too

struct Smem {
    float2 part[2][ROWS][MAX_SEGS];      // (m2, sum of 2^(x sc - m2)) of a segment; by sweep, in turn
    uint2 top[2][MAX_PER + 1][MAX_SEGS]; // its largest value and where (greedy: the target's rows)
    float sum[MAX_SEGS];                 // weights of the draw, by segment
    float wsum[16];                      // and of the warps' columns of the segment drawn
    double goal;                         // of the draw, within that segment
    int pick_seg, whole;
    uint2 hits[16];                      // a warp's first column past the goal; its last with a weight, + 1
    float xd[2][MAX_PER], yd[2][MAX_PER], u[2][MAX_PER];       // logits of the drafted tokens, random numbers
    uint32_t tok[2][MAX_PER];
    float rm[ROWS], rz[ROWS];            // rows' statistics, as the segments'
    int rat[ROWS];
    int run, ended, bad;                 // accepted in this sweep; how the sequence ends in it; a token past the vocabulary
};

// The two halves of cluster_sync_all.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_remote(uint32_t addr, uint32_t v) {
    asm volatile("st.shared::cluster.b32 [%0], %1;" :: "r"(addr), "r"(v) : "memory");
}

// Four 16-byte chunks a lane, 2 KB a warp: chunk-row i holds columns c0 + (32 i + lane) N and on.
template <typename T>
struct Piece {
    static constexpr int N = Pack<T>::N, COLS = 128 * N;
    uint4 r[4];
    static __device__ __forceinline__ int col(int c0, int i, int lane) { return c0 + (i * 32 + lane) * N; }
    // one chunk-row, as floats
    static __device__ __forceinline__ void row_of(const T* p, int c0, int V, int lane, bool chunks, float (&f)[N]) {
        const int c = c0 + lane * N;
        if (chunks && c >= 0 && c + N <= V) {
            Pack<T>::unpack(*reinterpret_cast<const uint4*>(p + c), f);
        } else {
#pragma unroll
            for (int j = 0; j < N; ++j) f[j] = c + j >= 0 && c + j < V ? ld_elem(p + c + j) : -INFINITY;
        }
    }
    // c0 such that chunks are aligned where the row is; -inf outside [0, V).  `chunks`: rows that can be read by chunks.
    __device__ __forceinline__ void load(const T* p, int c0, int V, int lane, bool chunks) {
        if (chunks && c0 >= 0 && c0 + COLS <= V) {
#pragma unroll
            for (int i = 0; i < 4; ++i) r[i] = *reinterpret_cast<const uint4*>(p + col(c0, i, lane));
            return;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int c = col(c0, i, lane);
            if (chunks && c >= 0 && c + N <= V) {
                r[i] = *reinterpret_cast<const uint4*>(p + c);
            } else if (c + N <= 0 || c >= V) {
                r[i] = sizeof(T) == 2 ? make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u)
                                      : make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
            } else {
                float f[N];
                row_of(p, c0 + i * 32 * N, V, lane, chunks, f);
                r[i] = Pack<T>::pack(f);             // exact: the values are of this type
            }
        }
    }
    // the largest value of the lane's (NaN left out)
    __device__ __forceinline__ float top() const {
        if constexpr (sizeof(T) == 2) {
            const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(r);
            __nv_bfloat162 m = h[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) m = __hmax2(m, h[i]);
            return fmaxf(__low2float(m), __high2float(m));
        } else {
            float m = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m = fmaxf(fmaxf(fmaxf(__uint_as_float(r[i].x), __uint_as_float(r[i].y)), fmaxf(__uint_as_float(r[i].z), __uint_as_float(r[i].w))), m);
            return m;
        }
    }
    // 2^(x sc - m2) of chunk-row i
    __device__ __forceinline__ void exps(int i, float m2, float sc, float (&e)[N]) const {
        Pack<T>::unpack(r[i], e);
#pragma unroll
        for (int j = 0; j < N; ++j) e[j] = ex2(fmaf(e[j], sc, -m2));
    }
    __device__ __forceinline__ float sum_exps(float m2, float sc) const {
        uint64_t s[2] = {0, 0};
        const uint64_t nm = both(-m2), sc2 = both(sc);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float f[N];
            Pack<T>::unpack(r[i], f);
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                float a, b;
                unpack2(fma2(pack2(f[2 * j], f[2 * j + 1]), sc2, nm), a, b);
                s[j & 1] = add2(s[j & 1], pack2(ex2(a), ex2(b)));
            }
        }
        return sum2(add2(s[0], s[1]));
    }
    // the lane's lowest column that holds v
    __device__ __forceinline__ int find(float v, int c0, int lane) const {
        int at = 0x7fffffff;
#pragma unroll
        for (int i = 3; i >= 0; --i) {
            float f[N];
            Pack<T>::unpack(r[i], f);
#pragma unroll
            for (int j = N - 1; j >= 0; --j) at = f[j] == v ? col(c0, i, lane) + j : at;
        }
        return at;
    }
};

template <typename T>
__device__ __forceinline__ int shift_of(const T* row) { return (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T)); }

template <typename T, int WARPS>
__global__ void __launch_bounds__(32 * WARPS, 32 / WARPS) verify(const VerifyParams P, int csize, int per, int seg, int nseg) {
    using Pc = Piece<T>;
    constexpr int N = Pc::N;
    extern __shared__ uint8_t raw[];
    Smem& S = *reinterpret_cast<Smem*>(raw);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int rank = csize > 1 ? (int)cluster_ctarank() : 0;
    const long long seq = blockIdx.x / csize;
    pdl_launch_dependents();
    cluster_arrive();                    // (waited for before another CTA's memory is first written)
    pdl_wait_primary();
    const int V = P.V, warps = csize * WARPS, gw = warp * csize + rank, pieces = seg / Pc::COLS;
    const long long s0 = min(max(P.start[seq], 0ll), P.nd), s1 = min(max(P.start[seq + 1], s0), P.nd);
    const long long k = s1 - s0, t0 = s0 + seq;        // drafted tokens; the target's first row
    const float heat = P.heat ? P.heat[seq] : 1.f;
    const float pick = P.pick[seq];
    const bool greedy = heat == 0.f, sane = greedy || (heat >= 1e-6f && heat <= 1e6f);
    const float sc = greedy || !sane ? kLog2e : kLog2e / heat;
    const bool with_q = P.draft != nullptr && !greedy;
    const T* const target = static_cast<const T*>(P.target);
    const T* const draft = static_cast<const T*>(P.draft);

    const bool scout = warp == WARPS - 1 && rank == csize - 1;
    uint32_t tok_ahead = 0;
    float u_ahead = 0.f;
    if (scout && lane < per && lane < k) {
        tok_ahead = P.drafted[s0 + lane];
        u_ahead = P.u[s0 + lane];
    }
    long long j0 = 0;
    int buf = 0, np = 0;
    bool started = false;                // every CTA of the cluster runs: its memory may be written
    bool refused = false, failed = false;
    for (;; buf ^= 1) {
        np = (int)min((long long)per, k + 1 - j0);                     // the target's rows of this sweep
        const int nd = (int)min((long long)per, k - j0), nq = with_q ? nd : 0;
        // what the decision needs besides the statistics, read once, for all CTAs: the tokens and random numbers a sweep
        // ahead, since their logits' addresses hang on them
        float x = 0.f, y = 0.f, u = 0.f;
        uint32_t d = 0;
        if (scout) {
            d = tok_ahead;
            u = u_ahead;
            if (lane < nd && d < (uint32_t)V) {
                x = ld_elem(target + (t0 + j0 + lane) * P.ldt + d);
                if (with_q) y = ld_elem(draft + (s0 + j0 + lane) * P.ldd + d);
            }
            if (lane < per && j0 + per + lane < k) {
                tok_ahead = P.drafted[s0 + j0 + per + lane];
                u_ahead = P.u[s0 + j0 + per + lane];
            }
        }
        // rows 0 .. np - 1 are the target's, then the drafter's
        auto row_of = [&](int r) { return r < np ? target + (t0 + j0 + r) * P.ldt : draft + (s0 + j0 + r - np) * P.ldd; };
        int r = gw / nseg, g = gw - r * nseg;
        if (r < np + nq) {
            Pc a, b;
            int pc = 0;
            const T* row = row_of(r);
            int c0 = g * seg - shift_of(row);
            a.load(row, c0, V, lane, true);
            float m2 = kLow, z = 0.f, top = -INFINITY;
            int at = 0x7fffffff;
            // One piece, the next one's loads before its arithmetic.  The two take turns by name: a copy would wait for the
            // loads (151 us against 131 for 256 sequences of 8 over 128256 bf16 columns).
            auto step = [&](const Pc& cur, Pc& next) {
                const bool last = ++pc == pieces;
                const int here_r = r, here_g = g, here_c0 = c0;
                c0 += Pc::COLS;
                if (last) {
                    pc = 0;
                    g += warps;
                    if (g >= nseg) {
                        do {
                            g -= nseg;
                            ++r;
                        } while (g >= nseg);
                        if (r < np + nq) row = row_of(r);
                    }
                    c0 = g * seg - shift_of(row);
                }
                const bool more = r < np + nq;
                if (more) next.load(row, c0, V, lane, true);
                if (!started) {
                    cluster_wait();
                    started = true;
                }
                const float t = cur.top();
                if (greedy && t > top) {
                    at = cur.find(t, here_c0, lane);
                    top = t;
                }
                const float nm = fmaxf(m2, t * sc);
                z = z * ex2(m2 - nm) + cur.sum_exps(nm, sc);
                m2 = nm;
                if (last) {
                    const float all = warp_max(m2);
                    z = warp_sum(z * ex2(m2 - all));
                    if (lane < csize) st_cluster_f32x2(map_to_rank(&S.part[buf][here_r][here_g], lane), all, z);
                    if (greedy) {
                        const float high = warp_max(top);
                        at = __reduce_min_sync(0xffffffffu, top == high ? at : 0x7fffffff);
                        if (lane < csize) st_cluster_f32x2(map_to_rank(&S.top[buf][here_r][here_g], lane), high, __int_as_float(at));
                        top = -INFINITY;
                        at = 0x7fffffff;
                    }
                    m2 = kLow;
                    z = 0.f;
                }
                return more;
            };
            while (step(a, b) && step(b, a)) {
            }
        }
        if (!started) {
            cluster_wait();
            started = true;
        }
        if (scout && lane < nd)
            for (int c = 0; c < csize; ++c) {
                st_remote(map_to_rank(&S.xd[buf][lane], c), __float_as_uint(x));
                st_remote(map_to_rank(&S.yd[buf][lane], c), __float_as_uint(y));
                st_remote(map_to_rank(&S.u[buf][lane], c), __float_as_uint(u));
                st_remote(map_to_rank(&S.tok[buf][lane], c), d);
            }
        cluster_sync_all();
        for (int r = warp; r < np + nq; r += WARPS) {
            float m2 = kLow, z = 0.f;
            for (int g = lane; g < nseg; g += 32) m2 = fmaxf(m2, S.part[buf][r][g].x);
            m2 = warp_max(m2);
            for (int g = lane; g < nseg; g += 32) {
                const float2 p = S.part[buf][r][g];
                z += p.y * ex2(p.x - m2);
            }
            z = warp_sum(z);
            if (lane == 0) {
                S.rm[r] = m2;
                S.rz[r] = z;
            }
            if (greedy) {
                float high = -INFINITY;
                int at = 0x7fffffff;
                for (int g = lane; g < nseg; g += 32) {
                    const uint2 p = S.top[buf][r][g];
                    if (__uint_as_float(p.x) > high) {
                        high = __uint_as_float(p.x);
                        at = (int)p.y;
                    }
                }
                const float all = warp_max(high);
                at = __reduce_min_sync(0xffffffffu, high == all ? at : 0x7fffffff);
                if (lane == 0) S.rat[r] = at;
            }
        }
        __syncthreads();
        if (warp == 0) {
            // a lane a position: 0 accepted, 1 refused, 2 the row after the last drafted token, 3 no statistics
            int verdict = 0;
            float lp = 0.f;
            if (lane < np) {
                const float m = S.rm[lane], z = S.rz[lane];
                bool fine = sane && z > 0.f && z < INFINITY;
                if (j0 + lane >= k) {
                    verdict = 2;
                } else {
                    const uint32_t d = S.tok[buf][lane];
                    const float x = S.xd[buf][lane];
                    const float x2 = fmaf(x, sc, -m);            // log2 p = x2 - log2 z
                    lp = (x2 - __log2f(z)) * kLn2;
                    if (greedy) {
                        verdict = d == (uint32_t)S.rat[lane] ? 0 : 1;
                    } else {
                        float ratio;
                        if (with_q) {
                            const float qm = S.rm[np + lane], qz = S.rz[np + lane];
                            fine = fine && qz > 0.f && qz < INFINITY;
                            ratio = ex2(x2 - fmaf(S.yd[buf][lane], sc, -qm)) * (qz / z);
                        } else {
                            ratio = ex2(x2) / z;
                        }
                        // where p is 0 the ratio does not count (it may be one of two masks); u = 0 is below any other p
                        const float u = S.u[buf][lane];
                        verdict = lp > kNever && (u < ratio || u == 0.f) ? 0 : 1;
                    }
                    if (d >= (uint32_t)V) verdict = 1;
                }
                if (!fine) verdict = 3;
            }
            const uint32_t stop = __ballot_sync(0xffffffffu, lane < np && verdict != 0);
            const int run = stop ? __ffs(stop) - 1 : np;
            const int how = __shfl_sync(0xffffffffu, verdict, run < 32 ? run : 0);
            if (lane == 0) {
                S.run = run;
                S.ended = stop ? how : 0;
                S.bad = stop && how == 1 && S.tok[buf][run] >= (uint32_t)V;
            }
            if (rank == 0 && lane < run) {
                P.tokens[t0 + j0 + lane] = S.tok[buf][lane];
                if (P.logp) P.logp[t0 + j0 + lane] = lp;
            }
        }
        __syncthreads();
        const int ended = S.ended;
        j0 += S.run;
        refused = ended == 1;
        failed = ended == 3;
        if (ended) break;
    }
    // the row that the next token is drawn from: row S.run of the last sweep
    const int r = S.run;
    const float m = S.rm[r], z = S.rz[r], inv = 1.f / z;
    const bool residual = refused && with_q;
    const float qm = residual ? S.rm[np + r] : 0.f, qinv = residual ? 1.f / S.rz[np + r] : 0.f;
    const T* const row = target + (t0 + j0) * P.ldt;
    const T* const qrow = residual ? draft + (s0 + j0) * P.ldd : nullptr;
    const int shift = shift_of(row);
    const bool same = residual && shift == shift_of(qrow);
    // refused without a q: left out of the draw
    const int out = refused && !greedy && !P.draft && S.tok[buf][r] < (uint32_t)V ? (int)S.tok[buf][r] : -1;
    const bool draws = !failed && !greedy;
    // weights of chunk-row i of a piece of the target's row and one of the drafter's: p - q where positive, or (plain) p without
    // the token left out
    auto weights = [&](const Pc& a, const Pc& b, int i, int c0, bool plain, float (&w)[N]) {
        float q[N];
        a.exps(i, m, sc, w);
        if (!plain) b.exps(i, qm, sc, q);
#pragma unroll
        for (int j = 0; j < N; ++j) {
            w[j] *= inv;
            if (!plain) w[j] = fmaxf(w[j] - q[j] * qinv, 0.f);
            if (Pc::col(c0, i, lane) + j == out) w[j] = 0.f;
        }
    };
    auto segment_sum = [&](int g, bool plain) {
        float s = 0.f;
        for (int pc = 0; pc < pieces; ++pc) {
            const int c0 = g * seg + pc * Pc::COLS - shift;
            Pc a, b;
            a.load(row, c0, V, lane, true);
            if (!plain) b.load(qrow, c0, V, lane, same);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float w[N];
                weights(a, b, i, c0, plain, w);
#pragma unroll
                for (int j = 0; j < N; ++j) s += w[j];
            }
        }
        return warp_sum(s);
    };
    if (draws && residual) {
        for (int g = gw; g < nseg; g += warps) {
            const float s = segment_sum(g, false);
            if (lane == 0) st_remote(map_to_rank(&S.sum[g], 0), __float_as_uint(s));
        }
        cluster_sync_all();
    }
    if (rank != 0) return;
    // the rest is the first CTA's: the segment, by one warp; the column, all warps side by side
    uint32_t token = kNone;
    if (greedy && !failed) token = (uint32_t)S.rat[r];
    if (draws) {
        // without a drafter's row the weights of the segments are there already
        if (!residual && warp == 0) {
            for (int g = lane; g < nseg; g += 32) {
                const float2 p = S.part[buf][r][g];
                S.sum[g] = p.y * ex2(p.x - m) * inv;
            }
            __syncwarp();
            if (out >= 0) {
                const int g = (out + shift) / seg;
                const float s = segment_sum(g, true);
                if (lane == 0) S.sum[g] = s;
                __syncwarp();
            }
        }
        if (warp == 0) {
            // a lane's neighbouring segments, then the lanes: sums in 64 bits
            const int own = (nseg + 31) / 32;
            double s = 0.0;
            for (int i = 0; i < own; ++i) s += lane * own + i < nseg ? (double)S.sum[lane * own + i] : 0.0;
            double incl = s;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            const double total = __shfl_sync(0xffffffffu, incl, 31), goal = (double)pick * total;
            // the first segment past the goal that has a weight; rounding at the end: the last one
            const uint32_t past = __ballot_sync(0xffffffffu, s > 0.0 && incl > goal), some = __ballot_sync(0xffffffffu, s > 0.0);
            const int at = past ? __ffs(past) - 1 : some ? 31 - __clz(some) : 0;
            double before = 0.0, upto = incl - s;
            int g1 = 0;
            for (int i = 0; i < own; ++i) {
                const int g = lane * own + i;
                const double w = g < nseg ? (double)S.sum[g] : 0.0;
                if (w > 0.0) {
                    g1 = g;
                    before = upto;
                    upto += w;
                    if (upto > goal) break;
                }
            }
            if (lane == at) {
                S.pick_seg = g1;
                S.goal = fmax(goal - before, 0.0);
                S.whole = !(total > 0.0);          // nothing is left (p and q alike, p all on the token refused): drawn from p
            }
        }
        __syncthreads();
        const bool whole = S.whole != 0;
        const int g0 = whole ? 0 : S.pick_seg, g1 = whole ? nseg : g0 + 1;
        const float want = whole ? pick : (float)S.goal;
        // chunk-rows of 32 x N columns, one a warp; the warps' sums in a row
        float cum = 0.f;
        for (int c00 = g0 * seg - shift; c00 < g1 * seg - shift && c00 < V; c00 += WARPS * 32 * N) {
            const int c0 = c00 + warp * 32 * N;
            float w[N];
            const bool in = c0 < g1 * seg - shift;
            Pc::row_of(row, c0, V, lane, true, w);
#pragma unroll
            for (int j = 0; j < N; ++j) w[j] = ex2(fmaf(w[j], sc, -m)) * inv;
            if (residual && !whole) {
                float q[N];
                Pc::row_of(qrow, c0, V, lane, same, q);
#pragma unroll
                for (int j = 0; j < N; ++j) w[j] = fmaxf(w[j] - ex2(fmaf(q[j], sc, -qm)) * qinv, 0.f);
            }
            float e = 0.f;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                if (!in || (c0 + lane * N + j == out && !whole)) w[j] = 0.f;
                e += w[j];
            }
            float incl = e;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const float up = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += up;
            }
            if (lane == 31) S.wsum[warp] = incl;
            __syncthreads();
            // this warp's first column past the goal, and its last one with a weight
            float run = cum;
            for (int v = 0; v < WARPS; ++v) {
                run += v < warp ? S.wsum[v] : 0.f;
                cum += S.wsum[v];
            }
            run += incl - e;
            uint32_t mine = kNone, any = kNone;
#pragma unroll
            for (int j = 0; j < N; ++j) {
                run += w[j];
                if (w[j] > 0.f) {
                    any = (uint32_t)(c0 + lane * N + j);
                    if (mine == kNone && run > want) mine = any;
                }
            }
            const uint32_t first = __reduce_min_sync(0xffffffffu, mine), last = __reduce_max_sync(0xffffffffu, any + 1u);
            if (lane == 0) S.hits[warp] = make_uint2(first, last);
            __syncthreads();
            uint32_t hit = kNone, has = 0;
            for (int v = 0; v < WARPS; ++v) {
                hit = min(hit, S.hits[v].x);
                has = max(has, S.hits[v].y);
            }
            if (has) token = has - 1u;
            if (hit != kNone) {
                token = hit;
                break;
            }
            __syncthreads();
        }
    }
    if (warp != 0) return;
    if (lane == 0) {
        if (P.err && (failed || S.bad)) atomicAdd(P.err, 1);
        P.accepted[seq] = (int)j0;
        P.tokens[t0 + j0] = token;
        if (P.logp) P.logp[t0 + j0] = token != kNone ? (fmaf(ld_elem(row + token), sc, -m) - __log2f(z)) * kLn2 : 0.f;
    }
    for (long long i = j0 + 1 + lane; i <= k; i += 32) {
        P.tokens[t0 + i] = kNone;
        if (P.logp) P.logp[t0 + i] = 0.f;
    }
}

template <typename T, int WARPS>
cudaError_t verify_launch(const VerifyParams& P, int csize, int per, int dev, cudaStream_t st) {
    static std::atomic<int> had[64];
    if (!had[dev].load(std::memory_order_acquire)) {
        const cudaError_t e = cudaFuncSetAttribute((const void*)verify<T, WARPS>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem));
        if (e != cudaSuccess) return e;
        had[dev].store(1, std::memory_order_release);
    }
    const long long cols = (long long)P.V + Pack<T>::N - 1, segs = (cols + SEG - 1) / SEG;
    const int seg = (int)((segs + MAX_SEGS - 1) / MAX_SEGS) * SEG, nseg = (int)((cols + seg - 1) / seg);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(P.nseq * csize), 1, 1);
    cfg.blockDim = dim3(32 * WARPS, 1, 1);
    cfg.dynamicSmemBytes = sizeof(Smem);
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)csize;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify<T, WARPS>, P, csize, per, seg, nseg);
}

template <typename T>
cudaError_t verify_go(const VerifyParams& P, cudaStream_t st) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int sms = num_sms();
    if (dev < 0 || dev >= 64 || sms <= 0) return cudaErrorInvalidDevice;
    // Positions a sweep: reading on past a refused token costs bytes, each sweep some 4 us of latency.  As many as are
    // read in that time (a cluster reads some 0.45 TB/s, all of them 6.5), 2 to 4, or 8 where rows are next to nothing
    // (7 sequences of 8 over 1447 fp32 columns: 13.4 us by 4, 9.2 by 8).
    const double rate = std::min(6.5e6, 0.45e6 * (double)P.nseq), bytes = (double)P.nseq * P.V * sizeof(T) * (P.draft ? 2 : 1);
    const double each = bytes / rate;
    const int per = each < 0.25 ? MAX_PER : (int)std::max(2.0, std::min(4.0, 4.0 / each + 1.0));
    // Warps a sequence: those that fill the GPU together (32 an SM), but for long rows, where a sequence takes long and
    // the last one alone even longer, no fewer than one for two pieces of 2 KB of a row; and no more than a sweep has pieces.
    // 256 sequences of up to 5 over 32000 bf16 columns: 16 warps 41 us, 32 45, 128 78; 256 of up to 8 over 128256: 64 warps
    // 129 us, 32 132, 16 211; 32 of up to 5: 128 27 us, 64 33.
    const long long pieces = ((long long)P.V + Piece<T>::COLS - 1) / Piece<T>::COLS, sweep = pieces * per * (P.draft ? 2 : 1);
    const long long want = std::min(sweep, std::max(32ll * sms / P.nseq, std::min(64ll, (pieces + 2) / 2)));
    int warps = 8;
    while (warps < 128 && 2 * warps <= want) warps *= 2;
    const int csize = warps > 64 ? 8 : warps / 8;       // 8: the largest cluster that every part of a GPU holds
    return warps <= 64 ? verify_launch<T, 8>(P, csize, per, dev, st) : verify_launch<T, 16>(P, csize, per, dev, st);
}

}  // namespace

cudaError_t launch_verify(const VerifyParams& P, int dtype, cudaStream_t st) {
    return dtype == kBf16 ? verify_go<__nv_bfloat16>(P, st) : verify_go<float>(P, st);
}

}  // namespace vl
