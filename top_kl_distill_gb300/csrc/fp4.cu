// The product in 4-bit floating point (sm_103a): D[m][n] = alpha ra[m] rb[n] sum_k sfa sfb A[m][k] B[n][k], A and B
// e2m1 with a scale for each 16 (NV) or 32 (MX) columns.
//
// The tensor cores multiply by the blocks' scales themselves (tcgen05.mma ... block_scale), so a tile's whole sum
// stays in tensor memory and the epilogue meets it once.  They take the scales from tensor memory: 512
// bytes, 128 rows x 4 blocks, go there in one tcgen05.cp, which is the order in which the quantiser leaves them.
//
// The weight's rows (B) are the tensor cores' 128 lanes, the hidden rows (A) their columns (D^T = B A^T): a
// lane of the epilogue then is a column of D, and each store of a warp one contiguous piece of a row.
//
// Up to 64 rows `fp4_gemm`: the weight plane is what has to be read; its 128-row tiles stream through two CTAs an SM (8 x
// 128256 x 4096 with its quantiser 48 us, 0.91 of the copy rate).  Per CTA: warp 0 the TMA producer (128 bytes = 256 columns
// of K a stage, 128-byte swizzle, and that stage's scales), warp 1 the scales' copies and the MMAs (into one of two accumulators),
// warps 2-5 the epilogue.  What was tried to bring the weights earlier made it slower: rows prefetched into L2 by 512 bytes to
// 2 KB (8 x 32000 x 4096: 15.2 to 21 us), tiles 8 to 16 stages ahead (8 x 128256 x 4096: 53 to 70 us).  Above 64 rows:
// `fp4_gemm_pairs`.
#include "vl_api.h"
#include "vl_device.cuh"
#include "vl_fp4.h"
#include "vl_internal.h"
#include "vl_launch.h"
#include "vl_pair.cuh"
#include "vl_rowio.cuh"
#include "vl_tc.cuh"

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

namespace vl {
namespace {

__device__ unsigned int g_watchdog;

constexpr int KB = 128;                  // bytes of a row a stage
constexpr int KE = 2 * KB;               // columns of K a stage
constexpr int SF_TILE = 512;             // 128 rows x 4 blocks of scales
template <int FMT>
constexpr int SF_TILES = FMT == kNv ? 4 : 2;                // tiles of scales a stage and 128 rows

// wait_parity by a whole warp: all lanes agree on whether it gave up.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, int* abort) {
    return __all_sync(0xffffffffu, wait_parity<false>(bar, parity, abort, &g_watchdog));
}

// Instruction descriptor: A, B e2m1 (bits 7-9, 10-12 = 1), N >> 3, scales e4m3 or e8m0 (bit 23), M >> 4; K = 64.
// Which bytes of a scale column an MMA takes (bits 4-5 for B, 29-30 for A): all four for blocks of 16, two for 32.
template <int FMT>
constexpr uint32_t idesc(int M, int N, int id = 0) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(FMT == kMx) << 23) | ((uint32_t)(M >> 4) << 24) |
           ((uint32_t)id << 4) | ((uint32_t)id << 29);
}

// A tile of scales in shared memory: 32 rows of 16 bytes, groups of 8 rows 128 bytes apart, no swizzle.
__device__ __forceinline__ uint64_t sf_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(16 >> 4) << 16 | (uint64_t)(128 >> 4) << 32 | (uint64_t)1 << 46;
}

// 512 bytes into four columns of tensor memory, the same in each quarter of the lanes (G = 2: in both CTAs of a pair,
// each from its own shared memory).
template <int G>
__device__ __forceinline__ void sf_copy(uint32_t taddr, uint64_t desc) {
    if constexpr (G == 1) asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" :: "r"(taddr), "l"(desc) : "memory");
}

#define VL_MMA_FP4(GROUP, KIND, VEC)                                                                                       \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                         \
                 "tcgen05.mma.cta_group::" GROUP ".kind::" KIND ".block_scale.scale_vec::" VEC                             \
                 " [%0], %1, %2, %3, [%4], [%5], p;\n\t}"                                                                  \
                 :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(id), "r"(sa), "r"(sb), "r"(acc) : "memory")

// G CTAs' MMA of K = 64; sa, sb: the scales' columns.
template <int G, int FMT>
__device__ __forceinline__ void mma_fp4(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t id, uint32_t sa, uint32_t sb,
                                        uint32_t acc) {
    if constexpr (G == 1 && FMT == kNv) VL_MMA_FP4("1", "mxf4nvf4", "4X");
    else if constexpr (G == 1) VL_MMA_FP4("1", "mxf4", "2X");
    else if constexpr (FMT == kNv) VL_MMA_FP4("2", "mxf4nvf4", "4X");
    else VL_MMA_FP4("2", "mxf4", "2X");
}
#undef VL_MMA_FP4

struct GemmParams {
    const uint8_t* sfw;       // scales of the weight's rows
    const uint8_t* sfx;       // and of the hidden rows
    const float* rw;          // row scales (NV)
    const float* rx;
    void* d;
    int bf16, pairs;          // bf16 out; its rows can be written two columns at a time
    long long ldd;
    int M, N;                 // hidden rows, weight rows
    int nk, tiles_k;          // stages; tiles of scales along K
    int mmas;                 // MMAs of 64 columns that K takes
    int splits;               // parts that K is taken in, by the CTAs (pairs) of a cluster: each has one tile then
    float alpha, am;          // alpha = am 2^ea
    int ea;
};

// A lane's factors: D = ((v p) rx) q, v the sum (0, or 2^-20 to 2^53 in NV), rx the scale of a row of A, p q = rb alpha.
// With p = 1 nothing on the way leaves fp32 that the result does not, if all rx are in 2^-64 to 2^64 and rb alpha is in fp32.
// Where a row's is not (a product is `far` then) or a lane's is not, q is a power of two that leaves p in 2^-100 to 2^71: then
// neither v p nor that times rx does.  (In fp64 on a path of their own such tiles cost the others 1 to 8%: whatever stands beside
// the epilogue's one path makes it slower.  A second factor for the rows too, beside theirs in shared memory: 2 to 5%.)
struct Lane {
    float p, q;
};
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(127 + e) << 23); }
__device__ __forceinline__ bool beyond(float rx) {
    const float a = fabsf(rx);
    return (a > 0.f && a < 5.421010862427522e-20f) || (a > 1.8446744073709552e19f && a < INFINITY);
}
// alpha = am 2^ea
__device__ __forceinline__ Lane lane_scale(float rn, float alpha, float am, int ea, bool far) {
    const float s = rn * am;
    const int e = (int)(__float_as_uint(s) >> 23 & 255u) - 127 + ea, k = e > 70 ? min(e - 70, 126) : e < -100 ? max(e + 100, -126) : 0;
    const int half = (ea - k) / 2;
    return far || e > 120 || e < -120 ? Lane{s * pow2(half) * pow2(ea - k - half), pow2(k)} : Lane{1.f, rn * alpha};
}

// Arithmetic on a loaded value stays behind this place, where it may wait for the load.
__device__ __forceinline__ void hold(float& r) { asm volatile("" : "+f"(r)); }

// Sixteen columns of the accumulator, scaled; rx in shared memory.
__device__ __forceinline__ void scale16(float (&y)[16], const uint32_t (&v)[16], const float* rx, Lane s) {
    const uint64_t p = both(s.p), q = both(s.q);
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
        const float4 r = *reinterpret_cast<const float4*>(rx + j);
        const uint64_t lo = mul2(pack2(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), p);
        const uint64_t hi = mul2(pack2(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), p);
        unpack2(mul2(mul2(lo, pack2(r.x, r.y)), q), y[j], y[j + 1]);
        unpack2(mul2(mul2(hi, pack2(r.z, r.w)), q), y[j + 2], y[j + 3]);
    }
}

// Sixteen scaled columns of the accumulator (rows m .. m + 15 of D, the first `rows` of them) of this lane's column n.
// ALL: nothing of the warp's 32 x 16 is past the edges.  A store of the warp is one contiguous piece of a row; in bf16 neighbouring lanes swap values, so that it is two
// rows' pieces of 4 bytes a lane.
template <bool ALL>
__device__ __forceinline__ void put16(const GemmParams& P, const float (&y)[16], int m, int rows, int n, int lane) {
    if (!P.bf16) {
        float* d = static_cast<float*>(P.d) + m * P.ldd + n;
#pragma unroll
        for (int j = 0; j < 16; ++j, d += P.ldd)
            if (ALL || (j < rows && n < P.N)) *d = y[j];
    } else if (ALL && P.pairs) {
        const bool odd = lane & 1;
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(P.d) + (m + odd) * P.ldd + (n - odd);
#pragma unroll
        for (int j = 0; j < 16; j += 2, d += 2 * P.ldd) {
            const float other = __shfl_xor_sync(0xffffffffu, odd ? y[j] : y[j + 1], 1);
            *reinterpret_cast<__nv_bfloat162*>(d) =
                odd ? __floats2bfloat162_rn(other, y[j + 1]) : __floats2bfloat162_rn(y[j], other);
        }
    } else {
        __nv_bfloat16* d = static_cast<__nv_bfloat16*>(P.d) + m * P.ldd + n;
#pragma unroll
        for (int j = 0; j < 16; ++j, d += P.ldd)
            if (ALL || (j < rows && n < P.N)) *d = __float2bfloat16_rn(y[j]);
    }
}

// `put16` by TMA, the warp's 32 columns from n0 on: 1 KB at a time (16 rows of bf16, 8 of fp32) through `buf`, which the copy
// before has to have left.
__device__ __forceinline__ void copy16(const GemmParams& P, const CUtensorMap* td, uint8_t* buf, const float (&y)[16], int m,
                                       int n0, int lane) {
    if (P.bf16) {
        if (lane == 0) tma_stores_read();
        __syncwarp();
        __nv_bfloat16* const b = reinterpret_cast<__nv_bfloat16*>(buf) + lane;
#pragma unroll
        for (int j = 0; j < 16; ++j) b[32 * j] = __float2bfloat16_rn(y[j]);
        fence_before_tma_store();
        __syncwarp();
        if (lane == 0) tma_store_2d(td, n0, m, buf);
    } else {
        float* const b = reinterpret_cast<float*>(buf) + lane;
#pragma unroll
        for (int h = 0; h < 16; h += 8) {
            if (lane == 0) tma_stores_read();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) b[32 * j] = y[h + j];
            fence_before_tma_store();
            __syncwarp();
            if (lane == 0 && m + h < P.M) tma_store_2d(td, n0, m + h, buf);
        }
    }
}

// K in parts: the CTAs (pairs) of a cluster have one tile, each the sums over its part of K.  A part owns NT / splits of the
// columns: it gets the others' sums of those in its shared memory, in the ring's place (whose last copy has been read once
// the sums are complete), and adds them and its own in the parts' order, so that the result is always the same bits.
// All threads of the cluster come here; `q`: the warp's quarter of the lanes, or -1 for those without a part in it; `side` of
// `sides` warps share the columns; `step`: CTAs of a part.  (4 columns of a lane a store: a store of one is four times as
// many to another SM, 8 us for 256 x 256 against 2.)
template <int NT>
__device__ __forceinline__ void join(const GemmParams& P, float4* ring, float* rx, int* far, uint32_t acc, int q, int side, int sides,
                                     int part, int step, int in_part, int n, int m0, int lane) {
    const int own = NT / P.splits;               // a multiple of 4
    acc += (uint32_t)(32 * max(q, 0)) << 16;
    // four columns of part p's for a part, in groups of four: [others][own / 4][128]
    auto place = [&](int from, int to, int c) { return ((from - (from > to)) * (own / 4) + c / 4) * 128 + 32 * q + lane; };
    float rn = 1.f;
    if (q >= 0) {                                // all that the end reads from memory, before anyone waits for anyone
        rn = P.rw && n < P.N ? P.rw[n] : 1.f;
        for (int c = (4 * side + q) * 32 + lane; c < NT; c += 128 * sides) {
            const int m = m0 + part * own + c;
            const float r = P.rx && c < own && m < P.M ? P.rx[m] : 1.f;
            if (beyond(r)) *far = 1;
            rx[c] = r;
        }
    }
    cluster_sync_all();
    if (q >= 0) {
        tc_fence_after();
#pragma unroll 1
        for (int c = 16 * side; c < NT; c += 16 * sides) {
            uint32_t v[16];
            tmem_ld16(acc + (uint32_t)c, v);
            tmem_wait16(v);
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                const int to = (c + j) / own;
                if (to != part) {
                    const uint32_t at = map_to_rank(ring + place(part, to, (c + j) % own), (uint32_t)(to * step + in_part));
                    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};"
                                 :: "r"(at), "r"(v[j]), "r"(v[j + 1]), "r"(v[j + 2]), "r"(v[j + 3]) : "memory");
                }
            }
        }
        __syncwarp();
    }
    cluster_sync_all();
    if (q < 0) return;
    const Lane sn = lane_scale(rn, P.alpha, P.am, P.ea, *far);
    const bool all = own >= 16 && m0 + (part + 1) * own <= P.M && n - lane + 32 <= P.N;
#pragma unroll 1
    for (int c = 16 * side; c < own; c += 16 * sides) {
        uint32_t v[16];
        tmem_ld16(acc + (uint32_t)(part * own + c), v);
        tmem_wait16(v);
        float s[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) s[j] = 0.f;
        for (int p = 0; p < P.splits; ++p) {
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                if (c + j >= own) continue;
                const float4 o = p == part ? make_float4(__uint_as_float(v[j]), __uint_as_float(v[j + 1]), __uint_as_float(v[j + 2]),
                                                         __uint_as_float(v[j + 3]))
                                           : ring[place(p, part, c + j)];
                s[j] += o.x;
                s[j + 1] += o.y;
                s[j + 2] += o.z;
                s[j + 3] += o.w;
            }
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(s[j]);
        scale16(s, v, rx + c, sn);
        const int m = m0 + part * own + c;
        if (all) put16<true>(P, s, m, 16, n, lane);
        else put16<false>(P, s, m, min(P.M - m, own - c), n, lane);
    }
}

template <int NT, int FMT>
struct Cfg {
    static constexpr int STAGES = NT <= 16 ? 5 : NT <= 32 ? 4 : 3;
    static constexpr int X_BYTES = NT * KB;
    static constexpr int SF_BYTES = SF_TILES<FMT> * SF_TILE;
    static constexpr uint32_t SF_COLS = 4 * SF_TILES<FMT>;     // of tensor memory, a stage and operand
    static constexpr uint32_t SF_AT = 2 * NT;                  // after the accumulators: two stages' scales in turn
    static constexpr uint32_t NEED = SF_AT + 4 * SF_COLS;
    static constexpr uint32_t COLS = NEED <= 128 ? 128 : 256;
    static_assert(NEED <= 256, "two CTAs an SM");
};

template <int NT, int FMT>
struct alignas(1024) Smem {
    uint8_t w[Cfg<NT, FMT>::STAGES][128 * KB];
    uint8_t x[Cfg<NT, FMT>::STAGES][Cfg<NT, FMT>::X_BYTES];
    uint8_t sfw[Cfg<NT, FMT>::STAGES][Cfg<NT, FMT>::SF_BYTES];
    uint8_t sfx[Cfg<NT, FMT>::STAGES][Cfg<NT, FMT>::SF_BYTES];
    alignas(16) float rx[4][NT];         // row scales, a copy a warp
    alignas(16) float rxj[NT];           // and where K is taken in parts
    uint64_t full[Cfg<NT, FMT>::STAGES], empty[Cfg<NT, FMT>::STAGES];
    uint64_t tfull[2], tempty[2], done;
    uint32_t tmem_base;
    int abort, far;                      // a wait ran out; rows' scales that `Lane` has to keep in range
};

template <int NT, int FMT>
__global__ void __launch_bounds__(192, 2)
    fp4_gemm(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx, const GemmParams P) {
    using C = Cfg<NT, FMT>;
    extern __shared__ uint8_t gsm_raw[];
    Smem<NT, FMT>& S = *reinterpret_cast<Smem<NT, FMT>*>((reinterpret_cast<uintptr_t>(gsm_raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int tiles = (P.N + 127) / 128, part = P.splits > 1 ? (int)cluster_ctarank() : 0;
    const int kb0 = P.nk * part / P.splits, kb1 = P.nk * (part + 1) / P.splits;
    const int first = blockIdx.x / P.splits, stride = gridDim.x / P.splits;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.tfull[b], 1);
            mbar_init(&S.tempty[b], 4);
        }
        mbar_init(&S.done, 1);
        S.abort = S.far = 0;
        fence_mbar_init_cluster();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(&S.tmem_base)), "r"(C::COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = S.tmem_base;

    if (warp == 0) {
        if (elect_one())
            for (int kb = kb0; kb < min(kb1, kb0 + (int)C::STAGES); ++kb) tma_prefetch_2d(&tw, kb * KB, first * 128);
        __syncwarp();
        pdl_wait_primary();
        uint32_t g = 0;
        bool stop = false;
        for (int t = first; t < tiles && !stop; t += stride) {
            const uint8_t* const sfw = P.sfw + (long long)t * P.tiles_k * SF_TILE;
            for (int kb = kb0; kb < kb1; ++kb, ++g) {
                const uint32_t s = g % C::STAGES, use = g / C::STAGES;
                if (use > 0 && !wait_all(&S.empty[s], (use - 1) & 1u, &S.abort)) {
                    stop = true;
                    break;
                }
                if (elect_one()) {
                    const int at = kb * SF_TILES<FMT>;
                    const uint32_t sfb = (uint32_t)min(SF_TILES<FMT>, P.tiles_k - at) * SF_TILE;
                    mbar_arrive_expect_tx(&S.full[s], 128 * KB + C::X_BYTES + 2 * sfb);
                    tma_load_1cta(S.w[s], &tw, kb * KB, t * 128, &S.full[s]);
                    bulk_g2s(S.sfw[s], sfw + (long long)at * SF_TILE, sfb, &S.full[s]);
                    tma_load_1cta(S.x[s], &tx, kb * KB, 0, &S.full[s]);
                    bulk_g2s(S.sfx[s], P.sfx + (long long)at * SF_TILE, sfb, &S.full[s]);
                }
                __syncwarp();
            }
        }
        if (lane == 0)                   // every copy issued has landed before the CTA can leave
            for (uint32_t gg = g > (uint32_t)C::STAGES ? g - C::STAGES : 0u; gg < g; ++gg)
                wait_parity_drain(&S.full[gg % C::STAGES], (gg / C::STAGES) & 1u);
    } else if (warp == 1) {
        pdl_wait_primary();              // no copy comes before: a wait for one would spend its limit on the work ahead
        uint32_t g = 0, tile = 0;
        bool stop = false;
        const uint64_t dw = sw128_desc(smem_u32(S.w[0])), dx = sw128_desc(smem_u32(S.x[0]));
        const uint64_t fw = sf_desc(smem_u32(S.sfw[0])), fx = sf_desc(smem_u32(S.sfx[0]));
        for (int t = first; t < tiles && !stop; t += stride, ++tile) {
            const uint32_t b = tile & 1u, use = tile >> 1;
            if (use > 0 && !wait_all(&S.tempty[b], (use - 1) & 1u, &S.abort)) break;
            for (int kb = kb0; kb < kb1; ++kb, ++g) {
                const uint32_t s = g % C::STAGES;
                if (!wait_all(&S.full[s], (g / C::STAGES) & 1u, &S.abort)) {
                    stop = true;
                    break;
                }
                tc_fence_after();
                if (elect_one()) {
                    const int mmas = min(4, P.mmas - 4 * kb), sft = min(SF_TILES<FMT>, P.tiles_k - kb * SF_TILES<FMT>);
                    const uint32_t ca = tmem + C::SF_AT + (g & 1u) * 2 * C::SF_COLS, cb = ca + C::SF_COLS;
                    for (int i = 0; i < sft; ++i) {
                        sf_copy<1>(ca + 4 * i, fw + (uint64_t)(s * C::SF_BYTES + i * SF_TILE >> 4));
                        sf_copy<1>(cb + 4 * i, fx + (uint64_t)(s * C::SF_BYTES + i * SF_TILE >> 4));
                    }
                    const uint64_t aw = dw + (uint64_t)(s * (128 * KB) >> 4), ax = dx + (uint64_t)(s * C::X_BYTES >> 4);
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        if (k < mmas) {
                            const uint32_t col = FMT == kNv ? 4 * k : 4 * (k >> 1);
                            mma_fp4<1, FMT>(tmem + b * NT, aw + 2 * k, ax + 2 * k, idesc<FMT>(128, NT, FMT == kNv ? 0 : 2 * (k & 1)),
                                            ca + col, cb + col, kb != kb0 || k != 0 ? 1u : 0u);
                        }
                    commit_1cta(&S.empty[s]);
                }
                __syncwarp();
            }
            if (!stop && elect_one()) commit_1cta(&S.tfull[b]);
            __syncwarp();
        }
        if (elect_one()) commit_1cta(&S.done);
    } else {
        pdl_wait_primary();
        const int q = warp & 3;
        float* const rx = S.rx[warp - 2];
        uint32_t tile = 0;
        bool far = false;
        if (FMT == kNv && P.splits == 1) {
            for (int i = lane; i < P.M; i += 32) far = far || beyond(P.rx[i]);
            far = __any_sync(0xffffffffu, far);
        }
        for (int t = first; t < tiles; t += stride, ++tile) {
            const uint32_t b = tile & 1u;
            const int n = t * 128 + 32 * q + lane;
            float rn = P.rw && n < P.N ? P.rw[n] : 1.f;
            __syncwarp();
            for (int i = lane; i < NT; i += 32) rx[i] = P.rx && i < P.M ? P.rx[i] : 1.f;
            __syncwarp();
            const bool cols = t * 128 + 128 <= P.N;
            if (!wait_all(&S.tfull[b], (tile >> 1) & 1u, &S.abort)) break;
            if (P.splits > 1) break;
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + b * NT;
            uint32_t v[2][16];
            tmem_ld16(acc, v[0]);
            hold(rn);
            const Lane sn = lane_scale(rn, P.alpha, P.am, P.ea, far);
#pragma unroll
            for (int c = 0; c < NT / 16; ++c) {
                tmem_wait16(v[c & 1]);
                if (c + 1 < NT / 16) tmem_ld16(acc + 16u * (c + 1), v[(c + 1) & 1]);
                else {                           // the accumulator has been read
                    tc_fence_before();
                    if (lane == 0) mbar_arrive(&S.tempty[b]);
                }
                float y[16];
                scale16(y, v[c & 1], rx + 16 * c, sn);
                if (cols && 16 * c + 16 <= P.M) put16<true>(P, y, 16 * c, 16, n, lane);
                else if (16 * c < P.M) put16<false>(P, y, 16 * c, P.M - 16 * c, n, lane);
            }
        }
    }
    __syncwarp();
    if (P.splits > 1)
        join<NT>(P, reinterpret_cast<float4*>(S.w), S.rxj, &S.far, tmem, warp >= 2 ? warp & 3 : -1, 0, 1, part, 1, 0,
                 first * 128 + 32 * (warp & 3) + lane, 0, lane);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        wait_parity_drain(&S.done, 0u);  // every MMA issued has completed before the columns are freed
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(C::COLS) : "memory");
    }
}

// ---------------------------------------------------------------- many rows

// More than 64 rows: two CTAs (two SMs) share a tile of 256 weight rows x NT hidden rows (tcgen05 with cta_group::2), each
// loading its 128 weight rows, half of the hidden rows and the scales that its own tensor memory needs.  One persistent
// pair per two SMs walks the tiles.  Per CTA: warp 0 the TMA producer (both CTAs' copies are counted on the leader's, the even
// CTA's, barrier), warp 1 of the leader the scales' copies and the MMAs, warp 2 tensor memory, warps 4-11 the epilogue.
//
// Tensor memory holds two accumulators and two stages' scales where they fit (NT <= 192); 2 x 256 columns do not leave
// room for scales, so there the second accumulator begins inside the first, and the epilogue empties the columns
// they share before it stores anything: the next tile's MMAs wait for those alone.
//
// 2048 x 128256 x 4096: 388 to 420 us by box and load (5.1 to 5.5 PFLOP/s), at the power limit (1.75 GHz); 2048 x 32000 x 8192 to bf16
// 163 to 176 (MX, half the scales: 152, 7.1 PFLOP/s).  A stage is four MMAs of 128 cycles and 12
// copies of scales, which take another 147 of the same pipe; it moves 76 KB through each SM's shared memory (38 in by TMA,
// 38 out to the MMAs), 594 cycles at 128 bytes.  Beside that D: 1 GB, 190 us alone.  Plain stores of D and the loads (221 us
// alone) do not hide behind one another (359 together, without MMAs; 430 with them): D goes by TMA where it may, see
// COPY_STAGES.  Tried, with plain stores: clusters of four CTAs with the hidden rows multicast (423 against 425, on the 144
// SMs that such clusters find).
//
// Where there are fewer tiles than pairs, several pairs of a cluster take a part of K each (see `join`).
template <int NT, int FMT>
struct Pair {
    static constexpr int X_ROWS = NT / 2;
    static constexpr int X_BYTES = X_ROWS * KB;
    static constexpr int X_TILES = (NT + 127) / 128;           // of scales, across the hidden rows
    static constexpr int SFW_BYTES = SF_TILES<FMT> * SF_TILE;
    static constexpr int SFX_BYTES = X_TILES * SFW_BYTES;
    static constexpr int STAGE = 128 * KB + X_BYTES + SFW_BYTES + SFX_BYTES;
    static constexpr int ROOM = 226 * 1024 - 8 * 1024 - 20 * NT - 512;     // beside the pieces of D, row scales and barriers
    static constexpr int STAGES = ROOM / STAGE < 8 ? ROOM / STAGE : 8;
    static constexpr int SF_COLS = 4 * SF_TILES<FMT> * (1 + X_TILES);      // a stage's
    static constexpr int SF_AT = (512 - 2 * SF_COLS) / 32 * 32;
    static constexpr int ACC1 = 2 * NT <= SF_AT ? NT : SF_AT - NT;         // where the second accumulator begins
    static constexpr int SHARED = NT - ACC1;                               // columns that both have
    static_assert(SHARED % 32 == 0 && NT % 32 == 0 && SHARED <= NT / 2, "chunks of 16 columns, split over two warps");
};

template <int NT, int FMT>
struct alignas(1024) PSmem {
    uint8_t w[Pair<NT, FMT>::STAGES][128 * KB];
    uint8_t x[Pair<NT, FMT>::STAGES][Pair<NT, FMT>::X_BYTES];
    uint8_t sfw[Pair<NT, FMT>::STAGES][Pair<NT, FMT>::SFW_BYTES];
    uint8_t sfx[Pair<NT, FMT>::STAGES][Pair<NT, FMT>::SFX_BYTES];
    alignas(128) uint8_t out[8][1024];           // a warp's piece of D on its way
    alignas(16) float rx[8][NT / 2];             // row scales of a warp's columns, in its order
    alignas(16) float rxj[NT];                   // and where K is taken in parts
    uint64_t full[Pair<NT, FMT>::STAGES];        // (leader) both CTAs' copies of a stage have landed
    uint64_t empty[Pair<NT, FMT>::STAGES];       // the MMAs have read a stage
    uint64_t tfull[2];                           // a tile's sums are complete
    uint64_t tempty[2];                          // (leader) both CTAs' epilogues have read what the next MMAs overwrite
    uint64_t done;                               // every MMA issued has completed
    uint32_t tmem_base;
    int abort, far;                              // a wait ran out; rows' scales that `Lane` has to keep in range
};

// COPIES: D is written by TMA (both ways in one kernel: 0.4 to 1 us slower at 256 x 32000 x 2048, 15).
template <int NT, int FMT, bool COPIES>
__global__ void __launch_bounds__(384, 1)
    fp4_gemm_pairs(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx,
                  const __grid_constant__ CUtensorMap tsw, const __grid_constant__ CUtensorMap tsx,
                  const __grid_constant__ CUtensorMap td, const GemmParams P) {
    using C = Pair<NT, FMT>;
    extern __shared__ uint8_t gsm_raw[];
    PSmem<NT, FMT>& S = *reinterpret_cast<PSmem<NT, FMT>*>((reinterpret_cast<uintptr_t>(gsm_raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), half = rank & 1, part = rank >> 1;
    const int cid = blockIdx.x / (2 * P.splits), ncl = gridDim.x / (2 * P.splits);
    const int kb0 = P.nk * part / P.splits, kb1 = P.nk * (part + 1) / P.splits;
    const int mt = (P.M + NT - 1) / NT, tiles = mt * ((P.N + 255) / 256);
    const int mine = 128 * half;         // this CTA's weight rows in a tile's 256
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::STAGES; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.tfull[b], 1);
            mbar_init(&S.tempty[b], 16);
        }
        mbar_init(&S.done, 1);
        S.abort = S.far = 0;
        fence_mbar_init_cluster();
    }
    __syncthreads();
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(&S.tmem_base)), "r"(512u) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    pdl_launch_dependents();
    const uint32_t tmem = S.tmem_base;

    if (warp == 0) {
        if (elect_one())
            for (int kb = kb0; kb < min(kb1, kb0 + C::STAGES); ++kb) tma_prefetch_2d(&tw, kb * KB, cid / mt * 256 + mine);
        __syncwarp();
        pdl_wait_primary();
        uint32_t g = 0;
        bool stop = false;
        for (int t = cid; t < tiles && !stop; t += ncl) {
            const int nt = t / mt, mi = t - nt * mt;
            for (int kb = kb0; kb < kb1; ++kb, ++g) {
                const uint32_t s = g % C::STAGES, use = g / C::STAGES;
                if (use > 0 && !wait_all(&S.empty[s], (use - 1) & 1u, &S.abort)) {
                    stop = true;
                    break;
                }
                if (elect_one()) {
                    const uint32_t bar = map_to_rank(&S.full[s], rank & ~1);
                    const int at = kb * SF_TILES<FMT>, xt = mi * NT / 128;
                    if (half == 0) mbar_arrive_expect_tx(&S.full[s], 2 * C::STAGE);
                    tma_load_2d(S.w[s], &tw, kb * KB, nt * 256 + mine, bar);
                    // scales past the last tile of K belong to other rows (or are zero) and are not used
                    tma_load_2d(S.sfw[s], &tsw, 0, (nt * 2 + half) * P.tiles_k + at, bar);
                    tma_load_2d(S.x[s], &tx, kb * KB, mi * NT + C::X_ROWS * half, bar);
#pragma unroll
                    for (int i = 0; i < C::X_TILES; ++i)
                        tma_load_2d(S.sfx[s] + i * C::SFW_BYTES, &tsx, 0, (xt + i) * P.tiles_k + at, bar);
                }
                __syncwarp();
            }
        }
    } else if (warp == 1 && half == 0) {
        // One thread from end to end, each stage in as few instructions as can be: what it takes between two stages shows
        // (2048 x 32000 x 8192, bf16 out: 163 us; a warp that meets in each stage 174, twice 204; the tile's first stage told
        // apart within the loop 1 to 3% more).  Every turn from copies to MMAs costs: copies a stage ahead, all before an
        // MMA (183) or four after each (192), are slower than all of a stage's together.
        pdl_wait_primary();              // no copy comes before: a wait for one would spend its limit on the work ahead
        if (elect_one()) {
            uint32_t g = 0, tile = 0;
            bool stop = false;
            const uint64_t dw = sw128_desc(smem_u32(S.w[0])), dx = sw128_desc(smem_u32(S.x[0]));
            const uint64_t fw = sf_desc(smem_u32(S.sfw[0])), fx = sf_desc(smem_u32(S.sfx[0]));
            auto scales = [&](uint32_t s) {
                const uint32_t ca = tmem + C::SF_AT + (g & 1u) * C::SF_COLS, cb = ca + 4 * SF_TILES<FMT>;
#pragma unroll
                for (int i = 0; i < SF_TILES<FMT>; ++i) {
                    sf_copy<2>(ca + 4 * i, fw + (uint64_t)(s * C::SFW_BYTES + i * SF_TILE >> 4));
#pragma unroll
                    for (int j = 0; j < C::X_TILES; ++j)
                        sf_copy<2>(cb + 4 * (C::X_TILES * i + j),
                                   fx + (uint64_t)(s * C::SFX_BYTES + j * C::SFW_BYTES + i * SF_TILE >> 4));
                }
            };
            auto multiply = [&](uint32_t s, uint32_t acc, uint32_t odd, int mmas, auto add) {
                const uint32_t ca = tmem + C::SF_AT + (g & 1u) * C::SF_COLS, cb = ca + 4 * SF_TILES<FMT>;
                const uint64_t aw = dw + (uint64_t)(s * (128 * KB) >> 4), ax = dx + (uint64_t)(s * C::X_BYTES >> 4);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    if (k < mmas) {
                        const int i = FMT == kNv ? k : k >> 1;
                        mma_fp4<2, FMT>(acc, aw + 2 * k, ax + 2 * k, idesc<FMT>(256, NT, FMT == kNv ? 0 : 2 * (k & 1)),
                                        ca + 4 * i, cb + 4 * C::X_TILES * i + odd, decltype(add)::value || k != 0 ? 1u : 0u);
                    }
                commit_2cta(&S.empty[s], 3u << rank);
                ++g;
            };
            for (int t = cid; t < tiles && !stop; t += ncl, ++tile) {
                const int mi = t % mt;
                // NT = 192: odd tiles of hidden rows begin in the middle of a tile of scales
                const uint32_t odd = (uint32_t)(mi * NT % 128) / 32u, acc = tmem + (tile & 1u) * C::ACC1;
                const uint32_t free = tile - (C::SHARED ? 1u : 2u);        // the tile whose columns these MMAs overwrite
                uint32_t s = g % C::STAGES;
                if ((int)free >= 0 && !wait_parity<false>(&S.tempty[free & 1u], (free >> 1) & 1u, &S.abort, &g_watchdog)) break;
                if (!wait_parity<false>(&S.full[s], (g / C::STAGES) & 1u, &S.abort, &g_watchdog)) break;
                tc_fence_after();
                scales(s);
                multiply(s, acc, odd, min(4, P.mmas - 4 * kb0), std::false_type());
                for (int kb = kb0 + 1; kb < kb1; ++kb) {
                    s = g % C::STAGES;
                    if (!wait_parity<false>(&S.full[s], (g / C::STAGES) & 1u, &S.abort, &g_watchdog)) {
                        stop = true;
                        break;
                    }
                    tc_fence_after();
                    scales(s);
                    multiply(s, acc, odd, min(4, P.mmas - 4 * kb), std::true_type());
                }
                if (!stop) commit_2cta(&S.tfull[tile & 1u], 3u << rank);
            }
            commit_2cta(&S.done, 3u << rank);
        }
        __syncwarp();
    } else if (warp >= 4) {
        pdl_wait_primary();
        const int q = warp & 3, side = (warp - 4) >> 2;
        const uint32_t tempty[2] = {map_to_rank(&S.tempty[0], rank & ~1), map_to_rank(&S.tempty[1], rank & ~1)};
        constexpr int CH = NT / 32, SH = C::SHARED / 32;       // a warp's chunks of 16 columns, and those shared
        float* const rx = S.rx[warp - 4];
        uint32_t tile = 0;
        // asked once, of all rows that this CTA meets: in the loop below even the question cost 1 to 5%
        if (FMT == kNv && P.splits == 1) {
            const int i = threadIdx.x - 128;
            bool any = false;
            // tile by tile, until the same rows come again
            const int count = min(mt, (tiles - cid + ncl - 1) / ncl), step = ncl % mt;
            int mi = cid % mt;
#pragma unroll 8
            for (int j = 0; j < count; ++j) {
                const int m = mi * NT + i;
                any = any | beyond(i < NT && m < P.M ? P.rx[m] : 1.f);
                mi += step;
                mi -= mi >= mt ? mt : 0;
            }
            if (any) S.far = 1;
            named_sync(1, 256);
        }
        const bool far = S.far != 0;
        for (int t = cid; t < tiles; t += ncl, ++tile) {
            const uint32_t b = tile & 1u, acc = tmem + ((uint32_t)(32 * q) << 16) + b * C::ACC1;
            const int n = t / mt * 256 + mine + 32 * q + lane, m0 = t % mt * NT;
            // the shared chunks first: the first accumulator's last columns, the second's first
            const int sh0 = (b ? 0 : C::ACC1) + 16 * SH * side, own0 = (b ? C::SHARED : 0) + 16 * (CH - SH) * side;
            auto col = [&](int i) { return i < SH ? sh0 + 16 * i : own0 + 16 * (i - SH); };
            float rn = P.rw && n < P.N ? P.rw[n] : 1.f;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < (CH + 1) / 2; ++i) {
                const int chunk = 2 * i + (lane >> 4), m = m0 + col(chunk) + (lane & 15);
                if (chunk < CH) rx[16 * chunk + (lane & 15)] = P.rx && m < P.M ? P.rx[m] : 1.f;
            }
            __syncwarp();
            const bool cols = t / mt * 256 + mine + 128 <= P.N;
            if (!wait_all(&S.tfull[b], (tile >> 1) & 1u, &S.abort)) break;
            if (P.splits > 1) break;
            tc_fence_after();
            Lane sn;
            auto put = [&](int i, const uint32_t (&w)[16]) {
                const int m = m0 + col(i);
                float y[16];
                scale16(y, w, rx + 16 * i, sn);
                if constexpr (COPIES) {
                    if (m < P.M && n - lane < P.N) copy16(P, &td, S.out[warp - 4], y, m, n - lane, lane);
                } else if (cols && m + 16 <= P.M) put16<true>(P, y, m, 16, n, lane);
                else if (m < P.M) put16<false>(P, y, m, P.M - m, n, lane);
            };
            uint32_t v[2][16];
            if constexpr (SH > 0) {
                // what the next MMAs overwrite is read before anything is stored
                uint32_t s[SH][16];
#pragma unroll
                for (int i = 0; i < SH; ++i) tmem_ld16(acc + (uint32_t)col(i), s[i]);
#pragma unroll
                for (int i = 0; i < SH; ++i) tmem_wait16(s[i]);
                tc_fence_before();
                if (lane == 0) arrive_cluster(tempty[b]);
                tmem_ld16(acc + (uint32_t)col(SH), v[SH & 1]);
                hold(rn);
                sn = lane_scale(rn, P.alpha, P.am, P.ea, far);
#pragma unroll
                for (int i = 0; i < SH; ++i) put(i, s[i]);
            } else {
                tmem_ld16(acc + (uint32_t)col(0), v[0]);
                hold(rn);
                sn = lane_scale(rn, P.alpha, P.am, P.ea, far);
            }
#pragma unroll
            for (int i = SH; i < CH; ++i) {
                tmem_wait16(v[i & 1]);
                if (i + 1 < CH) tmem_ld16(acc + (uint32_t)col(i + 1), v[(i + 1) & 1]);
                if (SH == 0 && i == CH - 1) {
                    tc_fence_before();
                    if (lane == 0) arrive_cluster(tempty[b]);
                }
                put(i, v[i & 1]);
            }
        }
        if (COPIES && lane == 0) tma_stores_done();
    }
    __syncwarp();
    if (P.splits > 1)
        join<NT>(P, reinterpret_cast<float4*>(S.w), S.rxj, &S.far, tmem, warp >= 4 ? warp & 3 : -1, (warp - 4) >> 2, 2, part, 2, half,
                 cid / mt * 256 + mine + 32 * (warp & 3) + lane, cid % mt * NT, lane);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    // Every MMA issued has completed, and with it every copy it read; after a wait that ran out,
    // give copies in flight into this CTA time to land.
    if (threadIdx.x == 0) {
        wait_parity_drain(&S.done, 0u);
        if (*(volatile int*)&S.abort)
            for (const long long t0 = clock64(); clock64() - t0 < 4000000;) {
            }
    }
    cluster_sync_all();
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(512u) : "memory");
    }
}

// The tiles of scales as rows of 128 words, `box` of them a copy.
bool make_sf_map(CUtensorMap* map, const void* base, long long tiles, int box) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {128, (cuuint64_t)tiles};
    const cuuint64_t strides[1] = {SF_TILE};
    const cuuint32_t boxes[2] = {128, (cuuint32_t)box};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, 2, const_cast<void*>(base), dims, strides, boxes, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// D, a warp's piece a copy.
bool make_out_map(CUtensorMap* map, const Fp4Gemm& G, int bytes) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)G.N, (cuuint64_t)G.M};
    const cuuint64_t strides[1] = {(cuuint64_t)G.ldd * bytes};
    const cuuint32_t boxes[2] = {32, (cuuint32_t)(32 / bytes)};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, bytes == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, G.d, dims, strides, boxes,
               estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_NONE,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename K, typename... Args>
cudaError_t launch_cluster(K kernel, long long grid, int threads, size_t smem, int cluster, cudaStream_t st, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)grid, 1, 1);
    cfg.blockDim = dim3((unsigned)threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Parts of K for `tiles` tiles where `places` CTAs run at once, up to `most`: those that fill the places, of four
// stages (1024 columns) each at least.  (8 x 4096 x 32000: 47 us in one part, 27 in two, 17 in four.)
int parts_of(long long tiles, long long places, int most, int nk) {
    int s = 1;
    while (2 * s <= most && tiles * 2 * s <= places && nk >= 8 * s) s *= 2;
    return s;
}

template <int NT, int FMT>
cudaError_t go(const Fp4Gemm& G, GemmParams P, int dev, int sms, cudaStream_t st) {
    static std::atomic<int> had[64];
    const size_t smem = sizeof(Smem<NT, FMT>) + 1024;
    static_assert(2 * (sizeof(Smem<NT, FMT>) + 2048) <= 228 * 1024, "shared memory of an SM's two CTAs");
    static_assert(sizeof(Smem<NT, FMT>::w) >= NT * 512, "the sums of a tile in the ring");
    if (!had[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute((const void*)fp4_gemm<NT, FMT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        had[dev].store(1, std::memory_order_release);
    }
    CUtensorMap tw, tx;
    const long long pitch = fp4_kp(G.K) / 2;
    if (!make_map(&tw, G.b, G.N, pitch, 128) || !make_map(&tx, G.a, G.M, pitch, NT)) return cudaErrorInvalidValue;
    const long long tiles = (G.N + 127) / 128, most = 2ll * sms;
    P.splits = parts_of(tiles, most, NT == 16 ? 4 : 8, P.nk);
    const long long ctas = P.splits > 1 ? tiles * P.splits : tiles < most ? tiles : most;
    return launch_cluster(fp4_gemm<NT, FMT>, ctas, 192, smem, P.splits, st, tw, tx, P);
}

// Stages of K from which on D goes by TMA, where its rows begin and end at 16 bytes (a copy that is cut off at a row's end writes
// whole blocks of 16 bytes, past it): the copies are the slower way, paced by their one
// buffer a warp, and leave the loads alone, so that a tile that takes longer than its epilogue hides them.  (2048 x 32000
// fp32, us by TMA and by plain stores: K = 2048 79 and 70, 2560 85 and 84 (MX 78 and 81), 2816 86 and 90, 4096 100 and 115;
// bf16 62 and 63, 74 and 76, 71 and 77, 90 and 103.  2048 x 128256 x 4096: 404 and 430.  With two buffers 403 against 390
// for one on one box, with 128 columns a copy 407 against 402.)
constexpr int COPY_STAGES = 10;

template <int NT, int FMT, bool COPIES>
cudaError_t pair_launch(const Fp4Gemm& G, GemmParams P, int dev, int sms, cudaStream_t st) {
    static std::atomic<int> had[64];
    const size_t smem = sizeof(PSmem<NT, FMT>) + 1024;
    static_assert(sizeof(PSmem<NT, FMT>) + 1024 <= 227 * 1024, "shared memory of a CTA");
    static_assert(sizeof(PSmem<NT, FMT>::w) + sizeof(PSmem<NT, FMT>::x) >= NT * 512, "the sums of a tile in the ring");
    if (!had[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute((const void*)fp4_gemm_pairs<NT, FMT, COPIES>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        had[dev].store(1, std::memory_order_release);
    }
    CUtensorMap tw, tx, tsw, tsx, td = {};
    const long long pitch = fp4_kp(G.K) / 2;
    // Rows that do not all begin at 256 bytes: lines of 128 alone (2048 x 4096 x 50257 MX 212 us, by 256 230; 512 NV 74 and 78).
    // Those that do: 256 (512 x 4096 x 50176 62.5 and, by 128, 63.9).  In `go` 256 is as good or better for either.
    const CUtensorMapL2promotion ahead = pitch % 256 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B;
    if (!make_map(&tw, G.b, G.N, pitch, 128, ahead) || !make_map(&tx, G.a, G.M, pitch, NT / 2, ahead) ||
        !make_sf_map(&tsw, G.sfb, (G.N + 127) / 128 * P.tiles_k, SF_TILES<FMT>) ||
        !make_sf_map(&tsx, G.sfa, (G.M + 127) / 128 * P.tiles_k, SF_TILES<FMT>) ||
        (COPIES && !make_out_map(&td, G, P.bf16 ? 2 : 4)))
        return cudaErrorInvalidValue;
    const long long tiles = (G.M + NT - 1) / NT * ((G.N + 255) / 256), most = sms / 2;
    if (tiles > 0x3fffffffLL) return cudaErrorInvalidValue;
    const long long pairs = P.splits > 1 ? tiles * P.splits : tiles < most ? tiles : most;
    return launch_cluster(fp4_gemm_pairs<NT, FMT, COPIES>, 2 * pairs, 384, smem, 2 * P.splits, st, tw, tx, tsw, tsx, td, P);
}

template <int NT, int FMT>
cudaError_t pair_go(const Fp4Gemm& G, GemmParams P, int splits, int dev, int sms, cudaStream_t st) {
    const int bytes = P.bf16 ? 2 : 4;
    P.splits = splits;
    const bool copies = splits == 1 && P.nk >= COPY_STAGES && reinterpret_cast<uintptr_t>(G.d) % 16 == 0 &&
                        G.ldd * bytes % 16 == 0 && G.N * bytes % 16 == 0 && G.ldd < (1ll << 36);
    return copies ? pair_launch<NT, FMT, true>(G, P, dev, sms, st) : pair_launch<NT, FMT, false>(G, P, dev, sms, st);
}

template <int FMT>
cudaError_t pick(const Fp4Gemm& G, const GemmParams& P, int dev, int sms, cudaStream_t st) {
    if (G.M <= 16) return go<16, FMT>(G, P, dev, sms, st);
    if (G.M <= 32) return go<32, FMT>(G, P, dev, sms, st);
    if (G.M <= 64) return go<64, FMT>(G, P, dev, sms, st);
    // The tile's width and the parts of K (at most two: clusters of eight CTAs of this size find too few places) by what a
    // pair takes, in microseconds as measured: a stage, what of a tile's epilogue shows, meeting.  2048 x 128256 x 4096:
    // 128 wide 508 us, 192 454, 256 414; 512 x 4096 x 32000: 36, 41 and 43, 256 in two parts 31; 512 x 4096 x 4096: 9.2, 10.1,
    // 10.4 and 13; 256 x 4096 x 32000: 34, 128 in two parts 24.
    static const struct {
        int nt;
        double stage, end, meet;
    } kinds[] = {{128, 0.29, 0.2, 3.0}, {192, 0.38, 0.2, 4.0}, {256, 0.42, 1.3, 5.0}};
    const long long pairs = sms / 2;
    double best = 0;
    int nt = 0, splits = 1;
    for (const auto& k : kinds) {
        const long long tiles = (G.M + k.nt - 1) / k.nt * ((G.N + 255) / 256);
        for (int s = 1; s <= 2; ++s) {
            if (s > 1 && (tiles * s > pairs || P.nk < 8)) break;
            const double waves = (double)((tiles * s + pairs - 1) / pairs);
            const double t = waves * ((double)P.nk / s * k.stage + k.end) + (s > 1 ? k.meet : 0.0);
            if (nt == 0 || t < best) best = t, nt = k.nt, splits = s;
        }
    }
    if (nt == 128) return pair_go<128, FMT>(G, P, splits, dev, sms, st);
    if (nt == 192) return pair_go<192, FMT>(G, P, splits, dev, sms, st);
    return pair_go<256, FMT>(G, P, splits, dev, sms, st);
}

}  // namespace

cudaError_t fp4_gemm_tn(const Fp4Gemm& G, cudaStream_t st) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int sms = num_sms();
    if (dev < 0 || dev >= 64 || sms <= 0) return cudaErrorInvalidDevice;
    GemmParams P;
    P.sfw = G.sfb;
    P.sfx = G.sfa;
    P.rw = G.rb;
    P.rx = G.ra;
    P.d = G.d;
    P.bf16 = G.dtype == kBf16;
    P.pairs = G.ldd % 2 == 0 && reinterpret_cast<uintptr_t>(G.d) % 4 == 0;
    P.ldd = G.ldd;
    P.M = (int)G.M;
    P.N = (int)G.N;
    P.nk = (int)((fp4_kp(G.K) + KE - 1) / KE);
    P.tiles_k = (int)fp4_tiles_k(G.K, G.fmt);
    P.mmas = (int)((G.K + 63) / 64);
    P.alpha = P.am = G.alpha;
    P.ea = 0;
    if (std::isfinite(G.alpha)) P.am = std::frexp(G.alpha, &P.ea);
    return G.fmt == kNv ? pick<kNv>(G, P, dev, sms, st) : pick<kMx>(G, P, dev, sms, st);
}

unsigned int fp4_watchdog(bool clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_watchdog, sizeof(v)) != cudaSuccess) return 0xffffffffu;
    if (clear && v) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_watchdog, &z, sizeof(z)) != cudaSuccess) return 0xffffffffu;
    }
    return v;
}

}  // namespace vl
