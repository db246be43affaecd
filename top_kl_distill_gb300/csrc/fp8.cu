// The head's product in 8-bit floating point (sm_103a): D[M][N] = alpha sum over blocks b of 128
// along K of sa[b][m] sb[n / 128][b] (sum over k in b of A[m][k] B[n][k]), A and B e4m3, and the
// quantisers that make A (a scale for each 1 x 128) and B (a scale for each 128 x 128).
//
// The scales change from one block of K to the next, so a block's sum cannot stay in the tensor
// cores' accumulator: each block's sum lands in one of two tensor-memory buffers, and eight
// epilogue warps add it, scaled, to fp32 registers while the tensor cores work on the next block.
// Two CTAs (two SMs) share a 256 x 256 tile of D (tcgen05 with cta_group::2): each loads its 128
// rows of A and half of B's 256, 32 KB a block instead of 48, which is what lets L2 keep up with
// the 8-bit rate (512 cycles a block).  One persistent pair per two SMs walks the tiles.  Per CTA:
//   warp 0      TMA producer: boxes of 128 x 128 bytes of A and B, 128-byte swizzle, one block of
//               K a stage, into a 6-stage ring; both CTAs' copies are counted on the leader's
//               (rank 0) barrier;
//   warp 1      of the leader: tcgen05.mma (kind::f8f6f4, M = 256, N = 256, K = 32; four a block)
//               into the buffer of the block's parity, once both CTAs' epilogues have handed it
//               back; commits to both CTAs' barriers;
//   warp 2      tensor memory;
//   warps 4-11  the epilogue: 32 rows (tensor-memory lanes) x 128 columns a warp, so that a thread
//               has one row and one 128-column group: one scale a block, 128 sums in registers
//               (setmaxnreg moves the other warps' registers here).  Tensor-memory loads run one
//               32-column chunk ahead of the multiply-adds.  D leaves through shared memory, whole
//               128-byte lines at a time.
// Rows, columns and K past the edges: the TMA fills zeros, the epilogue masks stores; warps whose
// rows are all past M only pass the barriers.
#include "vl_api.h"
#include "vl_device.cuh"
#include "vl_internal.h"
#include "vl_launch.h"
#include "vl_pair.cuh"
#include "vl_rowio.cuh"

#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>

namespace vl {
namespace {

constexpr int BLK = 128;                 // elements of K (and of N) that share a scale
constexpr float kInvE4m3Max = 1.f / 448.f;   // rounded to fp32: a scale is amax times this
constexpr float kAmaxFloor = 7.888609052210118e-31f;      // 2^-100

__device__ unsigned int g_watchdog;

// ---------------------------------------------------------------- quantisers

// Two floats to e4m3, nearest even, saturating; lo in the lower byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float warp_max(float a) {
    float d;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(d) : "f"(a));
    return d;
}

// Four consecutive elements, those before `n` (the others 0); VEC: all four in one load.
template <bool VEC>
__device__ __forceinline__ float4 ld4(const float* p, int n) {
    if (VEC) return n > 0 ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
    return make_float4(n > 0 ? p[0] : 0.f, n > 1 ? p[1] : 0.f, n > 2 ? p[2] : 0.f, n > 3 ? p[3] : 0.f);
}
template <bool VEC>
__device__ __forceinline__ float4 ld4(const __nv_bfloat16* p, int n) {
    if (VEC) {
        const uint2 r = n > 0 ? *reinterpret_cast<const uint2*>(p) : make_uint2(0u, 0u);
        return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xffff0000u), __uint_as_float(r.y << 16),
                           __uint_as_float(r.y & 0xffff0000u));
    }
    return make_float4(n > 0 ? ld_elem(p) : 0.f, n > 1 ? ld_elem(p + 1) : 0.f, n > 2 ? ld_elem(p + 2) : 0.f,
                       n > 3 ? ld_elem(p + 3) : 0.f);
}
__device__ __forceinline__ float amax4(float4 v) { return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w))); }
__device__ __forceinline__ float scale_of(float amax) { return __fmul_rn(fmaxf(amax, kAmaxFloor), kInvE4m3Max); }

// x / s as e4m3 needs it, from inv = fl(1 / s): p = x inv and one step of Newton's on its residual
// (exact in an fma) leaves a relative error of 2^-47 before the last rounding, so that the result
// can differ from fl(x / s) only where x / s is that near to the middle of two floats.  What
// matters is whether the result lies below, on or above the middle m of two e4m3 values, a
// 5-bit number: for the 24-bit X, S of x, s that takes |X 2^k - (M 2^20 +- 1) S| <= 4 with k >= 24,
// so S within 4 of a multiple of 2^20.  Scales like those (a margin of 8), and those whose
// residuals leave the normal floats, divide (inv = 0).  Weights 32000 x 4096: 85 us, 118 with a
// division an element; rows 2048 x 32000 bf16 48 and 55, fp32 53 and 58.
__device__ __forceinline__ float reciprocal_of(float s) {
    const bool sound = s >= 0x1p-80f && s <= 0x1p+120f && ((__float_as_uint(s) + 8u) & 0xfffffu) > 16u;
    return sound ? __frcp_rn(s) : 0.f;
}
__device__ __forceinline__ float quotient(float x, float s, float inv) {
    const float p = x * inv;
    return fmaf(fmaf(p, s, -x), -inv, p);       // signs so that a residual of 0 leaves -0 as it is
}

template <bool VEC>
__device__ __forceinline__ void st4(uint8_t* q, float4 v, float s, float inv, int n) {
    float4 p;
    if (inv != 0.f) p = make_float4(quotient(v.x, s, inv), quotient(v.y, s, inv), quotient(v.z, s, inv), quotient(v.w, s, inv));
    else p = make_float4(__fdiv_rn(v.x, s), __fdiv_rn(v.y, s), __fdiv_rn(v.z, s), __fdiv_rn(v.w, s));
    const uint32_t w = e4m3x2(p.x, p.y) | e4m3x2(p.z, p.w) << 16;
    if (VEC) {
        if (n > 0) *reinterpret_cast<uint32_t*>(q) = w;
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < n) q[j] = (uint8_t)(w >> (8 * j));
}

// Both quantisers are HBM bound: fp32 in and a byte out.  Where rows start on the right boundary
// and K is a multiple of 4 (VEC) a lane moves its four elements at once, else one by one.
//
// One warp takes RUN blocks of 1 x 128 of a row, all loaded before the first is reduced; the
// warps beside it take the next rows, so that a CTA's scales are neighbours.
constexpr int RUN = 4;

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) quant_rows(const T* x, long long ldx, long long M, int K, uint8_t* q, float* sa) {
    pdl_launch_dependents();
    pdl_wait_primary();
    const int nkb = (K + BLK - 1) / BLK, lane = threadIdx.x & 31;
    const long long total = M * ((nkb + RUN - 1) / RUN), stride = (long long)gridDim.x * 8;
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += stride) {
        const long long run = total <= 0xffffffffll ? (long long)((uint32_t)i / (uint32_t)M) : i / M, m = i - run * M;
        const int kb = (int)run * RUN, k0 = kb * BLK + 4 * lane;
        float4 v[RUN];
#pragma unroll
        for (int u = 0; u < RUN; ++u) v[u] = ld4<VEC>(x + m * ldx + k0 + u * BLK, K - k0 - u * BLK);
        // lane u works out block u's scale and its reciprocal
        float mine = 0.f;
#pragma unroll
        for (int u = 0; u < RUN; ++u) {
            const float a = warp_max(amax4(v[u]));
            mine = lane == u ? a : mine;
        }
        mine = scale_of(mine);
        const float minv = reciprocal_of(mine);
        if (lane < RUN && kb + lane < nkb) sa[(kb + lane) * M + m] = mine;
#pragma unroll
        for (int u = 0; u < RUN; ++u)
            st4<VEC>(q + m * K + k0 + u * BLK, v[u], __shfl_sync(0xffffffffu, mine, u), __shfl_sync(0xffffffffu, minv, u),
                     K - k0 - u * BLK);
    }
}

// One CTA a block of 128 x 128, 16 rows of it a warp, in registers between the two uses.
template <bool VEC>
__global__ void __launch_bounds__(256) quant_blocks(const __nv_bfloat16* w, long long N, int K, uint8_t* q, float* sb) {
    __shared__ float red[8];
    pdl_launch_dependents();
    pdl_wait_primary();
    const int nkb = (K + BLK - 1) / BLK, lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const long long blocks = (N + BLK - 1) / BLK * nkb;
    for (long long i = blockIdx.x; i < blocks; i += gridDim.x) {
        const long long n0 = i / nkb * BLK + wp;
        const int k0 = (int)(i % nkb) * BLK + 4 * lane;
        float4 v[16];
        float amax = 0.f;
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r] = ld4<VEC>(w + (n0 + 8 * r) * K + k0, n0 + 8 * r < N ? K - k0 : 0);
#pragma unroll
        for (int r = 0; r < 16; ++r) amax = fmaxf(amax, amax4(v[r]));
        amax = warp_max(amax);
        __syncthreads();
        if (lane == 0) red[wp] = amax;
        __syncthreads();
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, red[j]);
        const float s = scale_of(amax), inv = reciprocal_of(s);
#pragma unroll
        for (int r = 0; r < 16; ++r) st4<VEC>(q + (n0 + 8 * r) * K + k0, v[r], s, inv, n0 + 8 * r < N ? K - k0 : 0);
        if (threadIdx.x == 0) sb[i] = s;
    }
}

// ---------------------------------------------------------------- the product

constexpr int BM = 256, BN = 256, STAGES = 6;    // a pair's tile
constexpr int HALF = 128;                        // rows of A, and of B, that one CTA loads
constexpr int OP_BYTES = HALF * BLK;
constexpr int EPI_WARPS = 8;
constexpr int GT = 128 + 32 * EPI_WARPS;
constexpr uint32_t TMEM_COLS = 2 * BN;

struct alignas(1024) GSmem {
    uint8_t a[STAGES][OP_BYTES];
    uint8_t b[STAGES][OP_BYTES];
    alignas(128) float out[EPI_WARPS][32 * 32];  // a chunk of D on its way out, per warp
    uint64_t full[STAGES];               // (leader) both CTAs' copies of a stage have landed
    uint64_t empty[STAGES];              // the MMAs have read a stage
    uint64_t tfull[2];                   // a block's sum is complete
    uint64_t tempty[2];                  // (leader) both CTAs' epilogues have read it
    uint64_t done;                       // every MMA issued has completed
    uint32_t tmem_base;
    int abort;
};
static_assert(sizeof(GSmem) + 1024 <= 227 * 1024, "shared memory of one CTA");

// K-major operand tile of 128-byte rows, 128-byte swizzle, groups of 8 rows 1024 bytes apart
// (fields as in the bf16 product); 32 elements of K are 32 bytes.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

// kind::f8f6f4: D f32 (bits 4-5 = 1), A and B e4m3 (7-9, 10-12 = 0), both K-major, N >> 3, M >> 4.
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);

// bar: a shared::cluster address (the leader's barrier)
__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile("cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar) : "memory");
}

// Brings a box into L2.  Safe before the work ahead in the stream is done: what that still writes goes
// through L2 too.
__device__ __forceinline__ void tma_prefetch_2d(const CUtensorMap* map, int x, int y) {
    asm volatile("cp.async.bulk.prefetch.tensor.2d.L2.global.tile [%0, {%1, %2}];"
                 :: "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y) : "memory");
}

__device__ __forceinline__ void mma_fp8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(kIdesc), "r"(acc) : "memory");
}

// arrives at this barrier of both CTAs once every MMA issued before has completed
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 :: "r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}

// Arrives at a barrier of either CTA.  What it hands over is tensor memory that tcgen05.ld has
// already read (tcgen05.wait::ld and the fence before it order that), so it needs no release at
// cluster scope, which waits for every memory operation of the thread: 2.1 ms instead of 0.8 at
// 2048 x 128256 x 4096.
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(bar) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}

// wait_parity by a whole warp: all lanes agree on whether it gave up.
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity, int* abort) {
    return __all_sync(0xffffffffu, wait_parity<false>(bar, parity, abort, &g_watchdog));
}

// 32 accumulator columns of this warp's 32 lanes; complete only after tmem_wait().
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
                 "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
                   "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]),
                   "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]),
                   "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(taddr));
}
// Every tcgen05.ld of the warp has completed; the registers pass through, so that nothing reads
// them before it.
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32], uint32_t (&q)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 32; i += 4)
        asm volatile("" : "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(q[i]), "+r"(q[i + 1]), "+r"(q[i + 2]),
                          "+r"(q[i + 3]));
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(GT, 1)
    fp8_gemm(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb, const float* sa,
             const float* sb, float* D, long long ldd, int M, int N, int K, float alpha,
             int m_fast) {
    extern __shared__ uint8_t gsm_raw[];
    GSmem& S = *reinterpret_cast<GSmem*>((reinterpret_cast<uintptr_t>(gsm_raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int rank = (int)cluster_ctarank(), cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
    const int mt = (M + BM - 1) / BM, ntl = (N + BN - 1) / BN;
    const int tiles = mt * ntl;
    const int nk = (K + BLK - 1) / BLK;
    auto tile_at = [&](int t, int& m0, int& n0) {
        const int a = m_fast ? t % mt : t / ntl, b = m_fast ? t / mt : t % ntl;
        m0 = a * BM;
        n0 = b * BN;
    };
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&S.full[s], 1);
            mbar_init(&S.empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&S.tfull[b], 1);
            mbar_init(&S.tempty[b], 2 * EPI_WARPS);
        }
        mbar_init(&S.done, 1);
        S.abort = 0;
        fence_mbar_init_cluster();
    }
    __syncthreads();
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(&S.tmem_base)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    cluster_sync_all();
    tc_fence_after();
    pdl_launch_dependents();
    pdl_wait_primary();
    const uint32_t tmem = S.tmem_base;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        // The whole warp walks the loops, so that coordinates and descriptors stay in uniform
        // registers; one elected lane issues.  (With the loops inside one lane's branch an MMA
        // took some 80 cycles to issue, more than it takes to run.)
        if (warp == 0) {
            uint32_t g = 0;
            bool stop = false;
            for (int t = cid; t < tiles && !stop; t += ncl) {
                int m0, n0;
                tile_at(t, m0, n0);
                for (int kb = 0; kb < nk; ++kb, ++g) {
                    const uint32_t s = g % STAGES, use = g / STAGES;
                    if (use > 0 && !wait_all(&S.empty[s], (use - 1) & 1u, &S.abort)) {
                        stop = true;
                        break;
                    }
                    if (elect_one()) {
                        const uint32_t bar = map_to_rank(&S.full[s], 0);
                        if (rank == 0) mbar_arrive_expect_tx(&S.full[s], 4 * OP_BYTES);
                        tma_load_2d(S.a[s], &ta, kb * BLK, m0 + HALF * rank, bar);
                        tma_load_2d(S.b[s], &tb, kb * BLK, n0 + HALF * rank, bar);
                    }
                    __syncwarp();
                }
            }
        } else if (warp == 1 && rank == 0) {
            uint32_t g = 0;
            bool stop = false;
            const uint64_t da = sw128_desc(smem_u32(S.a[0])), db = sw128_desc(smem_u32(S.b[0]));
            for (int t = cid; t < tiles && !stop; t += ncl) {
                for (int kb = 0; kb < nk && !stop; ++kb, ++g) {
                    const uint32_t s = g % STAGES, b = g & 1u, use = g >> 1;
                    // a stage further: OP_BYTES; 32 elements of K further: 32 bytes (in 16-byte units)
                    const uint64_t ds = da + (uint64_t)s * (OP_BYTES >> 4), es = db + (uint64_t)s * (OP_BYTES >> 4);
                    if ((use > 0 && !wait_all(&S.tempty[b], (use - 1) & 1u, &S.abort)) ||
                        !wait_all(&S.full[s], (g / STAGES) & 1u, &S.abort)) {
                        stop = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t acc = tmem + b * (uint32_t)BN;
                    if (elect_one()) {
#pragma unroll
                        for (int k = 0; k < BLK / 32; ++k) mma_fp8(acc, ds + 2 * k, es + 2 * k, k != 0 ? 1u : 0u);
                        mma_commit(&S.tfull[b]);
                        mma_commit(&S.empty[s]);
                    }
                    __syncwarp();
                }
            }
            if (elect_one()) mma_commit(&S.done);
        }
        __syncwarp();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int q = warp & 3, half = (warp - 4) >> 2;
        const bool vec = (ldd & 3) == 0 && (reinterpret_cast<uintptr_t>(D) & 15u) == 0;
        float* const stage = S.out[warp - 4];
        const uint32_t tempty[2] = {map_to_rank(&S.tempty[0], 0), map_to_rank(&S.tempty[1], 0)};
        uint32_t g = 0;
        bool lost = false;
        for (int t = cid; t < tiles; t += ncl) {
            int m0, n0;
            tile_at(t, m0, n0);
            const int r0 = m0 + HALF * rank + 32 * q, c0 = n0 + 128 * half;
            const bool any = r0 < M && c0 < N;        // something of this warp's part is inside
            const float* sap = sa + min(r0 + lane, M - 1);
            const float* sbp = sb + (long long)(min(c0, N - 1) / BLK) * nk;
            uint64_t acc[64];
#pragma unroll
            for (int j = 0; j < 64; ++j) acc[j] = 0;
            // the next block's scales, multiplied only when they are used: a product here would wait for
            // the loads (600 cycles a block)
            float na = any ? sap[0] : 0.f, nb = any ? sbp[0] : 0.f;
            for (int kb = 0; kb < nk; ++kb, ++g) {
                const uint32_t b = g & 1u;
                const float fa = na, fb = nb;
                if (any && kb + 1 < nk) {
                    na = sap[(long long)(kb + 1) * M];
                    nb = sbp[kb + 1];
                }
                // A lane whose wait ran out goes on with the others: a tensor-memory load is the whole warp's.  (Agreeing
                // on it at every block costs 1.5% at 2048 x 128256 x 4096.)
                lost = lost || !wait_parity<false>(&S.tfull[b], (g >> 1) & 1u, &S.abort, &g_watchdog);
                tc_fence_after();
                const uint32_t ta0 = tmem + ((uint32_t)(32 * q) << 16) + b * (uint32_t)BN + 128u * half;
                if (any) {
                    uint32_t v[2][32];
                    const uint64_t sc = both(fa * fb);
                    auto add = [&](int c) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            acc[16 * c + j] = fma2(sc, pack2(__uint_as_float(v[c & 1][2 * j]), __uint_as_float(v[c & 1][2 * j + 1])),
                                                   acc[16 * c + j]);
                    };
                    tmem_ld32(ta0, v[0]);
                    tmem_ld32(ta0 + 32u, v[1]);
                    tmem_wait(v[0], v[1]);
                    add(0);
                    tmem_ld32(ta0 + 64u, v[0]);
                    add(1);
                    tmem_ld32(ta0 + 96u, v[1]);
                    tmem_wait(v[0], v[1]);
                    tc_fence_before();                // the buffer has been read
                    if (lane == 0 && !lost) arrive_cluster(tempty[b]);
                    add(2);
                    add(3);
                } else if (lane == 0 && !lost) {
                    arrive_cluster(tempty[b]);
                }
            }
            if (__any_sync(0xffffffffu, lost) || !any) continue;
            const uint64_t al = both(alpha);
            const int rows = min(32, M - r0);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int cc = c0 + 32 * c;
                __syncwarp();
                // row `lane`'s eight 16-byte pieces, their places rotated by the row so that neither the
                // writes nor the reads of whole rows meet in a bank
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    float x[4];
                    unpack2(mul2(acc[16 * c + 2 * j], al), x[0], x[1]);
                    unpack2(mul2(acc[16 * c + 2 * j + 1], al), x[2], x[3]);
                    *reinterpret_cast<float4*>(stage + 32 * lane + 4 * (j ^ (lane & 7))) = make_float4(x[0], x[1], x[2], x[3]);
                }
                __syncwarp();
                if (cc >= N) continue;
                if (vec && cc + 32 <= N) {
                    const int p = lane & 7;
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int r = 4 * i + (lane >> 3);
                        const float4 x = *reinterpret_cast<const float4*>(stage + 32 * r + 4 * (p ^ (r & 7)));
                        if (r < rows) *reinterpret_cast<float4*>(D + (long long)(r0 + r) * ldd + cc + 4 * p) = x;
                    }
                } else {
                    for (int r = 0; r < rows; ++r)
                        if (cc + lane < N)
                            D[(long long)(r0 + r) * ldd + cc + lane] = stage[32 * r + 4 * ((lane >> 2) ^ (r & 7)) + (lane & 3)];
                }
            }
        }
    }
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
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(TMEM_COLS) : "memory");
    }
}

// ---------------------------------------------------------------- few rows

// M <= 64 rows: what has to be read is the weight plane, so it is the weight's 128-row tiles that
// fill the tensor cores' 128 lanes (D^T = B A^T, M = 128 weight rows, N = NT rows of A rounded up),
// and two CTAs an SM stream them.  A pair's tile of the kernel above would spend 540 cycles of MMA on
// 32 KB of weights, which HBM brings an SM in 1500; here it is 64 to 128 on 16 KB.  (8 rows x 32000 x
// 4096: 26 us against 40; 64 x 128256 x 4096: 99 us, 0.83 of the copy rate; a 128-row form of this
// kernel took 162 us at 128256 columns, the one above 131.)  Per CTA: warp 0
// the TMA producer, warp 1 the MMAs (into one of two tensor-memory buffers), warps 2-5 the epilogue:
// a thread has one weight row and the NT columns; a block's scales differ by column and come from
// shared memory, brought eight blocks at a time, one batch ahead.  A warp's lanes are neighbouring
// columns of D, so D is stored straight from registers.
constexpr int XB = 8;                    // blocks of K whose scales are brought at once

template <int NT>
struct Thin {
    static constexpr int STAGES = NT <= 16 ? 6 : NT <= 32 ? 5 : 4;
    static constexpr int X_BYTES = NT * BLK;
    static constexpr uint32_t COLS = 2 * NT < 32 ? 32 : 2 * NT;
    static constexpr uint32_t IDESC = (1u << 4) | ((uint32_t)(NT >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
};

template <int NT>
struct alignas(1024) TSmem {
    uint8_t w[Thin<NT>::STAGES][OP_BYTES];
    uint8_t x[Thin<NT>::STAGES][Thin<NT>::X_BYTES];
    alignas(16) float scale[2][XB][NT];
    uint64_t full[Thin<NT>::STAGES], empty[Thin<NT>::STAGES];
    uint64_t tfull[2], tempty[2], done;
    uint32_t tmem_base;
    int abort;
};
static_assert(2 * (sizeof(TSmem<16>) + 2048) <= 228 * 1024 && 2 * (sizeof(TSmem<32>) + 2048) <= 228 * 1024 &&
                  2 * (sizeof(TSmem<64>) + 2048) <= 228 * 1024, "shared memory of an SM's two CTAs");

__device__ __forceinline__ void tma_load_1cta(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void mma_1cta(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(acc) : "memory");
}
__device__ __forceinline__ void commit_1cta(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" :: "r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 "
                 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
                   "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                      "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// W [N][K] with scales sw [ceil(N/128)][nk]; X [M][K] with scales sx [nk][M]; D [M][ldd].
template <int NT>
__global__ void __launch_bounds__(192, 2)
    fp8_gemm_thin(const __grid_constant__ CUtensorMap tw, const __grid_constant__ CUtensorMap tx, const float* sw,
                  const float* sx, float* D, long long ldd, int M, int N, int K, float alpha) {
    using C = Thin<NT>;
    extern __shared__ uint8_t gsm_raw[];
    TSmem<NT>& S = *reinterpret_cast<TSmem<NT>*>((reinterpret_cast<uintptr_t>(gsm_raw) + 1023) & ~uintptr_t(1023));
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const int tiles = (N + BLK - 1) / BLK, nk = (K + BLK - 1) / BLK;
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
        S.abort = 0;
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
        // the weights' first tiles on their way while the quantiser runs (8 x 32000 x 4096 with it: 26.6 -> 25.3 us)
        if (elect_one())
            for (int kb = 0; kb < min(nk, (int)C::STAGES); ++kb) tma_prefetch_2d(&tw, kb * BLK, (int)blockIdx.x * BLK);
        __syncwarp();
        pdl_wait_primary();
        uint32_t g = 0;
        bool stop = false;
        for (int t = blockIdx.x; t < tiles && !stop; t += gridDim.x)
            for (int kb = 0; kb < nk; ++kb, ++g) {
                const uint32_t s = g % C::STAGES, use = g / C::STAGES;
                if (use > 0 && !wait_all(&S.empty[s], (use - 1) & 1u, &S.abort)) {
                    stop = true;
                    break;
                }
                if (elect_one()) {
                    mbar_arrive_expect_tx(&S.full[s], OP_BYTES + C::X_BYTES);
                    tma_load_1cta(S.w[s], &tw, kb * BLK, t * BLK, &S.full[s]);
                    tma_load_1cta(S.x[s], &tx, kb * BLK, 0, &S.full[s]);
                }
                __syncwarp();
            }
        if (lane == 0)                   // every copy issued has landed before the CTA can leave
            for (uint32_t gg = g > (uint32_t)C::STAGES ? g - C::STAGES : 0u; gg < g; ++gg)
                wait_parity_drain(&S.full[gg % C::STAGES], (gg / C::STAGES) & 1u);
    } else if (warp == 1) {
        uint32_t g = 0;
        bool stop = false;
        const uint64_t dw = sw128_desc(smem_u32(S.w[0])), dx = sw128_desc(smem_u32(S.x[0]));
        for (int t = blockIdx.x; t < tiles && !stop; t += gridDim.x)
            for (int kb = 0; kb < nk; ++kb, ++g) {
                const uint32_t s = g % C::STAGES, b = g & 1u, use = g >> 1;
                if ((use > 0 && !wait_all(&S.tempty[b], (use - 1) & 1u, &S.abort)) ||
                    !wait_all(&S.full[s], (g / C::STAGES) & 1u, &S.abort)) {
                    stop = true;
                    break;
                }
                tc_fence_after();
                const uint64_t aw = dw + (uint64_t)s * (OP_BYTES >> 4), ax = dx + (uint64_t)s * (C::X_BYTES >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int k = 0; k < BLK / 32; ++k)
                        mma_1cta(tmem + b * (uint32_t)NT, aw + 2 * k, ax + 2 * k, C::IDESC, k != 0 ? 1u : 0u);
                    commit_1cta(&S.empty[s]);
                    commit_1cta(&S.tfull[b]);
                }
                __syncwarp();
            }
        if (elect_one()) commit_1cta(&S.done);
    } else {
        pdl_wait_primary();
        constexpr int PER = XB * NT / 128;           // scales of a batch that a thread brings
        const int q = warp & 3, tid = threadIdx.x - 64;
        uint32_t g = 0, batch = 0;
        bool lost = false;               // a wait ran out: the warp goes on through the barriers alone, which the others pass
        float na[PER], nb[PER];
        auto bring = [&](int t, int k0) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int e = tid + 128 * i, k = k0 + e / NT, m = e % NT;
                const bool in = t < tiles && m < M && k < nk;
                na[i] = in ? sx[(long long)k * M + m] : 0.f;
                nb[i] = in ? sw[(long long)t * nk + k] : 0.f;
            }
        };
        bring(blockIdx.x, 0);
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
            uint64_t acc[NT / 2];
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) acc[j] = 0;
            for (int k0 = 0; k0 < nk; k0 += XB, ++batch) {
                float* const sc = &S.scale[batch & 1u][0][0];
#pragma unroll
                for (int i = 0; i < PER; ++i) sc[tid + 128 * i] = na[i] * nb[i];
                named_sync(1, 128);
                if (k0 + XB < nk) bring(t, k0 + XB);
                else bring(t + gridDim.x, 0);
                for (int kb = k0; kb < min(k0 + XB, nk); ++kb, ++g) {
                    const uint32_t b = g & 1u;
                    if (!wait_all(&S.tfull[b], (g >> 1) & 1u, &S.abort)) {
                        lost = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t ta0 = tmem + ((uint32_t)(32 * q) << 16) + b * (uint32_t)NT;
                    const float* const sk = sc + (kb - k0) * NT;
#pragma unroll
                    for (int c = 0; c < NT / 16; ++c) {
                        uint32_t v[16];
                        tmem_ld16(ta0 + 16u * c, v);
                        tmem_wait16(v);
                        if (c == NT / 16 - 1) {       // the buffer has been read
                            tc_fence_before();
                            if (lane == 0) mbar_arrive(&S.tempty[b]);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float4 f = *reinterpret_cast<const float4*>(sk + 16 * c + 4 * j);
                            acc[8 * c + 2 * j] = fma2(pack2(f.x, f.y), pack2(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1])),
                                                      acc[8 * c + 2 * j]);
                            acc[8 * c + 2 * j + 1] = fma2(pack2(f.z, f.w), pack2(__uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3])),
                                                          acc[8 * c + 2 * j + 1]);
                        }
                    }
                }
            }
            const int n = t * BLK + 32 * q + lane;
            if (!lost && n < N) {
#pragma unroll
                for (int j = 0; j < NT / 2; ++j) {
                    float x, y;
                    unpack2(acc[j], x, y);
                    if (2 * j < M) D[(long long)(2 * j) * ldd + n] = alpha * x;
                    if (2 * j + 1 < M) D[(long long)(2 * j + 1) * ldd + n] = alpha * y;
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        wait_parity_drain(&S.done, 0u);  // every MMA issued has completed before the columns are freed
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(C::COLS) : "memory");
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// A 2-D map over a row-major byte matrix [rows][K] with boxes of box_rows x 128.
bool make_map(CUtensorMap* map, const void* base, long long rows, long long K, int box_rows) {
    const PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) return false;
    const cuuint64_t dims[2] = {(cuuint64_t)K, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)K};
    const cuuint32_t box[2] = {(cuuint32_t)BLK, (cuuint32_t)box_rows};
    const cuuint32_t estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

std::atomic<int> g_attr[64];

}  // namespace

template <typename T>
static cudaError_t quant_rows_go(const T* x, long long ldx, long long M, long long K, uint8_t* q, float* sa,
                                 cudaStream_t st) {
    const long long nkb = (K + BLK - 1) / BLK, ctas = (M * ((nkb + RUN - 1) / RUN) + 7) / 8;
    const long long grid = ctas < 16384 ? ctas : 16384;
    const bool vec = K % 4 == 0 && ldx % 4 == 0 && reinterpret_cast<uintptr_t>(x) % (4 * sizeof(T)) == 0 &&
                     reinterpret_cast<uintptr_t>(q) % 4 == 0;
    return vec ? launch_pdl(quant_rows<T, true>, grid, 256, 0, st, x, ldx, M, (int)K, q, sa)
               : launch_pdl(quant_rows<T, false>, grid, 256, 0, st, x, ldx, M, (int)K, q, sa);
}

cudaError_t launch_quant_rows(const void* x, int dtype, long long ldx, long long M, long long K, uint8_t* q, float* sa,
                              cudaStream_t st) {
    if (dtype == kBf16) return quant_rows_go(static_cast<const __nv_bfloat16*>(x), ldx, M, K, q, sa, st);
    return quant_rows_go(static_cast<const float*>(x), ldx, M, K, q, sa, st);
}

cudaError_t launch_quant_blocks(const void* w, long long N, long long K, uint8_t* q, float* sb, cudaStream_t st) {
    const long long blocks = (N + BLK - 1) / BLK * ((K + BLK - 1) / BLK), grid = blocks < 65536 ? blocks : 65536;
    const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(w);
    const bool vec = K % 4 == 0 && reinterpret_cast<uintptr_t>(w) % 8 == 0 && reinterpret_cast<uintptr_t>(q) % 4 == 0;
    return vec ? launch_pdl(quant_blocks<true>, grid, 256, 0, st, p, N, (int)K, q, sb)
               : launch_pdl(quant_blocks<false>, grid, 256, 0, st, p, N, (int)K, q, sb);
}

template <int NT>
static cudaError_t thin_go(const uint8_t* A, const float* sa, const uint8_t* B, const float* sb, float* D, long long M,
                           long long N, long long K, long long ldd, float alpha, int dev, int sms, cudaStream_t st) {
    static std::atomic<int> had[64];
    const size_t smem = sizeof(TSmem<NT>) + 1024;
    if (!had[dev].load(std::memory_order_acquire)) {
        const cudaError_t e =
            cudaFuncSetAttribute((const void*)fp8_gemm_thin<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        had[dev].store(1, std::memory_order_release);
    }
    CUtensorMap tw, tx;
    if (!make_map(&tw, B, N, K, BLK) || !make_map(&tx, A, M, K, NT)) return cudaErrorInvalidValue;
    const long long tiles = (N + BLK - 1) / BLK, most = 2ll * sms;
    return launch_pdl(fp8_gemm_thin<NT>, tiles < most ? tiles : most, 192, smem, st, tw, tx, sb, sa, D, ldd, (int)M, (int)N,
                      (int)K, alpha);
}

cudaError_t fp8_gemm_tn(const uint8_t* A, const float* sa, const uint8_t* B, const float* sb, float* D, long long M,
                        long long N, long long K, long long ldd, float alpha, cudaStream_t st) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const size_t smem = sizeof(GSmem) + 1024;
    if (!g_attr[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute((const void*)fp8_gemm, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        g_attr[dev].store(1, std::memory_order_release);
    }
    if ((sms = num_sms()) <= 0) return cudaErrorInvalidDevice;
    if (M <= 16) return thin_go<16>(A, sa, B, sb, D, M, N, K, ldd, alpha, dev, sms, st);
    if (M <= 32) return thin_go<32>(A, sa, B, sb, D, M, N, K, ldd, alpha, dev, sms, st);
    if (M <= 64) return thin_go<64>(A, sa, B, sb, D, M, N, K, ldd, alpha, dev, sms, st);
    CUtensorMap ta, tb;
    if (!make_map(&ta, A, M, K, HALF) || !make_map(&tb, B, N, K, HALF)) return cudaErrorInvalidValue;
    const long long tiles = (M + BM - 1) / BM * ((N + BN - 1) / BN);
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
    const long long pairs = tiles < sms / 2 ? tiles : sms / 2;
    return launch_pdl(fp8_gemm, 2 * pairs, GT, smem, st, ta, tb, sa, sb, D, ldd, (int)M, (int)N, (int)K, alpha,
                      M <= N ? 1 : 0);
}

unsigned int fp8_watchdog(bool clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_watchdog, sizeof(v)) != cudaSuccess) return 0xffffffffu;
    if (clear && v) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_watchdog, &z, sizeof(z)) != cudaSuccess) return 0xffffffffu;
    }
    return v;
}

}  // namespace vl
