// The head's product in 8-bit floating point (sm_103a): D[M][N] = alpha sum over blocks b of 128
// along K of sa[b][m] sb[n / 128][b] (sum over k in b of A[m][k] B[n][k]), A and B e4m3, and the
// quantisers that make A (a scale for each 1 x 128) and B (a scale for each 128 x 128).
//
// The scales change from one block of K to the next, so a block's sum cannot stay in the tensor
// cores' accumulator: each block's 128 x 256 sum lands in one of two tensor-memory buffers, and
// eight epilogue warps add it, scaled, to fp32 registers while the tensor cores work on the next
// block.  One persistent CTA per SM walks 128 x 256 tiles of D:
//   warp 0    TMA producer: boxes of 128 x 128 (A) and 256 x 128 (B) bytes, 128-byte swizzle, one
//             block of K a stage, into a 4-stage ring;
//   warp 1    tcgen05.mma (kind::f8f6f4, M = 128, N = 256, K = 32; four a stage) into the buffer
//             of the block's parity, once the epilogue has handed it back;
//   warps 2-9 the epilogue: 32 rows (tensor-memory lanes) x 128 columns a warp, so that a thread
//             has one row and one 128-column group: one scale a block.
// Rows, columns and K past the edges: the TMA fills zeros, the epilogue masks stores.
#include "vl_device.cuh"
#include "vl_internal.h"
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
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, off));
    return a;
}

// One warp a block of 1 x 128: lane l takes elements 4 l .. 4 l + 3.
template <typename T>
__global__ void __launch_bounds__(256) quant_rows(const T* __restrict__ x, long long ldx, long long M, int K,
                                                  uint8_t* __restrict__ q, float* __restrict__ sa) {
    pdl_wait_primary();
    pdl_launch_dependents();
    const int nkb = (K + BLK - 1) / BLK, lane = threadIdx.x & 31;
    const long long total = M * nkb, stride = (long long)gridDim.x * 8;
    for (long long i = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); i < total; i += stride) {
        const long long m = i / nkb;
        const int kb = (int)(i % nkb), k0 = kb * BLK + 4 * lane;
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = k0 + j < K ? ld_elem(x + m * ldx + k0 + j) : 0.f;
        const float amax = warp_max(fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3]))));
        const float s = __fmul_rn(fmaxf(amax, kAmaxFloor), kInvE4m3Max);
        const uint32_t w = e4m3x2(__fdiv_rn(v[0], s), __fdiv_rn(v[1], s)) |
                           e4m3x2(__fdiv_rn(v[2], s), __fdiv_rn(v[3], s)) << 16;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (k0 + j < K) q[m * K + k0 + j] = (uint8_t)(w >> (8 * j));
        if (lane == 0) sa[kb * M + m] = s;
    }
}

// One CTA a block of 128 x 128.
__global__ void __launch_bounds__(256) quant_blocks(const __nv_bfloat16* __restrict__ w, long long N, int K,
                                                    uint8_t* __restrict__ q, float* __restrict__ sb) {
    __shared__ float red[8];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int nkb = (K + BLK - 1) / BLK, lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
    const long long blocks = (N + BLK - 1) / BLK * nkb;
    for (long long i = blockIdx.x; i < blocks; i += gridDim.x) {
        const long long n0 = i / nkb * BLK;
        const int k0 = (int)(i % nkb) * BLK + 4 * lane;
        float amax = 0.f;
        for (int r = wp; r < BLK && n0 + r < N; r += 8)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k0 + j < K) amax = fmaxf(amax, fabsf(ld_elem(w + (n0 + r) * K + k0 + j)));
        amax = warp_max(amax);
        __syncthreads();
        if (lane == 0) red[wp] = amax;
        __syncthreads();
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, red[j]);
        const float s = __fmul_rn(fmaxf(amax, kAmaxFloor), kInvE4m3Max);
        for (int r = wp; r < BLK && n0 + r < N; r += 8) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = k0 + j < K ? ld_elem(w + (n0 + r) * K + k0 + j) : 0.f;
            const uint32_t b = e4m3x2(__fdiv_rn(v[0], s), __fdiv_rn(v[1], s)) |
                               e4m3x2(__fdiv_rn(v[2], s), __fdiv_rn(v[3], s)) << 16;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (k0 + j < K) q[(n0 + r) * K + k0 + j] = (uint8_t)(b >> (8 * j));
        }
        if (threadIdx.x == 0) sb[i] = s;
    }
}

// ---------------------------------------------------------------- the product

constexpr int BM = 128, BN = 256, STAGES = 4;
constexpr int A_BYTES = BM * BLK;
constexpr int B_BYTES = BN * BLK;
constexpr int EPI_WARPS = 8;
constexpr int GT = 64 + 32 * EPI_WARPS;
constexpr uint32_t TMEM_COLS = 2 * BN;

struct alignas(1024) GSmem {
    uint8_t a[STAGES][A_BYTES];
    uint8_t b[STAGES][B_BYTES];
    uint64_t full[STAGES];
    uint64_t empty[STAGES];
    uint64_t tfull[2];                   // a block's sum is complete (MMA commit)
    uint64_t tempty[2];                  // the epilogue has read it
    uint64_t done;
    uint32_t tmem_base;
    int abort;
};

// K-major operand tile of 128-byte rows, 128-byte swizzle, groups of 8 rows 1024 bytes apart
// (fields as in the bf16 product); 32 elements of K are 32 bytes.
__device__ __forceinline__ uint64_t sw128_desc(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

// kind::f8f6f4: D f32 (bits 4-5 = 1), A and B e4m3 (7-9, 10-12 = 0), both K-major, N >> 3, M >> 4.
constexpr uint32_t kIdesc = (1u << 4) | ((uint32_t)(BN >> 3) << 17) | ((uint32_t)(BM >> 4) << 24);

__device__ __forceinline__ void tma_load_2d(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
    asm volatile("cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
                 :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ void mma_fp8(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                 "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
                 :: "r"(tmem_d), "l"(adesc), "l"(bdesc), "r"(kIdesc), "r"(acc) : "memory");
}

__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 :: "r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

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
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
    // the registers pass through the wait, so that nothing reads them before it
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                   "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                   "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                   "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28])
                 :: "memory");
    asm volatile("" : "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) :: "memory");
}

__global__ void __launch_bounds__(GT, 1) fp8_gemm(const __grid_constant__ CUtensorMap ta,
                                                  const __grid_constant__ CUtensorMap tb, const float* __restrict__ sa,
                                                  const float* __restrict__ sb, float* __restrict__ D, long long ldd,
                                                  int M, int N, int K, float alpha, int m_fast) {
    extern __shared__ uint8_t gsm_raw[];
    GSmem& S = *reinterpret_cast<GSmem*>((reinterpret_cast<uintptr_t>(gsm_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
            mbar_init(&S.tempty[b], EPI_WARPS);
        }
        mbar_init(&S.done, 1);
        S.abort = 0;
        fence_mbar_init_cluster();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(&S.tmem_base)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait_primary();
    pdl_launch_dependents();
    const uint32_t tmem = S.tmem_base;

    if (warp == 0) {
        if (lane == 0) {
            uint32_t g = 0, issued = 0;
            bool stop = false;
            for (int t = blockIdx.x; t < tiles && !stop; t += gridDim.x) {
                int m0, n0;
                tile_at(t, m0, n0);
                for (int kb = 0; kb < nk; ++kb, ++g) {
                    const uint32_t s = g % STAGES, use = g / STAGES;
                    if (use > 0 && !wait_parity<false>(&S.empty[s], (use - 1) & 1u, &S.abort, &g_watchdog)) {
                        stop = true;
                        break;
                    }
                    mbar_arrive_expect_tx(&S.full[s], A_BYTES + B_BYTES);
                    tma_load_2d(S.a[s], &ta, kb * BLK, m0, &S.full[s]);
                    tma_load_2d(S.b[s], &tb, kb * BLK, n0, &S.full[s]);
                    issued = g + 1;
                }
            }
            for (uint32_t gg = issued > (uint32_t)STAGES ? issued - STAGES : 0u; gg < issued; ++gg)
                wait_parity_drain(&S.full[gg % STAGES], (gg / STAGES) & 1u);
        }
    } else if (warp == 1) {
        if (lane == 0) {
            uint32_t g = 0;
            bool stop = false;
            for (int t = blockIdx.x; t < tiles && !stop; t += gridDim.x) {
                for (int kb = 0; kb < nk; ++kb, ++g) {
                    const uint32_t s = g % STAGES, b = g & 1u, use = g >> 1;
                    if ((use > 0 && !wait_parity<false>(&S.tempty[b], (use - 1) & 1u, &S.abort, &g_watchdog)) ||
                        !wait_parity<false>(&S.full[s], (g / STAGES) & 1u, &S.abort, &g_watchdog)) {
                        stop = true;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t acc = tmem + b * (uint32_t)BN;
                    const uint32_t a0 = smem_u32(S.a[s]), b0 = smem_u32(S.b[s]);
#pragma unroll
                    for (int k = 0; k < BLK / 32; ++k)
                        mma_fp8(acc, sw128_desc(a0 + 32u * k), sw128_desc(b0 + 32u * k), k != 0 ? 1u : 0u);
                    mma_commit(&S.empty[s]);
                    mma_commit(&S.tfull[b]);
                }
            }
            mma_commit(&S.done);
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;
        const bool vec = (ldd & 3) == 0 && (reinterpret_cast<uintptr_t>(D) & 15u) == 0;
        uint32_t g = 0;
        bool stop = false;
        for (int t = blockIdx.x; t < tiles && !stop; t += gridDim.x) {
            int m0, n0;
            tile_at(t, m0, n0);
            const int row = m0 + 32 * q + lane, c0 = n0 + 128 * half;
            const float* sap = sa + min(row, M - 1);
            const float* sbp = sb + (long long)min(c0, N - 1) / BLK * nk;
            float acc[128];
#pragma unroll
            for (int j = 0; j < 128; ++j) acc[j] = 0.f;
            for (int kb = 0; kb < nk; ++kb, ++g) {
                const uint32_t b = g & 1u;
                const float sc = sap[(long long)kb * M] * sbp[kb];
                if (!wait_parity<false>(&S.tfull[b], (g >> 1) & 1u, &S.abort, &g_watchdog)) {
                    stop = true;
                    break;
                }
                tc_fence_after();
                const uint32_t ta0 = tmem + ((uint32_t)(32 * q) << 16) + b * (uint32_t)BN + 128u * half;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t v[32];
                    tmem_ld32(ta0 + 32u * c, v);
                    tmem_wait(v);
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[32 * c + j] = fmaf(sc, __uint_as_float(v[j]), acc[32 * c + j]);
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&S.tempty[b]);
            }
            if (stop || row >= M) continue;
            float* out = D + (long long)row * ldd + c0;
#pragma unroll
            for (int j = 0; j < 128; j += 4) {
                if (vec && c0 + j + 4 <= N) {
                    *reinterpret_cast<float4*>(out + j) =
                        make_float4(alpha * acc[j], alpha * acc[j + 1], alpha * acc[j + 2], alpha * acc[j + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (c0 + j + i < N) out[j + i] = alpha * acc[j + i];
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        wait_parity_drain(&S.done, 0u);
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" :: "r"(tmem), "r"(TMEM_COLS) : "memory");
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

cudaError_t device_sms(int dev, int* sms) {
    static std::atomic<int> cache[64];
    *sms = cache[dev].load(std::memory_order_acquire);
    if (*sms > 0) return cudaSuccess;
    const cudaError_t e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) cache[dev].store(*sms, std::memory_order_release);
    return e;
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

}  // namespace

cudaError_t launch_quant_rows(const void* x, int dtype, long long ldx, long long M, long long K, uint8_t* q, float* sa,
                              cudaStream_t st) {
    const long long warps = M * ((K + BLK - 1) / BLK), grid = (warps + 7) / 8 < 16384 ? (warps + 7) / 8 : 16384;
    if (dtype == kBf16)
        return launch_pdl(quant_rows<__nv_bfloat16>, grid, 256, 0, st, static_cast<const __nv_bfloat16*>(x), ldx, M, (int)K,
                          q, sa);
    return launch_pdl(quant_rows<float>, grid, 256, 0, st, static_cast<const float*>(x), ldx, M, (int)K, q, sa);
}

cudaError_t launch_quant_blocks(const void* w, long long N, long long K, uint8_t* q, float* sb, cudaStream_t st) {
    const long long blocks = (N + BLK - 1) / BLK * ((K + BLK - 1) / BLK);
    return launch_pdl(quant_blocks, blocks < 65536 ? blocks : 65536, 256, 0, st, static_cast<const __nv_bfloat16*>(w), N,
                      (int)K, q, sb);
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
    if ((e = device_sms(dev, &sms)) != cudaSuccess) return e;
    CUtensorMap ta, tb;
    if (!make_map(&ta, A, M, K, BM) || !make_map(&tb, B, N, K, BN)) return cudaErrorInvalidValue;
    const long long tiles = (M + BM - 1) / BM * ((N + BN - 1) / BN);
    if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
    return launch_pdl(fp8_gemm, tiles < sms ? tiles : sms, GT, smem, st, ta, tb, sa, sb, D, ldd, (int)M, (int)N, (int)K,
                      alpha, M <= N ? 1 : 0);
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
