// C entry points of the post-training operators: argument checks on the host, then one of
// the launches of post.cu, norm.cu or fp8.cu.  Declarations and contracts: include/vloss.h.
#include "vl_api.h"
#include "vl_internal.h"

#include <cmath>
#include <cstring>

using namespace vl;

namespace {

vl_status check_ptr(const void* p, const char* what, const char* fn) {
    if (p == nullptr) return fail(VL_EINVAL, "%s: %s is NULL", fn, what);
    return VL_OK;
}

bool overlap(const void* a, long long an, const void* b, long long bn) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return an > 0 && bn > 0 && x < y + (uintptr_t)bn && y < x + (uintptr_t)an;
}

// Bytes from the first element of a strided matrix to past its last.
long long span(long long rows, long long ld, long long cols, int es) {
    return rows > 0 ? ((rows - 1) * ld + cols) * es : 0;
}

// Whether two matrices of the same number of rows and columns share bytes.  Rows of one stride may lie between
// one another (the two halves of a wider buffer); of different strides, one matrix has to end before the other.
bool overlap_rows(const void* a, long long lda, int aes, const void* b, long long ldb, int bes, long long rows,
                  long long cols) {
    if (!overlap(a, span(rows, lda, cols, aes), b, span(rows, ldb, cols, bes))) return false;
    const long long pitch = lda * aes;
    if (rows < 2 || pitch != ldb * bes) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const long long ahead = (long long)((x < y ? y - x : x - y) % (uintptr_t)pitch);
    const long long d = x < y || ahead == 0 ? ahead : pitch - ahead;       // from a row of a to the next start of one of b
    return d < cols * aes || d + cols * bes > pitch;
}

// The logits and gradient of a post-training call.
vl_status check_logits(const void* x, int64_t ld, int64_t ntok, int64_t V, const void* g, int64_t ldg, int es,
                       const char* fn) {
    if (ntok < 0) return fail(VL_EINVAL, "%s: ntok < 0", fn);
    if (V < 1 || V > VL_MAX_COLS) return fail(VL_EINVAL, "%s: V must be in [1, %lld]", fn, (long long)VL_MAX_COLS);
    if (ld < V) return fail(VL_EINVAL, "%s: ld (%lld) < V (%lld)", fn, (long long)ld, (long long)V);
    if (ntok > 0 && x == nullptr) return fail(VL_EINVAL, "%s: logits is NULL", fn);
    if (ntok > (1LL << 62) / 4 / ld) return fail(VL_EINVAL, "%s: ntok * ld is out of range", fn);
    if (g != nullptr) {
        if (ldg < V) return fail(VL_EINVAL, "%s: ldg (%lld) < V (%lld)", fn, (long long)ldg, (long long)V);
        if (ntok > (1LL << 62) / 4 / ldg) return fail(VL_EINVAL, "%s: ntok * ldg is out of range", fn);
        if (g == x) {
            if (ldg != ld) return fail(VL_EINVAL, "%s: in place needs ldg == ld", fn);
        } else if (overlap_rows(x, ld, es, g, ldg, es, ntok, V)) {
            return fail(VL_EINVAL, "%s: grad overlaps logits (it may be logits itself, or apart from it)", fn);
        }
    }
    return VL_OK;
}

vl_status policy_impl(const char* fn, const void* logits, int dtype, int64_t ld, int64_t ntok, int64_t V,
                      const uint32_t* actions, const float* old_logp, const float* ref_logp, const float* adv,
                      const float* weight, float clip_lo, float clip_hi, float kl_coef, float scale, void* grad,
                      int64_t ldg, float* loss, float* logp, float* kl, float* total, int32_t* err, void* stream) {
    vl_status s = check_logits(logits, ld, ntok, V, grad, ldg, dtype == kBf16 ? 2 : 4, fn);
    if (s) return s;
    if (!(clip_lo >= 0.f && clip_lo <= 1.f)) return fail(VL_EINVAL, "%s: clip_lo must be in [0, 1]", fn);
    if (!(clip_hi >= 0.f)) return fail(VL_EINVAL, "%s: clip_hi must be >= 0", fn);
    if (ntok > 0) {
        if ((s = check_ptr(actions, "actions", fn)) || (s = check_ptr(old_logp, "old_logp", fn)) ||
            (s = check_ptr(adv, "adv", fn)) || (s = check_ptr(weight, "weight", fn)) ||
            (s = check_ptr(loss, "loss", fn)))
            return s;
    } else if (total == nullptr) {
        return VL_OK;
    }
    PostParams P;
    std::memset(&P, 0, sizeof(P));
    P.x = logits;
    P.dtype = dtype;
    P.ld = ld;
    P.ntok = ntok;
    P.V = V;
    P.label = actions;
    P.weight = weight;
    P.old_logp = old_logp;
    P.ref_logp = ref_logp;
    P.adv = adv;
    P.lo = 1.f - clip_lo;
    P.hi = 1.f + clip_hi;
    P.kl_coef = kl_coef;
    P.scale = scale;
    P.g = grad;
    P.ldg = ldg;
    P.loss = loss;
    P.logp = logp;
    P.kl = kl;
    P.err = err;
    const cudaError_t e = launch_policy(P, total, as_stream(stream));
    return e == cudaSuccess ? VL_OK : cuda_fail(e, fn);
}

vl_status preference_impl(const char* fn, const void* logits, int dtype, int64_t ld, int64_t ntok, int64_t V,
                          const uint32_t* labels, const float* weight, const int64_t* seq_start, int64_t npairs,
                          const float* ref_logp, float beta, float smooth, int kind, float scale, void* grad,
                          int64_t ldg, float* loss, float* margin, float* seq_logp, float* mean, int32_t* err,
                          void* workspace, int64_t workspace_bytes, void* stream) {
    vl_status s = check_logits(logits, ld, ntok, V, grad, ldg, dtype == kBf16 ? 2 : 4, fn);
    if (s) return s;
    if (npairs < 0 || npairs > (1LL << 30)) return fail(VL_EINVAL, "%s: npairs must be in [0, 2^30]", fn);
    if (ntok > 0 && npairs == 0) return fail(VL_EINVAL, "%s: %lld rows but no pair", fn, (long long)ntok);
    if (kind != VL_PREF_SIGMOID && kind != VL_PREF_IPO && kind != VL_PREF_HINGE)
        return fail(VL_EINVAL, "%s: unknown kind %d", fn, kind);
    if (!(beta > 0.f) || std::isinf(beta)) return fail(VL_EINVAL, "%s: beta must be positive", fn);
    if (!(smooth >= 0.f && smooth < 1.f)) return fail(VL_EINVAL, "%s: smooth must be in [0, 1)", fn);
    if (ntok > 0 && ((s = check_ptr(labels, "labels", fn)) || (s = check_ptr(weight, "weight", fn)))) return s;
    if (npairs > 0) {
        if ((s = check_ptr(seq_start, "seq_start", fn)) || (s = check_ptr(loss, "loss", fn)) ||
            (s = check_ptr(margin, "margin", fn)))
            return s;
    } else if (mean == nullptr) {
        return VL_OK;
    }
    const int64_t need = vl_preference_workspace_bytes(ntok, npairs);
    if (need > 0) {
        if (workspace == nullptr || workspace_bytes < need)
            return fail(VL_EINVAL, "%s: needs %lld bytes of workspace", fn, (long long)need);
        if (reinterpret_cast<uintptr_t>(workspace) & 15u)
            return fail(VL_EINVAL, "%s: workspace must be 16-byte aligned", fn);
    }
    float* ws = static_cast<float*>(workspace);
    PostParams P;
    std::memset(&P, 0, sizeof(P));
    P.x = logits;
    P.dtype = dtype;
    P.ld = ld;
    P.ntok = ntok;
    P.V = V;
    P.label = labels;
    P.weight = weight;
    P.scale = scale;
    P.g = grad;
    P.ldg = ldg;
    P.stats = ws;
    P.logp = ws ? ws + 2 * ntok : nullptr;
    P.coef = ws ? ws + 3 * ntok : nullptr;
    P.err = err;
    PairParams Q;
    std::memset(&Q, 0, sizeof(Q));
    Q.weight = weight;
    Q.logp = P.logp;
    Q.coef = P.coef;
    Q.start = reinterpret_cast<const long long*>(seq_start);
    Q.ref = ref_logp;
    Q.ntok = ntok;
    Q.npairs = npairs;
    Q.beta = beta;
    Q.smooth = smooth;
    Q.scale = scale;
    Q.kind = kind;
    Q.loss = loss;
    Q.margin = margin;
    Q.seq = seq_logp;
    Q.mean = mean;
    const cudaError_t e = launch_preference(P, Q, as_stream(stream));
    return e == cudaSuccess ? VL_OK : cuda_fail(e, fn);
}

vl_status check_norm(const char* fn, const void* p, const char* what, int64_t ld, int64_t rows, int64_t hs) {
    if (rows < 0) return fail(VL_EINVAL, "%s: rows < 0", fn);
    if (hs < 1) return fail(VL_EINVAL, "%s: hs must be positive", fn);
    if (hs > VL_NORM_MAX_HS) return fail(VL_EUNSUPPORTED, "%s: hs above %d", fn, VL_NORM_MAX_HS);
    if (ld < hs) return fail(VL_EINVAL, "%s: the stride of %s (%lld) < hs (%lld)", fn, what, (long long)ld, (long long)hs);
    if (rows > (1LL << 62) / 4 / ld) return fail(VL_EINVAL, "%s: rows * stride of %s is out of range", fn, what);
    if (rows > 0 && p == nullptr) return fail(VL_EINVAL, "%s: %s is NULL", fn, what);
    return VL_OK;
}

// An output may be an input itself (same address and stride, same element size), or apart from it.
vl_status check_alias(const char* fn, const void* out, const char* oname, int64_t ldo, int oes, const void* in,
                      const char* iname, int64_t ldi, int ies, int64_t rows, int64_t hs) {
    if (out == in && ldo == ldi && oes == ies) return VL_OK;
    if (overlap_rows(out, ldo, oes, in, ldi, ies, rows, hs))
        return fail(VL_EINVAL, "%s: %s overlaps %s (it may be %s itself, with the same type and stride)", fn, oname, iname,
                    iname);
    return VL_OK;
}

vl_status norm_fwd_impl(const char* fn, const void* x, int dtype, int64_t ldx, int64_t rows, int64_t hs,
                        const float* gamma, const float* beta, float eps, void* y, int64_t ldy, float* mu, float* rstd,
                        void* stream) {
    vl_status s = check_norm(fn, x, "x", ldx, rows, hs);
    if (s || (s = check_norm(fn, y, "y", ldy, rows, hs))) return s;
    if (!(eps >= 0.f)) return fail(VL_EINVAL, "%s: eps must be >= 0", fn);
    const int es = dtype == kBf16 ? 2 : 4;
    if ((s = check_alias(fn, y, "y", ldy, es, x, "x", ldx, es, rows, hs))) return s;
    if (rows == 0) return VL_OK;
    NormParams P;
    std::memset(&P, 0, sizeof(P));
    P.x = x;
    P.dtype = dtype;
    P.ldx = ldx;
    P.rows = rows;
    P.hs = (int)hs;
    P.gamma = gamma;
    P.beta = beta;
    P.eps = eps;
    P.y = y;
    P.ldy = ldy;
    P.mu_out = mu;
    P.rstd_out = rstd;
    const cudaError_t e = launch_norm_fwd(P, as_stream(stream));
    return e == cudaSuccess ? VL_OK : cuda_fail(e, fn);
}

vl_status norm_bwd_impl(const char* fn, const void* dy, int dy_f32, int64_t lddy, const void* x, int dtype, int64_t ldx,
                        int64_t rows, int64_t hs, const float* gamma, const float* mu, const float* rstd, void* dx,
                        int64_t lddx, float* dgamma, float* dbeta, void* ws, int64_t ws_bytes, void* stream) {
    vl_status s = check_norm(fn, x, "x", ldx, rows, hs);
    if (s || (s = check_norm(fn, dy, "dy", lddy, rows, hs)) || (s = check_norm(fn, dx, "dx", lddx, rows, hs))) return s;
    if (rows > 0 && ((s = check_ptr(mu, "mu", fn)) || (s = check_ptr(rstd, "rstd", fn)))) return s;
    const int es = dtype == kBf16 ? 2 : 4, des = dy_f32 ? 4 : 2;
    if ((s = check_alias(fn, dx, "dx", lddx, es, x, "x", ldx, es, rows, hs)) ||
        (s = check_alias(fn, dx, "dx", lddx, es, dy, "dy", lddy, des, rows, hs)))
        return s;
    if (dgamma || dbeta) {
        const int64_t need = vl_layernorm_bwd_workspace_bytes(rows, hs);
        if (need > 0 && (ws == nullptr || ws_bytes < need))
            return fail(VL_EINVAL, "%s: needs %lld bytes of workspace", fn, (long long)need);
        if (reinterpret_cast<uintptr_t>(ws) & 15u) return fail(VL_EINVAL, "%s: workspace must be 16-byte aligned", fn);
    } else if (rows == 0) {
        return VL_OK;
    }
    NormParams P;
    std::memset(&P, 0, sizeof(P));
    P.x = x;
    P.dtype = dtype;
    P.ldx = ldx;
    P.rows = rows;
    P.hs = (int)hs;
    P.gamma = gamma;
    P.y = dx;
    P.ldy = lddx;
    P.dy = dy;
    P.dy_f32 = dy_f32;
    P.lddy = lddy;
    P.mu = mu;
    P.rstd = rstd;
    P.dgamma = dgamma;
    P.dbeta = dbeta;
    P.part = static_cast<float*>(ws);
    const cudaError_t e = launch_norm_bwd(P, as_stream(stream));
    return e == cudaSuccess ? VL_OK : cuda_fail(e, fn);
}

vl_status quant_check(const char* fn, const void* x, int64_t ldx, int64_t M, int64_t K, const void* q, const void* sc) {
    if (M < 0 || K < 0) return fail(VL_EINVAL, "%s: negative size", fn);
    // the kernels count a row's columns in 32-bit ints, a few blocks past its end
    if (K > (1LL << 30) || M > (1LL << 31)) return fail(VL_EINVAL, "%s: at most 2^31 rows of at most 2^30 columns", fn);
    if (ldx < K) return fail(VL_EINVAL, "%s: ldx (%lld) < K (%lld)", fn, (long long)ldx, (long long)K);
    if (M > 0 && ldx > 0 && M > (1LL << 62) / 4 / ldx) return fail(VL_EINVAL, "%s: M * ldx is out of range", fn);
    if (M > 0 && K > 0 && (!x || !q || !sc)) return fail(VL_EINVAL, "%s: NULL pointer", fn);
    return VL_OK;
}

}  // namespace

extern "C" {

vl_status vl_policy_loss(const float* logits, int64_t ld, int64_t ntok, int64_t V, const uint32_t* actions,
                         const float* old_logp, const float* ref_logp, const float* adv, const float* weight,
                         float clip_lo, float clip_hi, float kl_coef, float scale, float* grad, int64_t ldg, float* loss,
                         float* logp, float* kl, float* total, int32_t* err, void* stream) {
    return policy_impl("vl_policy_loss", logits, kF32, ld, ntok, V, actions, old_logp, ref_logp, adv, weight, clip_lo,
                       clip_hi, kl_coef, scale, grad, ldg, loss, logp, kl, total, err, stream);
}

vl_status vl_policy_loss_bf16(const uint16_t* logits, int64_t ld, int64_t ntok, int64_t V, const uint32_t* actions,
                              const float* old_logp, const float* ref_logp, const float* adv, const float* weight,
                              float clip_lo, float clip_hi, float kl_coef, float scale, uint16_t* grad, int64_t ldg,
                              float* loss, float* logp, float* kl, float* total, int32_t* err, void* stream) {
    return policy_impl("vl_policy_loss_bf16", logits, kBf16, ld, ntok, V, actions, old_logp, ref_logp, adv, weight,
                       clip_lo, clip_hi, kl_coef, scale, grad, ldg, loss, logp, kl, total, err, stream);
}

// Per row: (m, lnS), the log-probability and the gradient's factor.
int64_t vl_preference_workspace_bytes(int64_t ntok, int64_t npairs) {
    (void)npairs;
    return ntok > 0 ? 16 * ntok : 0;
}

vl_status vl_preference_loss(const float* logits, int64_t ld, int64_t ntok, int64_t V, const uint32_t* labels,
                             const float* weight, const int64_t* seq_start, int64_t npairs, const float* ref_logp,
                             float beta, float smooth, int kind, float scale, float* grad, int64_t ldg, float* loss,
                             float* margin, float* seq_logp, float* mean, int32_t* err, void* workspace,
                             int64_t workspace_bytes, void* stream) {
    return preference_impl("vl_preference_loss", logits, kF32, ld, ntok, V, labels, weight, seq_start, npairs, ref_logp,
                           beta, smooth, kind, scale, grad, ldg, loss, margin, seq_logp, mean, err, workspace,
                           workspace_bytes, stream);
}

vl_status vl_preference_loss_bf16(const uint16_t* logits, int64_t ld, int64_t ntok, int64_t V, const uint32_t* labels,
                                  const float* weight, const int64_t* seq_start, int64_t npairs, const float* ref_logp,
                                  float beta, float smooth, int kind, float scale, uint16_t* grad, int64_t ldg,
                                  float* loss, float* margin, float* seq_logp, float* mean, int32_t* err,
                                  void* workspace, int64_t workspace_bytes, void* stream) {
    return preference_impl("vl_preference_loss_bf16", logits, kBf16, ld, ntok, V, labels, weight, seq_start, npairs,
                           ref_logp, beta, smooth, kind, scale, grad, ldg, loss, margin, seq_logp, mean, err, workspace,
                           workspace_bytes, stream);
}

vl_status vl_layernorm_fwd(const float* x, int64_t ldx, int64_t rows, int64_t hs, const float* gamma, const float* beta,
                           float eps, float* y, int64_t ldy, float* mu, float* rstd, void* stream) {
    return norm_fwd_impl("vl_layernorm_fwd", x, kF32, ldx, rows, hs, gamma, beta, eps, y, ldy, mu, rstd, stream);
}

vl_status vl_layernorm_fwd_bf16(const uint16_t* x, int64_t ldx, int64_t rows, int64_t hs, const float* gamma,
                                const float* beta, float eps, uint16_t* y, int64_t ldy, float* mu, float* rstd,
                                void* stream) {
    return norm_fwd_impl("vl_layernorm_fwd_bf16", x, kBf16, ldx, rows, hs, gamma, beta, eps, y, ldy, mu, rstd, stream);
}

int64_t vl_layernorm_bwd_workspace_bytes(int64_t rows, int64_t hs) {
    if (rows < 1 || hs < 1 || hs > VL_NORM_MAX_HS) return 0;
    return norm_bwd_ws_bytes(rows, hs);
}

vl_status vl_layernorm_bwd(const float* dy, int64_t lddy, const float* x, int64_t ldx, int64_t rows, int64_t hs,
                           const float* gamma, const float* mu, const float* rstd, float* dx, int64_t lddx,
                           float* dgamma, float* dbeta, void* workspace, int64_t workspace_bytes, void* stream) {
    return norm_bwd_impl("vl_layernorm_bwd", dy, 1, lddy, x, kF32, ldx, rows, hs, gamma, mu, rstd, dx, lddx, dgamma,
                         dbeta, workspace, workspace_bytes, stream);
}

vl_status vl_layernorm_bwd_bf16(const void* dy, int dy_f32, int64_t lddy, const uint16_t* x, int64_t ldx, int64_t rows,
                                int64_t hs, const float* gamma, const float* mu, const float* rstd, uint16_t* dx,
                                int64_t lddx, float* dgamma, float* dbeta, void* workspace, int64_t workspace_bytes,
                                void* stream) {
    return norm_bwd_impl("vl_layernorm_bwd_bf16", dy, dy_f32 != 0, lddy, x, kBf16, ldx, rows, hs, gamma, mu, rstd, dx,
                         lddx, dgamma, dbeta, workspace, workspace_bytes, stream);
}

vl_status vl_quant_fp8_rows(const float* x, int64_t ldx, int64_t M, int64_t K, uint8_t* q, float* sa, void* stream) {
    const char* fn = "vl_quant_fp8_rows";
    const vl_status s = quant_check(fn, x, ldx, M, K, q, sa);
    if (s || M == 0 || K == 0) return s;
    const cudaError_t e = launch_quant_rows(x, kF32, ldx, M, K, q, sa, as_stream(stream));
    return e == cudaSuccess ? VL_OK : cuda_fail(e, fn);
}

vl_status vl_quant_fp8_rows_bf16(const uint16_t* x, int64_t ldx, int64_t M, int64_t K, uint8_t* q, float* sa,
                                 void* stream) {
    const char* fn = "vl_quant_fp8_rows_bf16";
    const vl_status s = quant_check(fn, x, ldx, M, K, q, sa);
    if (s || M == 0 || K == 0) return s;
    const cudaError_t e = launch_quant_rows(x, kBf16, ldx, M, K, q, sa, as_stream(stream));
    return e == cudaSuccess ? VL_OK : cuda_fail(e, fn);
}

vl_status vl_quant_fp8_blocks_bf16(const uint16_t* w, int64_t N, int64_t K, uint8_t* q, float* sb, void* stream) {
    const char* fn = "vl_quant_fp8_blocks_bf16";
    const vl_status s = quant_check(fn, w, K, N, K, q, sb);
    if (s || N == 0 || K == 0) return s;
    const cudaError_t e = launch_quant_blocks(w, N, K, q, sb, as_stream(stream));
    return e == cudaSuccess ? VL_OK : cuda_fail(e, fn);
}

vl_status vl_gemm_fp8_tn(const uint8_t* A, const float* sa, const uint8_t* B, const float* sb, float* D, int64_t M,
                         int64_t N, int64_t K, int64_t ldd, float alpha, void* stream) {
    const char* fn = "vl_gemm_fp8_tn";
    if (M < 0 || N < 0 || K < 16 || K % 16 != 0) return fail(VL_EINVAL, "%s: need M, N >= 0 and K a positive multiple of 16", fn);
    if (M > (1LL << 30) || N > (1LL << 30) || K > (1LL << 30)) return fail(VL_EINVAL, "%s: sizes must be at most 2^30", fn);
    if (ldd < N) return fail(VL_EINVAL, "%s: ldd (%lld) < N (%lld)", fn, (long long)ldd, (long long)N);
    if (M == 0 || N == 0) return VL_OK;
    if (!A || !B || !sa || !sb || !D) return fail(VL_EINVAL, "%s: NULL pointer", fn);
    if ((reinterpret_cast<uintptr_t>(A) | reinterpret_cast<uintptr_t>(B)) & 15u)
        return fail(VL_EINVAL, "%s: A and B must be 16-byte aligned", fn);
    const cudaError_t e = fp8_gemm_tn(A, sa, B, sb, D, M, N, K, ldd, alpha, as_stream(stream));
    return e == cudaSuccess ? VL_OK : cuda_fail(e, fn);
}

}  // extern "C"
