// C ABI of the training-step operators between the GEMMs (declared in
// include/ufp4.h): argument checks and dispatch.  Nothing is launched when an
// argument is rejected, and nothing here allocates device memory.
#include <cmath>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/ufp4.h"
#include "train.h"

using namespace ufp4;

namespace {

ufp4_status to_status(cudaError_t e) {
    if (e == cudaSuccess) return UFP4_OK;
    return e == cudaErrorNotSupported ? UFP4_ERR_UNSUPPORTED : UFP4_ERR_CUDA;
}

bool is_dtype(int32_t t) { return t == UFP4_BF16 || t == UFP4_F32; }
int size_of(int32_t t) { return t == UFP4_F32 ? 4 : 2; }

// A rows x cols matrix with leading dimension ld, elements of `bytes` bytes.
ufp4_status check_matrix(const void* p, int64_t cols, int64_t ld, int bytes, bool optional) {
    if (!p) return optional ? UFP4_OK : UFP4_ERR_INVALID_ARG;
    if (ld < cols) return UFP4_ERR_INVALID_ARG;
    return (uintptr_t)p % bytes ? UFP4_ERR_ALIGNMENT : UFP4_OK;
}

ufp4_status check_ckpt(const ufp4_qtensor* q, int64_t rows, int64_t cols, Ckpt* out) {
    if (!q->codes || !q->scales || q->rows != rows || q->cols != cols) return UFP4_ERR_INVALID_ARG;
    if (q->codes_ld < cols || q->scales_ld < (cols + 31) / 32) return UFP4_ERR_INVALID_ARG;
    *out = {(uint8_t*)q->codes, (uint8_t*)q->scales, q->codes_ld, q->scales_ld};
    return UFP4_OK;
}

constexpr int64_t kMaxExtent = 1ll << 30;  // 32-bit column indices and tile counts

}  // namespace

#define UFP4_CHECK(expr)                          \
    do {                                          \
        const ufp4_status s_ = (expr);            \
        if (s_ != UFP4_OK) return s_;             \
    } while (0)

extern "C" {

ufp4_status ufp4_glu(const void* gate, int64_t ld_gate, const void* up, int64_t ld_up, int32_t in_dtype, int64_t rows,
                     int64_t cols, int32_t act, void* y, int64_t ldy, const ufp4_qtensor* ckpt_gate,
                     const ufp4_qtensor* ckpt_up, cudaStream_t stream) {
    if (rows < 0 || cols < 0 || !is_dtype(in_dtype) || (act != UFP4_ACT_SILU && act != UFP4_ACT_GELU))
        return UFP4_ERR_INVALID_ARG;
    if (!ckpt_gate != !ckpt_up) return UFP4_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return UFP4_OK;
    if (cols > kMaxExtent) return UFP4_ERR_UNSUPPORTED;
    GluArgs a = {};
    UFP4_CHECK(check_matrix(gate, cols, ld_gate, size_of(in_dtype), false));
    UFP4_CHECK(check_matrix(up, cols, ld_up, size_of(in_dtype), false));
    UFP4_CHECK(check_matrix(y, cols, ldy, 2, false));
    a.ckpt = ckpt_gate != nullptr;
    if (a.ckpt) {
        UFP4_CHECK(check_ckpt(ckpt_gate, rows, cols, &a.cg));
        UFP4_CHECK(check_ckpt(ckpt_up, rows, cols, &a.cu));
    }
    a.gate = gate;
    a.up = up;
    a.ld_gate = ld_gate;
    a.ld_up = ld_up;
    a.f32 = in_dtype == UFP4_F32;
    a.act = act;
    a.rows = rows;
    a.cols = cols;
    a.y = y;
    a.ldy = ldy;
    current_num_sms();  // loads the kernels
    return to_status(launch_glu(a, stream));
}

ufp4_status ufp4_glu_backward(const void* dy, int64_t ld_dy, int32_t dy_dtype, const ufp4_qtensor* ckpt_gate,
                              const ufp4_qtensor* ckpt_up, int64_t rows, int64_t cols, int32_t act, void* dgate,
                              int64_t ld_dgate, void* dup, int64_t ld_dup, void* y, int64_t ldy, cudaStream_t stream) {
    if (rows < 0 || cols < 0 || !is_dtype(dy_dtype) || (act != UFP4_ACT_SILU && act != UFP4_ACT_GELU))
        return UFP4_ERR_INVALID_ARG;
    if (!ckpt_gate || !ckpt_up) return UFP4_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return UFP4_OK;
    if (cols > kMaxExtent) return UFP4_ERR_UNSUPPORTED;
    GluArgs a = {};
    UFP4_CHECK(check_matrix(dy, cols, ld_dy, size_of(dy_dtype), false));
    UFP4_CHECK(check_ckpt(ckpt_gate, rows, cols, &a.cg));
    UFP4_CHECK(check_ckpt(ckpt_up, rows, cols, &a.cu));
    UFP4_CHECK(check_matrix(dgate, cols, ld_dgate, 2, false));
    UFP4_CHECK(check_matrix(dup, cols, ld_dup, 2, false));
    UFP4_CHECK(check_matrix(y, cols, ldy, 2, true));
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.f32 = dy_dtype == UFP4_F32;
    a.act = act;
    a.rows = rows;
    a.cols = cols;
    a.dgate = dgate;
    a.ld_dgate = ld_dgate;
    a.dup = dup;
    a.ld_dup = ld_dup;
    a.y = y;
    a.ldy = ldy;
    current_num_sms();  // loads the kernels
    return to_status(launch_glu_backward(a, stream));
}

ufp4_status ufp4_rms_norm(const void* x, int64_t ldx, int32_t x_dtype, const void* residual, int64_t ld_residual,
                          const void* gamma, int32_t gamma_dtype, int64_t rows, int64_t cols, float eps, void* y,
                          int64_t ldy, void* total, int64_t ld_total, float* rstd, const ufp4_qtensor* ckpt,
                          cudaStream_t stream) {
    if (rows < 0 || cols < 1 || !is_dtype(x_dtype) || !is_dtype(gamma_dtype)) return UFP4_ERR_INVALID_ARG;
    if (!(eps > 0.0f) || !std::isfinite(eps) || (ckpt && !rstd)) return UFP4_ERR_INVALID_ARG;
    if (rows == 0) return UFP4_OK;
    if (cols > kNormMaxCols) return UFP4_ERR_UNSUPPORTED;
    NormArgs a = {};
    UFP4_CHECK(check_matrix(x, cols, ldx, size_of(x_dtype), false));
    UFP4_CHECK(check_matrix(residual, cols, ld_residual, 2, true));
    UFP4_CHECK(check_matrix(gamma, cols, cols, size_of(gamma_dtype), false));
    UFP4_CHECK(check_matrix(y, cols, ldy, 2, false));
    UFP4_CHECK(check_matrix(total, cols, ld_total, 2, true));
    UFP4_CHECK(check_matrix(rstd, 1, 1, 4, true));
    a.ckpt = ckpt != nullptr;
    if (a.ckpt) UFP4_CHECK(check_ckpt(ckpt, rows, cols, &a.ck));
    a.x = x;
    a.ldx = ldx;
    a.f32 = x_dtype == UFP4_F32;
    a.residual = residual;
    a.ld_residual = ld_residual;
    a.gamma = gamma;
    a.gamma_f32 = gamma_dtype == UFP4_F32;
    a.rows = rows;
    a.cols = cols;
    a.eps = eps;
    a.y = y;
    a.ldy = ldy;
    a.total = total;
    a.ld_total = ld_total;
    a.rstd = rstd;
    return to_status(launch_rms_norm(a, current_num_sms(), stream));
}

ufp4_status ufp4_rms_norm_backward_workspace_size(int64_t rows, int64_t cols, size_t* bytes) {
    if (rows < 0 || cols < 1 || !bytes) return UFP4_ERR_INVALID_ARG;
    if (cols > kNormMaxCols) return UFP4_ERR_UNSUPPORTED;
    *bytes = (size_t)norm_parts(rows, cols, current_num_sms()) * (size_t)cols * sizeof(float);
    return UFP4_OK;
}

ufp4_status ufp4_rms_norm_backward(const void* dy, int64_t ld_dy, int32_t dy_dtype, const ufp4_qtensor* ckpt,
                                   const float* rstd, const void* gamma, int32_t gamma_dtype, const void* dtotal,
                                   int64_t ld_dtotal, int64_t rows, int64_t cols, void* dx, int64_t ld_dx,
                                   float* dgamma, void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
    if (rows < 0 || cols < 1 || !is_dtype(dy_dtype) || !is_dtype(gamma_dtype)) return UFP4_ERR_INVALID_ARG;
    if (cols > kNormMaxCols) return UFP4_ERR_UNSUPPORTED;
    NormArgs a = {};
    if (rows > 0) {
        if (!ckpt) return UFP4_ERR_INVALID_ARG;
        UFP4_CHECK(check_matrix(dy, cols, ld_dy, size_of(dy_dtype), false));
        UFP4_CHECK(check_ckpt(ckpt, rows, cols, &a.ck));
        UFP4_CHECK(check_matrix(rstd, 1, 1, 4, false));
        UFP4_CHECK(check_matrix(gamma, cols, cols, size_of(gamma_dtype), false));
        UFP4_CHECK(check_matrix(dtotal, cols, ld_dtotal, 2, true));
        UFP4_CHECK(check_matrix(dx, cols, ld_dx, 2, false));
        UFP4_CHECK(check_matrix(y, cols, ldy, 2, true));
    }
    UFP4_CHECK(check_matrix(dgamma, cols, cols, 4, false));
    const int sms = current_num_sms();
    if (!workspace || workspace_bytes < (size_t)norm_parts(rows, cols, sms) * (size_t)cols * sizeof(float))
        return UFP4_ERR_INVALID_ARG;
    if ((uintptr_t)workspace % 256) return UFP4_ERR_ALIGNMENT;
    a.dy = dy;
    a.ld_dy = ld_dy;
    a.f32 = dy_dtype == UFP4_F32;
    a.rstd = const_cast<float*>(rstd);
    a.gamma = gamma;
    a.gamma_f32 = gamma_dtype == UFP4_F32;
    a.dtotal = dtotal;
    a.ld_dtotal = ld_dtotal;
    a.rows = rows;
    a.cols = cols;
    a.dx = dx;
    a.ld_dx = ld_dx;
    a.dgamma = dgamma;
    a.y = y;
    a.ldy = ldy;
    a.partials = (float*)workspace;
    return to_status(launch_rms_norm_backward(a, sms, stream));
}

// Whether the loss's extents and the tiles of its products (dH's up to 32 times, in shares) are 32-bit numbers.
static bool head_fits(int64_t tokens, int64_t vocab, int64_t hidden) {
    if (tokens > kMaxExtent || vocab > kMaxExtent || hidden > kMaxExtent) return false;
    const int64_t t = tokens / 256 + 1, v = vocab / 256 + 1, k = hidden / 256 + 1;
    return t * v + v * k + 32 * t * k < (1ll << 29);
}

static ufp4_status check_head(const void* h, int64_t ldh, const void* w, int64_t ldw, const int64_t* targets,
                              int64_t tokens, int64_t vocab, int64_t hidden, float z_loss) {
    if (tokens < 0 || vocab < 1 || hidden < 1 || !std::isfinite(z_loss)) return UFP4_ERR_INVALID_ARG;
    if (!head_fits(tokens, vocab, hidden)) return UFP4_ERR_UNSUPPORTED;
    if (!w || ldw < hidden || (tokens && (!h || !targets || ldh < hidden))) return UFP4_ERR_INVALID_ARG;
    if ((uintptr_t)w % 16 || ldw % 8) return UFP4_ERR_ALIGNMENT;
    if (tokens && ((uintptr_t)h % 16 || ldh % 8 || (uintptr_t)targets % 8)) return UFP4_ERR_ALIGNMENT;
    return UFP4_OK;
}

static ufp4_status check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (!workspace || bytes < need) return UFP4_ERR_INVALID_ARG;
    return (uintptr_t)workspace % 256 ? UFP4_ERR_ALIGNMENT : UFP4_OK;
}

static ufp4_status head_bytes(int64_t tokens, int64_t vocab, int64_t hidden,
                              size_t (*f)(int64_t, int64_t, int64_t, int), size_t* bytes) {
    if (tokens < 0 || vocab < 1 || hidden < 1 || !bytes) return UFP4_ERR_INVALID_ARG;
    if (!head_fits(tokens, vocab, hidden)) return UFP4_ERR_UNSUPPORTED;
    *bytes = f(tokens, vocab, hidden, current_num_sms());
    return UFP4_OK;
}

ufp4_status ufp4_head_loss_workspace_size(int64_t tokens, int64_t vocab, int64_t hidden, size_t* bytes) {
    return head_bytes(tokens, vocab, hidden, head_loss_bytes, bytes);
}

ufp4_status ufp4_head_loss_backward_workspace_size(int64_t tokens, int64_t vocab, int64_t hidden, size_t* bytes) {
    return head_bytes(tokens, vocab, hidden, head_loss_backward_bytes, bytes);
}

ufp4_status ufp4_head_loss(const void* h, int64_t ldh, const void* w, int64_t ldw, const int64_t* targets,
                           int64_t tokens, int64_t vocab, int64_t hidden, float z_loss, float* loss, float* lse,
                           void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    UFP4_CHECK(check_head(h, ldh, w, ldw, targets, tokens, vocab, hidden, z_loss));
    if (tokens == 0) return UFP4_OK;
    UFP4_CHECK(check_matrix(loss, 1, 1, 4, false));
    UFP4_CHECK(check_matrix(lse, 1, 1, 4, false));
    UFP4_CHECK(check_workspace(workspace, workspace_bytes, head_loss_bytes(tokens, vocab, hidden, current_num_sms())));
    HeadArgs a = {};
    a.h = h;
    a.ldh = ldh;
    a.w = w;
    a.ldw = ldw;
    a.targets = targets;
    a.T = tokens;
    a.V = vocab;
    a.K = hidden;
    a.z = z_loss;
    a.loss = loss;
    a.lse = lse;
    a.workspace = workspace;
    return to_status(launch_head_loss(a, current_num_sms(), stream));
}

ufp4_status ufp4_head_loss_backward(const void* h, int64_t ldh, const void* w, int64_t ldw, const int64_t* targets,
                                    int64_t tokens, int64_t vocab, int64_t hidden, float z_loss, const float* lse,
                                    const float* token_weight, const float* scale, void* dh, int64_t ld_dh,
                                    int32_t dh_dtype, void* dw, int64_t ld_dw, int32_t dw_dtype, int32_t accumulate_dw,
                                    void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    UFP4_CHECK(check_head(h, ldh, w, ldw, targets, tokens, vocab, hidden, z_loss));
    if (!is_dtype(dh_dtype) || !is_dtype(dw_dtype) || accumulate_dw < 0 || accumulate_dw > 1) return UFP4_ERR_INVALID_ARG;
    if (!dh && !dw) return UFP4_ERR_INVALID_ARG;
    if (accumulate_dw && dw_dtype != UFP4_F32) return UFP4_ERR_UNSUPPORTED;
    if (tokens) {
        UFP4_CHECK(check_matrix(lse, 1, 1, 4, false));
        UFP4_CHECK(check_matrix(token_weight, 1, 1, 4, true));
        UFP4_CHECK(check_matrix(dh, hidden, ld_dh, size_of(dh_dtype), true));
    }
    UFP4_CHECK(check_matrix(scale, 1, 1, 4, true));
    UFP4_CHECK(check_matrix(dw, hidden, ld_dw, size_of(dw_dtype), true));
    UFP4_CHECK(check_workspace(workspace, workspace_bytes, head_loss_backward_bytes(tokens, vocab, hidden, current_num_sms())));
    HeadArgs a = {};
    a.h = h;
    a.ldh = ldh;
    a.w = w;
    a.ldw = ldw;
    a.targets = targets;
    a.T = tokens;
    a.V = vocab;
    a.K = hidden;
    a.z = z_loss;
    a.lse = const_cast<float*>(lse);
    a.weight = token_weight;
    a.scale = scale;
    a.dh = tokens ? dh : nullptr;
    a.ld_dh = ld_dh;
    a.dh_f32 = dh_dtype == UFP4_F32;
    a.dw = dw;
    a.ld_dw = ld_dw;
    a.dw_f32 = dw_dtype == UFP4_F32;
    a.accumulate = accumulate_dw;
    a.workspace = workspace;
    return to_status(launch_head_loss_backward(a, current_num_sms(), stream));
}

}  // extern "C"
