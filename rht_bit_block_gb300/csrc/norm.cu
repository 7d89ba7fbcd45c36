// Residual add and RMS norm with an 8-bit checkpoint, before the projections
// of a block and before the vocabulary head (UFP4 summary, section 方法: the
// quantized GEMMs of FPROP, DGRAD and WGRAD take what this writes), and its
// backward pass from the checkpoint.
//
//   forward:   s = x + residual, r = (mean s^2 + eps)^-1/2, y = s r gamma,
//              total = bf16(s), checkpoint(s)
//   backward:  h = checkpoint(s) r, q = dy gamma, c = mean(q h),
//              dx = r (q - h c) + dtotal, dgamma = sum over rows of dy h,
//              and y = h gamma again, if asked
//
// Memory bounds both passes.  A CTA holds a whole row in registers (8
// elements a thread and step, ITER steps), so a row is read once although its
// norm needs all of it; the sums are fp32, by thread, warp and CTA in a fixed
// order.  Backward, a CTA walks rows with a stride and keeps dgamma of its
// columns in registers; the CTAs' sums are written apart and added in their
// order by a second kernel, so results do not depend on timing.
#include <algorithm>

#include "ckpt8.cuh"
#include "internal.h"
#include "train.h"

namespace ufp4 {
namespace {

struct NormParams {
    const void* x;
    const __nv_bfloat16* add;  // residual, or dtotal
    const void* gamma;
    int64_t ldx, ld_add;
    int gamma_f32;
    int64_t rows;
    int cols;
    float eps;
    __nv_bfloat16* y;
    __nv_bfloat16* out;  // total, or dx
    int64_t ldy, ld_out;
    float* rstd;
    Ckpt ck;
    float* partials;
};

// Sum over the CTA, the same value in every thread.  `slots`: 33 floats.
__device__ __forceinline__ float cta_sum(float v, float* slots) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    const int warps = blockDim.x >> 5;
    __syncthreads();  // the slots' last readers are done
    if ((threadIdx.x & 31) == 0) slots[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = (threadIdx.x & 31) < warps ? slots[threadIdx.x & 31] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    return s;
}

template <bool VEC>
__device__ __forceinline__ void load_gamma8(const NormParams& p, int c, int n, float v[kVec]) {
    if (p.gamma_f32)
        load8<true, VEC>((const float*)p.gamma + c, n, v);
    else
        load8<false, VEC>((const __nv_bfloat16*)p.gamma + c, n, v);
}

template <bool F32, bool VEC, int ITER>
__global__ void __launch_bounds__(1024) norm_kernel(const NormParams p) {
    __shared__ float slots[32];
    griddep_wait();
    griddep_launch();
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float s[ITER][kVec];
        float sum = 0.0f;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * kVec;
            const int n = p.cols - c;
#pragma unroll
            for (int i = 0; i < kVec; ++i) s[k][i] = 0.0f;
            if (n > 0) {
                load8<F32, VEC>((const char*)p.x + (row * p.ldx + c) * (F32 ? 4 : 2), n, s[k]);
                if (p.add) {
                    float r[kVec];
                    load8<false, VEC>(p.add + row * p.ld_add + c, n, r);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) s[k][i] += r[i];
                }
            }
        }
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * kVec;
            const int n = p.cols - c;
#pragma unroll
            for (int i = 0; i < kVec; ++i) sum = fmaf(s[k][i], s[k][i], sum);
            if (p.ck.codes) ckpt_store8<VEC>(p.ck, row, c, n, s[k]);
            if (p.out && n > 0) store8_bf16<VEC>(p.out + row * p.ld_out + c, n, s[k]);
        }
        const float r = 1.0f / sqrtf(cta_sum(sum, slots) / (float)p.cols + p.eps);
        if (threadIdx.x == 0 && p.rstd) p.rstd[row] = r;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * kVec;
            const int n = p.cols - c;
            if (n <= 0) continue;
            float g[kVec];
            load_gamma8<VEC>(p, c, n, g);
#pragma unroll
            for (int i = 0; i < kVec; ++i) g[i] = s[k][i] * r * g[i];
            store8_bf16<VEC>(p.y + row * p.ldy + c, n, g);
        }
    }
}

template <bool F32, bool VEC, int ITER>
__global__ void __launch_bounds__(1024) norm_backward_kernel(const NormParams p) {
    __shared__ float slots[32];
    griddep_wait();
    griddep_launch();
    float dgamma[ITER][kVec];
#pragma unroll
    for (int k = 0; k < ITER; ++k)
#pragma unroll
        for (int i = 0; i < kVec; ++i) dgamma[k][i] = 0.0f;
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float h[ITER][kVec], q[ITER][kVec];
        const float r = p.rstd[row];
        float dot = 0.0f;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * kVec;
            const int n = p.cols - c;
            if (n > 0) {
                load8<F32, VEC>((const char*)p.x + (row * p.ldx + c) * (F32 ? 4 : 2), n, q[k]);
                ckpt_load8<VEC>(p.ck, row, c, n, h[k]);
            } else {
#pragma unroll
                for (int i = 0; i < kVec; ++i) h[k][i] = q[k][i] = 0.0f;
            }
        }
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * kVec;
            const int n = p.cols - c;
            if (n <= 0) continue;
            float g[kVec], y[kVec];
            load_gamma8<VEC>(p, c, n, g);
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                h[k][i] *= r;
                dgamma[k][i] = fmaf(q[k][i], h[k][i], dgamma[k][i]);
                q[k][i] *= g[i];
                dot = fmaf(q[k][i], h[k][i], dot);
                y[i] = h[k][i] * g[i];
            }
            if (p.y) store8_bf16<VEC>(p.y + row * p.ldy + c, n, y);
        }
        const float mean = cta_sum(dot, slots) / (float)p.cols;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = (k * blockDim.x + threadIdx.x) * kVec;
            const int n = p.cols - c;
            if (n <= 0) continue;
            float t[kVec];
#pragma unroll
            for (int i = 0; i < kVec; ++i) t[i] = 0.0f;
            if (p.add) load8<false, VEC>(p.add + row * p.ld_add + c, n, t);
#pragma unroll
            for (int i = 0; i < kVec; ++i) t[i] = fmaf(r, fmaf(-h[k][i], mean, q[k][i]), t[i]);
            store8_bf16<VEC>(p.out + row * p.ld_out + c, n, t);
        }
    }
#pragma unroll
    for (int k = 0; k < ITER; ++k) {
        const int c = (k * blockDim.x + threadIdx.x) * kVec;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (c + i < p.cols) p.partials[(int64_t)blockIdx.x * p.cols + c + i] = dgamma[k][i];
    }
}

// dgamma[c] = sum over the parts, in their order: 8 slices of parts, then the slices.
__global__ void __launch_bounds__(256) norm_dgamma_kernel(const float* partials, int parts, int cols, float* dgamma) {
    __shared__ float slice[8][32];
    griddep_wait();
    griddep_launch();
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), j = threadIdx.x >> 5;
    float s = 0.0f;
    if (c < cols)
        for (int q = j; q < parts; q += 8) s += partials[(int64_t)q * cols + c];
    slice[j][threadIdx.x & 31] = s;
    __syncthreads();
    if (j == 0 && c < cols) {
#pragma unroll
        for (int k = 1; k < 8; ++k) s += slice[k][threadIdx.x];
        dgamma[c] = s;
    }
}

bool vec_ok(const void* p, int64_t ld, int64_t bytes_per_elem, int64_t align) {
    return (uintptr_t)p % align == 0 && (ld * bytes_per_elem) % align == 0;
}

// Threads of a CTA and steps a thread takes for a row.
struct Shape {
    int threads, iter;
};
Shape shape_of(int64_t cols) {
    const int64_t groups = (cols + kCkptBlock - 1) / kCkptBlock * 4;
    const int iter = groups <= 1024 ? 1 : (groups <= 2048 ? 2 : 4);
    const int64_t t = (groups + iter - 1) / iter;
    return {(int)((t + 31) / 32 * 32), iter};
}

template <template <bool, bool, int> class L, typename... A>
cudaError_t dispatch(bool f32, bool vec, int iter, A&&... a) {
#define UFP4_ITER(F, V)                                                        \
    return iter == 1 ? L<F, V, 1>::run(a...) : (iter == 2 ? L<F, V, 2>::run(a...) : L<F, V, 4>::run(a...))
    if (f32) {
        if (vec) UFP4_ITER(true, true);
        UFP4_ITER(true, false);
    }
    if (vec) UFP4_ITER(false, true);
    UFP4_ITER(false, false);
#undef UFP4_ITER
}
template <bool F32, bool VEC, int ITER>
struct Fwd {
    static cudaError_t run(const NormParams& p, unsigned grid, int threads, cudaStream_t st) {
        return launch_pdl(norm_kernel<F32, VEC, ITER>, dim3(grid), dim3(threads), 0, st, p);
    }
};
template <bool F32, bool VEC, int ITER>
struct Bwd {
    static cudaError_t run(const NormParams& p, unsigned grid, int threads, cudaStream_t st) {
        return launch_pdl(norm_backward_kernel<F32, VEC, ITER>, dim3(grid), dim3(threads), 0, st, p);
    }
};
template <bool F32, bool VEC, int ITER>
struct Preload {
    static cudaError_t run() {
        cudaFuncAttributes at;
        cudaFuncGetAttributes(&at, norm_kernel<F32, VEC, ITER>);
        return cudaFuncGetAttributes(&at, norm_backward_kernel<F32, VEC, ITER>);
    }
};

NormParams common(const NormArgs& a) {
    NormParams p = {};
    p.gamma = a.gamma;
    p.gamma_f32 = a.gamma_f32;
    p.rows = a.rows;
    p.cols = (int)a.cols;
    p.eps = a.eps;
    p.y = (__nv_bfloat16*)a.y;
    p.ldy = a.ldy;
    p.rstd = a.rstd;
    return p;
}

}  // namespace

int norm_parts(int64_t rows, int64_t cols, int num_sms) {
    // rows in flight per SM: what fits 1024 threads of backward registers
    const int per_sm = std::max(1, 1024 / shape_of(cols).threads);
    return (int)std::max<int64_t>(1, std::min<int64_t>(rows, (int64_t)num_sms * std::min(per_sm, 8)));
}

cudaError_t launch_rms_norm(const NormArgs& a, int num_sms, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    NormParams p = common(a);
    p.x = a.x;
    p.ldx = a.ldx;
    p.add = (const __nv_bfloat16*)a.residual;
    p.ld_add = a.ld_residual;
    p.out = (__nv_bfloat16*)a.total;
    p.ld_out = a.ld_total;
    if (a.ckpt) p.ck = a.ck;
    const bool vec = a.cols % kVec == 0 && vec_ok(a.x, a.ldx, a.f32 ? 4 : 2, 16) && vec_ok(a.gamma, 0, 1, 16) &&
                     vec_ok(a.y, a.ldy, 2, 16) && (!a.residual || vec_ok(a.residual, a.ld_residual, 2, 16)) &&
                     (!a.total || vec_ok(a.total, a.ld_total, 2, 16)) &&
                     (!a.ckpt || vec_ok(a.ck.codes, a.ck.codes_ld, 1, 8));
    const Shape s = shape_of(a.cols);
    const int64_t grid = std::min<int64_t>(a.rows, (int64_t)num_sms * 64);
    return dispatch<Fwd>(a.f32, vec, s.iter, p, (unsigned)grid, s.threads, st);
}

cudaError_t launch_rms_norm_backward(const NormArgs& a, int num_sms, cudaStream_t st) {
    NormParams p = common(a);
    p.x = a.dy;
    p.ldx = a.ld_dy;
    p.add = (const __nv_bfloat16*)a.dtotal;
    p.ld_add = a.ld_dtotal;
    p.out = (__nv_bfloat16*)a.dx;
    p.ld_out = a.ld_dx;
    p.ck = a.ck;
    p.partials = a.partials;
    const bool vec = a.cols % kVec == 0 && vec_ok(a.dy, a.ld_dy, a.f32 ? 4 : 2, 16) && vec_ok(a.gamma, 0, 1, 16) &&
                     vec_ok(a.dx, a.ld_dx, 2, 16) && (!a.dtotal || vec_ok(a.dtotal, a.ld_dtotal, 2, 16)) &&
                     (!a.y || vec_ok(a.y, a.ldy, 2, 16)) && vec_ok(a.ck.codes, a.ck.codes_ld, 1, 8);
    const Shape s = shape_of(a.cols);
    const int parts = norm_parts(a.rows, a.cols, num_sms);  // with no rows: one part of zeros
    cudaError_t e = dispatch<Bwd>(a.f32, vec, s.iter, p, (unsigned)parts, s.threads, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_dgamma_kernel, dim3((unsigned)((a.cols + 31) / 32)), dim3(256), 0, st,
                      (const float*)a.partials, parts, (int)a.cols, a.dgamma);
}

cudaError_t preload_norm_kernels() {
    for (int i = 0; i < 12; ++i) dispatch<Preload>(i & 1, i & 2, 1 << (i >> 2));
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, norm_dgamma_kernel);
}

}  // namespace ufp4
