// Gated activation with 8-bit checkpoints: y = act(gate) * up between the
// gate/up GEMM and the down GEMM of a feed-forward block (UFP4 summary,
// section 方法: FPROP, DGRAD and WGRAD of each linear layer are quantized
// GEMMs; this is what stands between two of them), and its backward pass from
// the checkpoints alone.
//
//   forward:   y = a(g) u                       checkpoint(g), checkpoint(u)
//   backward:  dg = dy u a'(g), du = dy a(g)    and y = a(g) u again, if asked
//   silu:      a(g) = g s(g), a' = s (1 + g (1 - s)), s the logistic function
//   gelu:      a(g) = g s(2 t), t = sqrt(2/pi) (g + 0.044715 g^3), which is the
//              tanh form g (1 + tanh t) / 2; a' = s + g s (1 - s) 2 t'
//
// Every element is read and written once, so memory bounds both passes:
// 8.06 bytes an element forward (bf16), 8.06 backward.  A thread carries 8
// elements, four threads a checkpoint block, so a block's scale takes two
// shuffles and nothing goes through shared memory; no element waits for
// another, so one short-lived thread an octet is enough to keep memory busy.
// Measured on a GB300: forward 8192 x 5632 from fp32 83.9 us, 6.64 TB/s;
// backward 16384 x 7168 from fp32 with y again 209.7 us, 6.75 TB/s (a plain
// copy there: 6.78).  4109 x 1408 backward takes 12 us, 5 of them the launch.
#include "ckpt8.cuh"
#include "internal.h"
#include "train.h"

namespace ufp4 {
namespace {

constexpr int kGluThreads = 256;

__device__ __forceinline__ float logistic(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// act(g) and, with GRAD, its derivative
template <int ACT, bool GRAD>
__device__ __forceinline__ float act(float g, float& d) {
    if (ACT == 0) {
        const float s = logistic(g);
        if (GRAD) d = s * fmaf(g, 1.0f - s, 1.0f);
        return g * s;
    }
    constexpr float c = 0.7978845608028654f;  // sqrt(2 / pi)
    const float g2 = g * g;
    const float s = logistic(2.0f * c * g * fmaf(0.044715f, g2, 1.0f));
    if (GRAD) {
        // where s is 0 or 1 the second term is 0 (g^2 may have overflowed there)
        const float w = g * s * (1.0f - s);
        d = w == 0.0f ? s : fmaf(2.0f * c * w, fmaf(0.134145f, g2, 1.0f), s);
    }
    return g * s;
}

struct GluParams {
    const void* in0;  // gate, or dy
    const void* in1;  // up
    int64_t ld0, ld1;
    Ckpt cg, cu;
    __nv_bfloat16* y;
    __nv_bfloat16* dg;
    __nv_bfloat16* du;
    int64_t ldy, ld_dg, ld_du;
    int64_t blocks;   // checkpoint blocks in all
    int64_t cols, nb; // columns, blocks a row
};

// Row and first column of this thread's 8 elements, and how many of them exist.
__device__ __forceinline__ void place(const GluParams& p, int64_t& row, int& c, int& n) {
    const int64_t t = (int64_t)blockIdx.x * kGluThreads + threadIdx.x;
    const int64_t b = t >> 2;
    if (p.blocks <= 0xFFFFFFFFll) {
        row = (uint32_t)b / (uint32_t)p.nb;
    } else {
        row = b / p.nb;
    }
    c = (int)(b - row * p.nb) * kCkptBlock + (int)(t & 3) * kVec;
    n = b < p.blocks ? (int)p.cols - c : 0;
}

template <int ACT, bool F32, bool VEC, bool CKPT>
__global__ void __launch_bounds__(kGluThreads) glu_kernel(const GluParams p) {
    griddep_wait();
    griddep_launch();
    int64_t row;
    int c, n;
    place(p, row, c, n);
    constexpr int es = F32 ? 4 : 2;
    float g[kVec], u[kVec];
    if (VEC && n <= 0) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) g[i] = u[i] = 0.0f;
    } else {
        load8<F32, VEC>((const char*)p.in0 + (row * p.ld0 + c) * es, n, g);
        load8<F32, VEC>((const char*)p.in1 + (row * p.ld1 + c) * es, n, u);
    }
    if (CKPT) {
        ckpt_store8<VEC>(p.cg, row, c, n, g);
        ckpt_store8<VEC>(p.cu, row, c, n, u);
    }
    if (n <= 0) return;
    float d;
#pragma unroll
    for (int i = 0; i < kVec; ++i) u[i] *= act<ACT, false>(g[i], d);
    store8_bf16<VEC>(p.y + row * p.ldy + c, n, u);
}

template <int ACT, bool F32, bool VEC, bool REMAKE>
__global__ void __launch_bounds__(kGluThreads) glu_backward_kernel(const GluParams p) {
    griddep_wait();
    griddep_launch();
    int64_t row;
    int c, n;
    place(p, row, c, n);
    if (n <= 0) return;
    float dy[kVec], g[kVec], u[kVec], y[kVec];
    load8<F32, VEC>((const char*)p.in0 + (row * p.ld0 + c) * (F32 ? 4 : 2), n, dy);
    ckpt_load8<VEC>(p.cg, row, c, n, g);
    ckpt_load8<VEC>(p.cu, row, c, n, u);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
        float d;
        const float a = act<ACT, true>(g[i], d);
        if (REMAKE) y[i] = a * u[i];
        g[i] = dy[i] * u[i] * d;
        u[i] = dy[i] * a;
    }
    store8_bf16<VEC>(p.dg + row * p.ld_dg + c, n, g);
    store8_bf16<VEC>(p.du + row * p.ld_du + c, n, u);
    if (REMAKE) store8_bf16<VEC>(p.y + row * p.ldy + c, n, y);
}

// Vector accesses need every row's start aligned to them and whole vectors.
bool vec_ok(const void* p, int64_t ld, int64_t bytes_per_elem, int64_t align) {
    return (uintptr_t)p % align == 0 && (ld * bytes_per_elem) % align == 0;
}

GluParams make_params(const GluArgs& a) {
    GluParams p = {};
    p.cg = a.cg;
    p.cu = a.cu;
    p.y = (__nv_bfloat16*)a.y;
    p.ldy = a.ldy;
    p.cols = a.cols;
    p.nb = (a.cols + kCkptBlock - 1) / kCkptBlock;
    p.blocks = a.rows * p.nb;
    return p;
}

template <typename K>
cudaError_t run(K kernel, const GluParams& p, cudaStream_t st) {
    const int64_t grid = (p.blocks * 4 + kGluThreads - 1) / kGluThreads;
    if (grid > 0x7FFFFFFF) return cudaErrorNotSupported;
    return launch_pdl(kernel, dim3((unsigned)grid), dim3(kGluThreads), 0, st, p);
}

template <int ACT, bool F32, bool VEC>
cudaError_t fwd3(const GluArgs& a, const GluParams& p, cudaStream_t st) {
    return a.ckpt ? run(glu_kernel<ACT, F32, VEC, true>, p, st) : run(glu_kernel<ACT, F32, VEC, false>, p, st);
}
template <int ACT, bool F32, bool VEC>
cudaError_t bwd3(const GluArgs& a, const GluParams& p, cudaStream_t st) {
    return a.y ? run(glu_backward_kernel<ACT, F32, VEC, true>, p, st)
               : run(glu_backward_kernel<ACT, F32, VEC, false>, p, st);
}
template <int ACT>
cudaError_t fwd1(const GluArgs& a, const GluParams& p, bool vec, cudaStream_t st) {
    if (a.f32) return vec ? fwd3<ACT, true, true>(a, p, st) : fwd3<ACT, true, false>(a, p, st);
    return vec ? fwd3<ACT, false, true>(a, p, st) : fwd3<ACT, false, false>(a, p, st);
}
template <int ACT>
cudaError_t bwd1(const GluArgs& a, const GluParams& p, bool vec, cudaStream_t st) {
    if (a.f32) return vec ? bwd3<ACT, true, true>(a, p, st) : bwd3<ACT, true, false>(a, p, st);
    return vec ? bwd3<ACT, false, true>(a, p, st) : bwd3<ACT, false, false>(a, p, st);
}

template <int ACT, bool F32, bool VEC>
cudaError_t preload3() {
    cudaFuncAttributes at;
    cudaFuncGetAttributes(&at, glu_kernel<ACT, F32, VEC, true>);
    cudaFuncGetAttributes(&at, glu_kernel<ACT, F32, VEC, false>);
    cudaFuncGetAttributes(&at, glu_backward_kernel<ACT, F32, VEC, true>);
    return cudaFuncGetAttributes(&at, glu_backward_kernel<ACT, F32, VEC, false>);
}

}  // namespace

cudaError_t launch_glu(const GluArgs& a, cudaStream_t st) {
    GluParams p = make_params(a);
    p.in0 = a.gate;
    p.in1 = a.up;
    p.ld0 = a.ld_gate;
    p.ld1 = a.ld_up;
    const int es = a.f32 ? 4 : 2;
    const bool vec = a.cols % kVec == 0 && vec_ok(a.gate, a.ld_gate, es, 16) && vec_ok(a.up, a.ld_up, es, 16) &&
                     vec_ok(a.y, a.ldy, 2, 16) &&
                     (!a.ckpt || (vec_ok(a.cg.codes, a.cg.codes_ld, 1, 8) && vec_ok(a.cu.codes, a.cu.codes_ld, 1, 8)));
    return a.act == 0 ? fwd1<0>(a, p, vec, st) : fwd1<1>(a, p, vec, st);
}

cudaError_t launch_glu_backward(const GluArgs& a, cudaStream_t st) {
    GluParams p = make_params(a);
    p.in0 = a.dy;
    p.ld0 = a.ld_dy;
    p.dg = (__nv_bfloat16*)a.dgate;
    p.du = (__nv_bfloat16*)a.dup;
    p.ld_dg = a.ld_dgate;
    p.ld_du = a.ld_dup;
    const bool vec = a.cols % kVec == 0 && vec_ok(a.dy, a.ld_dy, a.f32 ? 4 : 2, 16) &&
                     vec_ok(a.dgate, a.ld_dgate, 2, 16) && vec_ok(a.dup, a.ld_dup, 2, 16) &&
                     (!a.y || vec_ok(a.y, a.ldy, 2, 16)) && vec_ok(a.cg.codes, a.cg.codes_ld, 1, 8) &&
                     vec_ok(a.cu.codes, a.cu.codes_ld, 1, 8);
    return a.act == 0 ? bwd1<0>(a, p, vec, st) : bwd1<1>(a, p, vec, st);
}

cudaError_t preload_glu_kernels() {
    preload3<0, true, true>();
    preload3<0, true, false>();
    preload3<0, false, true>();
    preload3<0, false, false>();
    preload3<1, true, true>();
    preload3<1, true, false>();
    preload3<1, false, true>();
    return preload3<1, false, false>();
}

}  // namespace ufp4
