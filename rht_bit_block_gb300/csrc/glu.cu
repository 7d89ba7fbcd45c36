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
// What is left is to keep the instructions below the memory time: elements are
// taken in pairs, the block's amax three at a time, and rows are found by
// multiplication.  Measured on a GB300: forward 8192 x 5632 from fp32 82.7 us,
// 6.73 TB/s, 4096 x 5632 from bf16 31 us; backward 16384 x 7168 from fp32 with y
// again 207 us, 6.83 TB/s (a plain copy there: 6.78), from bf16 141 us, 6.72
// TB/s (one element an instruction: 41 us forward, 169 us backward; two or four
// octets a thread: 220 and 275 us).  4109 x 1408 backward takes 10.3 us, 5 of
// them the launch.  Rows off 16-byte alignment, and widths that are no multiple
// of 8, are read and written element by element: 8192 x 5632 from bf16 58 us
// forward and 70 backward with y again, with gate or dy one element off 126 and
// 212, 8192 x 5631 184 and 311.
#include "ckpt8.cuh"
#include "internal.h"
#include "train.h"

namespace ufp4 {
namespace {

constexpr int kGluThreads = 256;

// exp2 and reciprocal to about an ulp; results below the normal range are 0.
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint64_t both(float x) { return pk2(x, x); }

// On pairs of elements, an instruction for two: act(g), and with GRAD its
// derivative.
template <int ACT, bool GRAD>
__device__ __forceinline__ uint64_t act2(uint64_t g, uint64_t& d) {
    const uint64_t g2 = mul2(g, g);
    // the logistic function of x: 1 / (1 + 2^(-x log2 e)); gelu's x is 2 sqrt(2/pi) (g + 0.044715 g^3)
    constexpr float kLog2e = 1.4426950408889634f, kC2 = 1.5957691216057308f;  // 2 sqrt(2/pi)
    const uint64_t x = ACT == 0 ? mul2(g, both(-kLog2e))
                                : mul2(g, fma2(g2, both(-kLog2e * kC2 * 0.044715f), both(-kLog2e * kC2)));
    float x0, x1;
    up2(x, x0, x1);
    const uint64_t q = add2(pk2(ex2(x0), ex2(x1)), both(1.0f));
    up2(q, x0, x1);
    const uint64_t s = pk2(rcp(x0), rcp(x1)), a = mul2(g, s);
    if (GRAD) {
        const uint64_t rest = fma2(s, both(-1.0f), both(1.0f));  // 1 - s
        if (ACT == 0) {
            d = mul2(s, fma2(g, rest, both(1.0f)));
        } else {
            // where s is 0 or 1 the second term is 0 (g^2 may have overflowed there)
            float w0, w1, t0, t1, s0, s1;
            up2(mul2(a, rest), w0, w1);
            up2(fma2(g2, both(3.0f * 0.044715f * kC2), both(kC2)), t0, t1);
            up2(s, s0, s1);
            d = pk2(w0 == 0.0f ? s0 : fmaf(w0, t0, s0), w1 == 0.0f ? s1 : fmaf(w1, t1, s1));
        }
    }
    return a;
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
    int64_t blocks;     // checkpoint blocks in all
    int64_t cols, nb;   // columns, blocks a row
    uint32_t magic;     // division by nb of block numbers below 2^31
    int shift;
};

// Row and first column of this thread's 8 elements, and how many of them
// exist.  SMALL: fewer than 2^31 blocks.
template <bool SMALL>
__device__ __forceinline__ void place(const GluParams& p, int64_t& row, int& c, int& n) {
    const int64_t t = (int64_t)blockIdx.x * kGluThreads + threadIdx.x;
    const int64_t b = t >> 2;
    if (SMALL)
        row = (uint32_t)(((uint64_t)(uint32_t)b * p.magic) >> p.shift);
    else
        row = b / p.nb;
    c = (int)(b - row * p.nb) * kCkptBlock + (int)(t & 3) * kVec;
    n = b < p.blocks ? (int)p.cols - c : 0;
}
// Element (row, c) of a matrix.  SMALL: rows and leading dimensions are below 2^31.
template <bool SMALL>
__device__ __forceinline__ int64_t at(int64_t row, int64_t ld, int c) {
    return SMALL ? (int64_t)(int)row * (int)ld + c : row * ld + c;
}

// VEC (aligned vectors) also means SMALL.
template <int ACT, bool F32, bool VEC, bool CKPT>
__global__ void __launch_bounds__(kGluThreads) glu_kernel(const GluParams p) {
    griddep_wait();
    griddep_launch();
    int64_t row;
    int c, n;
    place<VEC>(p, row, c, n);
    constexpr int es = F32 ? 4 : 2;
    float g[kVec], u[kVec];
    if (VEC && n <= 0) {
#pragma unroll
        for (int i = 0; i < kVec; ++i) g[i] = u[i] = 0.0f;
    } else {
        load8<F32, VEC>((const char*)p.in0 + at<VEC>(row, p.ld0, c) * es, n, g);
        load8<F32, VEC>((const char*)p.in1 + at<VEC>(row, p.ld1, c) * es, n, u);
    }
    if (CKPT) {
        ckpt_store8<VEC>(p.cg, row, c, n, g);
        ckpt_store8<VEC>(p.cu, row, c, n, u);
    }
    if (n <= 0) return;
    uint64_t d;
#pragma unroll
    for (int i = 0; i < kVec; i += 2)
        up2(mul2(act2<ACT, false>(pk2(g[i], g[i + 1]), d), pk2(u[i], u[i + 1])), u[i], u[i + 1]);
    store8_bf16<VEC>(p.y + at<VEC>(row, p.ldy, c), n, u);
}

template <int ACT, bool F32, bool VEC, bool REMAKE>
__global__ void __launch_bounds__(kGluThreads) glu_backward_kernel(const GluParams p) {
    griddep_wait();
    griddep_launch();
    int64_t row;
    int c, n;
    place<VEC>(p, row, c, n);
    if (n <= 0) return;
    float dy[kVec], g[kVec], u[kVec], y[kVec];
    load8<F32, VEC>((const char*)p.in0 + at<VEC>(row, p.ld0, c) * (F32 ? 4 : 2), n, dy);
    ckpt_load8<VEC>(p.cg, row, c, n, g);
    ckpt_load8<VEC>(p.cu, row, c, n, u);
#pragma unroll
    for (int i = 0; i < kVec; i += 2) {
        uint64_t d;
        const uint64_t a = act2<ACT, true>(pk2(g[i], g[i + 1]), d);
        const uint64_t up = pk2(u[i], u[i + 1]), t = pk2(dy[i], dy[i + 1]);
        if (REMAKE) up2(mul2(a, up), y[i], y[i + 1]);
        up2(mul2(mul2(t, up), d), g[i], g[i + 1]);
        up2(mul2(t, a), u[i], u[i + 1]);
    }
    store8_bf16<VEC>(p.dg + at<VEC>(row, p.ld_dg, c), n, g);
    store8_bf16<VEC>(p.du + at<VEC>(row, p.ld_du, c), n, u);
    if (REMAKE) store8_bf16<VEC>(p.y + at<VEC>(row, p.ldy, c), n, y);
}

// Vector accesses need every row's start aligned to them and whole vectors.
bool vec_ok(const void* p, int64_t ld, int64_t bytes_per_elem, int64_t align) {
    return (uintptr_t)p % align == 0 && (ld * bytes_per_elem) % align == 0 && ld < (1ll << 31);
}

// Fewer than 2^31 blocks, those of the last CTA that do not exist included.
bool small(const GluParams& p) { return p.blocks < (1ll << 31) - kGluThreads; }

GluParams make_params(const GluArgs& a) {
    GluParams p = {};
    p.cg = a.cg;
    p.cu = a.cu;
    p.y = (__nv_bfloat16*)a.y;
    p.ldy = a.ldy;
    p.cols = a.cols;
    p.nb = (a.cols + kCkptBlock - 1) / kCkptBlock;
    p.blocks = a.rows * p.nb;
    // b / nb = b * magic >> shift for b < 2^31: magic = floor(2^shift / nb) + 1, shift = 31 + ceil(log2 nb)
    // (Granlund and Montgomery, division by invariant integers)
    int log = 0;
    while ((1ll << log) < p.nb) ++log;
    p.shift = 31 + log;
    p.magic = (uint32_t)((1ull << p.shift) / (uint64_t)p.nb + 1);
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
    const bool vec = a.cols % kVec == 0 && small(p) && vec_ok(a.gate, a.ld_gate, es, 16) && vec_ok(a.up, a.ld_up, es, 16) &&
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
    const bool vec = a.cols % kVec == 0 && small(p) && vec_ok(a.dy, a.ld_dy, a.f32 ? 4 : 2, 16) &&
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
