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
// Memory bounds both passes, and a row has to be read whole before its first
// result, so what counts is how many rows are on their way while others are
// reduced, at few instructions an element.  A thread carries up to 32 elements
// of a row, its warp 1024 neighbouring ones (4 steps of 256, so that a step is
// an address offset known to the compiler): a row of 2048 takes two warps and
// an SM holds 8 to 16 rows.  Each thread copies its own elements of its group's
// next row into shared memory with cp.async while the current one, in
// registers, is summed and written, and waits for its own copies alone: no
// barrier but those of the row's sum.  Sums are fp32, by thread, warp and group
// in a fixed order.  Backward, a thread keeps dgamma of its columns in
// registers over its rows, a CTA adds its groups' sums, and a second kernel
// adds the CTAs' in their order, so results do not depend on timing.
//
// Measured on a GB300: forward 16384 x 7168 fp32 214 us, 6.05 TB/s (with both
// 16-byte halves of a lane's 8 fp32 fetched apart, so that every sector came
// twice: 248 us; without the copies ahead, one row a CTA: 278 us).  Backward
// 8192 x 2048 31 us with the 5 us of the dgamma kernel, 16384 x 7168 164 us,
// 5.0 TB/s: 512 threads an SM without a spill are its optimum (768 threads at
// 80 registers, spilling 44 bytes: 45 and 210 us; the decoded row kept beside
// dy gamma, spilling 140: 38 and 212 us; two rows ahead: 32 and 159 us).  That
// is for up to 8192 columns.  Wider rows take CTAs of more than 256 threads,
// built for up to 1024 with 64 registers a thread, of which the backward pass
// spills about 570 bytes: 4096 x 8192 59 us (4.0 TB/s), x 12288 186 us (1.9), x
// 16384 219 us (2.2), 2048 x 32768 216 us (2.2); forward 99 us (6.1) there.
//
// Rows off 16-byte alignment, and widths that are no multiple of 8, are read
// and written element by element, with nothing copied ahead: 8192 x 2048 from
// bf16 takes 25 us forward and 28 backward, with x or dy one element off 78 and
// 76, 8192 x 2047 105 and 80, 8192 x 2049 93 and 126 (fp32 dy: 107).
#include <algorithm>

#include "ckpt8.cuh"
#include "internal.h"
#include "norm_rows.cuh"
#include "train.h"
#include "ufp4_device.cuh"

namespace ufp4 {
namespace {

// Threads that an SM's registers should hold.
constexpr int kForwardThreads = 1024, kBackwardThreads = 512;

struct NormParams {
    const void* x;
    const __nv_bfloat16* add;  // residual, or dtotal
    const void* gamma;
    int64_t ldx, ld_add;
    int gamma_f32;
    int64_t rows;
    int cols;
    int group_warps, groups;  // warps a row, rows a CTA works on at once
    float inv_cols, eps;
    __nv_bfloat16* y;
    __nv_bfloat16* out;  // total, or dx
    int64_t ldy, ld_out;
    float* rstd;
    Ckpt ck;
    float* partials;
};

template <bool VEC>
__device__ __forceinline__ void load_gamma8(const NormParams& p, int c, int n, float v[kVec]) {
    if (!VEC) {
        if (p.gamma_f32)
            load8<true, false>((const float*)p.gamma + c, n, v);
        else
            load8<false, false>((const __nv_bfloat16*)p.gamma + c, n, v);
    } else if (p.gamma_f32) {
        const float4* q = (const float4*)((const float*)p.gamma + c);
        widen8(__ldg(q), __ldg(q + 1), v);
    } else {
        widen8(__ldg((const uint4*)((const __nv_bfloat16*)p.gamma + c)), v);
    }
}

// A warp's share of its group's next row: for each of ITER steps, the
// first input (512 bytes of bf16 or 1024 of fp32, copied 16 consecutive bytes a
// lane, so that every 32-byte sector is fetched once), 512 bytes of the second
// input and, backward, 256 of codes.
template <bool F32, int ITER, bool CODES>
struct Stage {
    static constexpr int kX = F32 ? 1024 : 512;
    static constexpr int kStep = kX + 512 + (CODES ? 256 : 0);  // bytes of a step
    static constexpr int kWarp = ITER * kStep;                  // and in all
    const uint8_t* warp;
    uint32_t saddr;  // of this lane's copies
    int lane;
    __device__ __forceinline__ explicit Stage(const uint8_t* smem) {
        lane = threadIdx.x & 31;
        warp = smem + (threadIdx.x >> 5) * kWarp;
        saddr = (uint32_t)__cvta_generic_to_shared(warp) + lane * 16;
    }
    // Starts the copies of this warp's elements of a row: of the first input and the codes ...
    __device__ __forceinline__ void fetch(const NormParams& p, int64_t row, int first) const {
        if (row >= p.rows) return;
        const int c0 = first - lane * kVec;  // the warp's first column
        const char* x = (const char*)p.x + row * p.ldx * (F32 ? 4 : 2) + c0 * (F32 ? 4 : 2) + lane * 16;
        const uint8_t* q = p.ck.codes + row * p.ck.codes_ld + first;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int left = p.cols - c0 - k * kStepCols;
            if (left <= 0) break;
            if (lane * (F32 ? 4 : 8) < left) copy16(saddr + k * kStep, x + k * kX);
            if (F32 && 128 + lane * 4 < left) copy16(saddr + k * kStep + 512, x + k * kX + 512);
            if (CODES && lane * kVec < left) copy8(saddr - lane * 8 + k * kStep + kX + 512, q + k * kStepCols);
        }
    }
    // ... and of the second input.
    __device__ __forceinline__ void fetch_add(const NormParams& p, int64_t row, int first) const {
        if (row >= p.rows || !p.add) return;
        const __nv_bfloat16* a = p.add + row * p.ld_add + first;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            if (first + k * kStepCols >= p.cols) break;
            copy16(saddr + k * kStep + kX, a + k * kStepCols);
        }
    }
    // Waits for the copies of all lanes.
    __device__ __forceinline__ void wait() const {
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
    }
    // The 8 elements of step k of this lane: of the first input as two or one 16-byte words, the second, the codes.
    __device__ __forceinline__ const uint8_t* x(int k) const { return warp + k * kStep + lane * (F32 ? 32 : 16); }
    __device__ __forceinline__ const uint8_t* add(int k) const { return warp + k * kStep + kX + lane * 16; }
    __device__ __forceinline__ const uint8_t* codes(int k) const { return warp + k * kStep + kX + 512 + lane * 8; }
    __device__ __forceinline__ void x8(int k, float v[kVec]) const {
        if (F32)
            widen8(*(const float4*)x(k), *(const float4*)(x(k) + 16), v);
        else
            widen8(*(const uint4*)x(k), v);
    }
    __device__ __forceinline__ void add8(int k, float v[kVec]) const { widen8(*(const uint4*)add(k), v); }
};

// THREADS: the most a CTA has.
template <bool F32, bool VEC, int ITER, int THREADS>
__global__ void __launch_bounds__(THREADS, kForwardThreads / THREADS) norm_kernel(const NormParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float slots[32];
    griddep_wait();
    griddep_launch();
    const Group<true> g(p.group_warps);
    const int first = g.template first<ITER>();
    const Stage<F32, ITER, false> st(smem);
    auto fetch = [&](int64_t row) {
        st.fetch(p, row, first);
        st.fetch_add(p, row, first);
    };
    if (VEC) fetch(blockIdx.x);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float s[ITER][kVec];
        float sum = 0.0f;
        if (VEC) st.wait();
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = first + k * kStepCols;
            const int n = p.cols - c;
#pragma unroll
            for (int i = 0; i < kVec; ++i) s[k][i] = 0.0f;
            if (n > 0) {
                float r[kVec];
                if (VEC)
                    st.x8(k, s[k]);
                else
                    load8<F32, false>((const char*)p.x + (row * p.ldx + c) * (F32 ? 4 : 2), n, s[k]);
                if (p.add) {
                    if (VEC)
                        st.add8(k, r);
                    else
                        load8<false, false>(p.add + row * p.ld_add + c, n, r);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) s[k][i] += r[i];
                }
            }
#pragma unroll
            for (int i = 0; i < kVec; ++i) sum = fmaf(s[k][i], s[k][i], sum);
        }
        if (VEC) {  // the warp's copies are in registers
            __syncwarp();
            fetch(row + gridDim.x);
        }
        const float r = rsqrtf(fmaf(g.sum(sum, slots), p.inv_cols, p.eps));
        if (p.rstd && g.warp == 0 && g.lane == 0) p.rstd[row] = r;
        __nv_bfloat16* y = p.y + row * p.ldy + first;
        __nv_bfloat16* out = p.out + row * p.ld_out + first;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = first + k * kStepCols;
            const int n = p.cols - c;
            if (p.ck.codes) ckpt_store8<VEC>(p.ck, row, c, n, s[k]);
            if (n <= 0) continue;
            if (p.out) store8_bf16<VEC>(out + k * kStepCols, n, s[k]);
            float w[kVec];
            load_gamma8<VEC>(p, c, n, w);
#pragma unroll
            for (int i = 0; i < kVec; ++i) w[i] = s[k][i] * r * w[i];
            store8_bf16<VEC>(y + k * kStepCols, n, w);
        }
    }
}

// The backward pass has about twice the arithmetic of the forward one per byte,
// so it works on pairs of fp32.
template <bool F32, bool VEC, int ITER, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > kBackwardThreads ? 1 : kBackwardThreads / THREADS)
norm_backward_kernel(const NormParams p) {
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float slots[32];
    griddep_wait();
    griddep_launch();
    const Group<false> g(p.group_warps);
    const int first = g.template first<ITER>();
    const int64_t stride = (int64_t)gridDim.x * p.groups;
    const Stage<F32, ITER, true> st(smem);
    // scale bytes of the steps' blocks and rstd, read one row ahead
    uint32_t byte[ITER];
    float rstd = 0.0f;
    auto scales = [&](int64_t row) {
        if (row >= p.rows) return;
        rstd = p.rstd[row];
        const uint8_t* b = p.ck.scales + row * p.ck.scales_ld + first / kCkptBlock;
#pragma unroll
        for (int k = 0; k < ITER; ++k)
            if (first + k * kStepCols < p.cols) byte[k] = b[k * kStepCols / kCkptBlock];
    };
    int64_t row = (int64_t)blockIdx.x * p.groups + g.index;
    if (VEC) {
        st.fetch(p, row, first);
        st.fetch_add(p, row, first);
        scales(row);
    }
    uint64_t dgamma[ITER][4];
#pragma unroll
    for (int k = 0; k < ITER; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) dgamma[k][i] = 0;
    for (; row < p.rows; row += stride) {
        if (!VEC) scales(row);
        const float r = rstd;
        uint64_t q[ITER][4];  // dy gamma
        uint2 codes[ITER];    // the normalised row, decoded again after its sum (decoded, it takes registers that spill)
        float unit[ITER];
        uint64_t dot = 0;
        __nv_bfloat16* y = p.y + row * p.ldy + first;
        // Step k of the normalised row.
        auto decode = [&](int k, int c, int n, uint64_t h[4]) {
            float v[kVec];
            if (VEC) {
                ckpt_unpack4(codes[k].x, v);
                ckpt_unpack4(codes[k].y, v + 4);
            } else {
                ckpt_load8<false>(p.ck, row, c, n, v);
            }
            pair8(v, h);
            const uint64_t u = VEC ? pk2(unit[k], unit[k]) : pk2(r, r);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = mul2(h[i], u);
        };
        if (VEC) st.wait();
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = first + k * kStepCols;
            const int n = p.cols - c;
            if (n <= 0) break;
            float v[kVec];
            if (VEC)
                st.x8(k, v);
            else
                load8<F32, false>((const char*)p.x + (row * p.ldx + c) * (F32 ? 4 : 2), n, v);
            pair8(v, q[k]);
            uint64_t w[4];
            load_gamma8<VEC>(p, c, n, v);
            pair8(v, w);
            if (VEC) {
                codes[k] = *(const uint2*)st.codes(k);
                unit[k] = r * ckpt_unit(byte[k]);  // a power of two: the product rounds once
            }
            uint64_t h[4];
            decode(k, c, n, h);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                dgamma[k][i] = fma2(q[k][i], h[i], dgamma[k][i]);
                q[k][i] = mul2(q[k][i], w[i]);
                dot = fma2(q[k][i], h[i], dot);
            }
            if (p.y) {
#pragma unroll
                for (int i = 0; i < 4; ++i) up2(mul2(w[i], h[i]), v[2 * i], v[2 * i + 1]);
                store8_bf16<VEC>(y + k * kStepCols, n, v);
            }
        }
        if (VEC) {  // the warp's first inputs and codes are in registers
            __syncwarp();
            st.fetch(p, row + stride, first);
            scales(row + stride);
        }
        float d0, d1;
        up2(dot, d0, d1);
        const float mean = g.sum(d0 + d1, slots) * p.inv_cols;
        const uint64_t minus = pk2(-mean, -mean), r2 = pk2(r, r);
        __nv_bfloat16* out = p.out + row * p.ld_out + first;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = first + k * kStepCols;
            const int n = p.cols - c;
            if (n <= 0) break;
            float t[kVec];
            uint64_t h[4], add[4] = {0, 0, 0, 0};
            decode(k, c, n, h);
            if (p.add) {
                if (VEC)
                    st.add8(k, t);
                else
                    load8<false, false>(p.add + row * p.ld_add + c, n, t);
                pair8(t, add);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                up2(fma2(r2, fma2(h[i], minus, q[k][i]), add[i]), t[2 * i], t[2 * i + 1]);
            store8_bf16<VEC>(out + k * kStepCols, n, t);
        }
        if (VEC) {
            __syncwarp();
            st.fetch_add(p, row + stride, first);
        }
    }
    // the groups' sums, added in their order by the last one; no copy is in flight, and their memory is free
    // once every group is here
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
    for (int j = 0; j < p.groups; ++j) {
        if (j) __syncthreads();
        if (g.index != j) continue;
        float* dst = j == p.groups - 1 ? p.partials + (int64_t)blockIdx.x * p.cols : sums;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = first + k * kStepCols;
            if (c >= p.cols) break;
            float v[kVec];
#pragma unroll
            for (int i = 0; i < 4; ++i) up2(dgamma[k][i], v[2 * i], v[2 * i + 1]);
            if (VEC) {
                float4* d = reinterpret_cast<float4*>(dst + c);
                const float4* s = reinterpret_cast<const float4*>(sums + c);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float4 t = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                    if (j) {
                        const float4 o = s[i];
                        t = make_float4(o.x + t.x, o.y + t.y, o.z + t.z, o.w + t.w);
                    }
                    d[i] = t;
                }
            } else {
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    if (c + i < p.cols) dst[c + i] = j ? sums[c + i] + v[i] : v[i];
            }
        }
    }
}

// dgamma[c] = sum over the parts, in their order: a CTA takes 8 columns (one
// 32-byte sector a part), 128 slices of parts, then the slices.
__global__ void __launch_bounds__(1024) norm_dgamma_kernel(const float* partials, int parts, int cols, float* dgamma) {
    __shared__ float slice[8][128 + 1];
    griddep_wait();
    griddep_launch();
    const int i = threadIdx.x & 7, j = threadIdx.x >> 3;
    const int c = blockIdx.x * 8 + i;
    float s = 0.0f;
    if (c < cols) {
#pragma unroll 4
        for (int q = j; q < parts; q += 128) s += partials[(int64_t)q * cols + c];
    }
    slice[i][j] = s;
    __syncthreads();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (w >= 8) return;
    s = (slice[w][lane] + slice[w][lane + 32]) + (slice[w][lane + 64] + slice[w][lane + 96]);
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (lane == 0 && blockIdx.x * 8 + w < cols) dgamma[blockIdx.x * 8 + w] = s;
}

Shape backward_shape(int64_t cols) {  // CTAs of about 256 threads, which leave fewer sums of dgamma
    Shape s = forward_shape(cols);
    s.groups = std::max(1, 8 / s.warps);
    return s;
}
// Dynamic shared memory of a CTA of so many warps.  Forward: its copies.
template <bool F32, bool VEC, int ITER>
constexpr int forward_smem(int warps) {
    return VEC ? warps * Stage<F32, ITER, false>::kWarp : 0;
}
// Backward: its copies; at least the sums of dgamma, which the groups but the
// last leave there (four bytes for each of `cols`).
template <bool F32, bool VEC, int ITER>
constexpr int backward_smem(int warps, int cols) {
    return VEC ? warps * Stage<F32, ITER, true>::kWarp : cols * 4;
}

template <bool F32, bool VEC, int ITER, int THREADS>
struct Fwd {
    static cudaError_t run(const NormParams& p, const Shape& s, int num_sms, cudaStream_t st) {
        const size_t smem = forward_smem<F32, VEC, ITER>(s.warps * s.groups);
        const int64_t grid = std::min<int64_t>(p.rows, (int64_t)num_sms * ctas_per_sm(s, kForwardThreads, smem));
        return launch_pdl(norm_kernel<F32, VEC, ITER, THREADS>, dim3((unsigned)grid), dim3(s.threads()), smem, st, p);
    }
};
template <bool F32, bool VEC, int ITER, int THREADS>
struct Bwd {
    static cudaError_t run(const NormParams& p, const Shape& s, int parts, cudaStream_t st) {
        const size_t smem = backward_smem<F32, VEC, ITER>(s.warps * s.groups, p.cols);
        return launch_pdl(norm_backward_kernel<F32, VEC, ITER, THREADS>, dim3((unsigned)parts), dim3(s.threads()), smem, st,
                          p);
    }
};
// Loads both kernels, and lets them have as much shared memory as the widest
// row they serve takes: the limit belongs to the kernel, which calls of other
// widths use at the same time, so no call may set it to its own need.
template <bool F32, bool VEC, int ITER, int THREADS>
struct Preload {
    static cudaError_t run() {
        constexpr int warps = THREADS / 32, cols = warps * ITER * kStepCols;
        constexpr int fwd = forward_smem<F32, VEC, ITER>(warps), bwd = backward_smem<F32, VEC, ITER>(warps, cols);
        static_assert(fwd <= 232448 - 128 && bwd <= 232448 - 128, "shared memory overflow");
        cudaFuncAttributes at;
        cudaFuncGetAttributes(&at, norm_kernel<F32, VEC, ITER, THREADS>);
        cudaFuncGetAttributes(&at, norm_backward_kernel<F32, VEC, ITER, THREADS>);
        const cudaError_t e =
            cudaFuncSetAttribute(norm_kernel<F32, VEC, ITER, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize, fwd);
        return e != cudaSuccess ? e
                                : cudaFuncSetAttribute(norm_backward_kernel<F32, VEC, ITER, THREADS>,
                                                       cudaFuncAttributeMaxDynamicSharedMemorySize, bwd);
    }
};

// L<f32, vec, steps, most threads>::run(args...) for a row's shape.
template <template <bool, bool, int, int> class L, bool F32, bool VEC, typename... A>
cudaError_t by_shape(const Shape& s, A&&... a) {
    if (s.iter == 1) return L<F32, VEC, 1, 256>::run(a...);
    if (s.iter == 2) return L<F32, VEC, 2, 256>::run(a...);
    return s.threads() > 256 ? L<F32, VEC, 4, 1024>::run(a...) : L<F32, VEC, 4, 256>::run(a...);
}
template <template <bool, bool, int, int> class L, typename... A>
cudaError_t dispatch(bool f32, bool vec, const Shape& s, A&&... a) {
    if (f32) return vec ? by_shape<L, true, true>(s, a...) : by_shape<L, true, false>(s, a...);
    return vec ? by_shape<L, false, true>(s, a...) : by_shape<L, false, false>(s, a...);
}

NormParams common(const NormArgs& a) {
    NormParams p = {};
    p.gamma = a.gamma;
    p.gamma_f32 = a.gamma_f32;
    p.rows = a.rows;
    p.cols = (int)a.cols;
    p.inv_cols = 1.0f / (float)a.cols;
    p.eps = a.eps;
    p.y = (__nv_bfloat16*)a.y;
    p.ldy = a.ldy;
    p.rstd = a.rstd;
    return p;
}

}  // namespace

int norm_parts(int64_t rows, int64_t cols, int num_sms) {
    const Shape s = backward_shape(cols);
    const size_t smem = (size_t)s.threads() * s.iter * 56;  // fp32 dy: bf16 needs less, and takes as many
    return (int)std::max<int64_t>(1, std::min<int64_t>((rows + s.groups - 1) / s.groups,
                                                       (int64_t)num_sms * ctas_per_sm(s, kBackwardThreads, smem)));
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
    const Shape s = forward_shape(a.cols);
    p.group_warps = s.warps;
    p.groups = s.groups;
    return dispatch<Fwd>(a.f32, vec, s, p, s, num_sms, st);
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
    const Shape s = backward_shape(a.cols);
    p.group_warps = s.warps;
    p.groups = s.groups;
    const int parts = norm_parts(a.rows, a.cols, num_sms);  // with no rows: one part of zeros
    cudaError_t e = dispatch<Bwd>(a.f32, vec, s, p, s, parts, st);
    if (e != cudaSuccess) return e;
    return launch_pdl(norm_dgamma_kernel, dim3((unsigned)((a.cols + 7) / 8)), dim3(1024), 0, st,
                      (const float*)a.partials, parts, (int)a.cols, a.dgamma);
}

cudaError_t preload_norm_kernels() {
    const Shape shapes[] = {{1, 1, 1}, {2, 1, 1}, {4, 1, 1}, {4, 32, 1}};
    for (const Shape& s : shapes)
        for (int i = 0; i < 4; ++i) dispatch<Preload>(i & 1, i & 2, s);
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, norm_dgamma_kernel);
}

}  // namespace ufp4
