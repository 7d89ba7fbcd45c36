// Residual add and layer norm, before the projections of a block (UFP4
// summary, section 方法: the quantized GEMMs of FPROP, DGRAD and WGRAD take what
// this writes), and its gradients.
//
//   forward:   s = x + residual, m = mean s, r = (mean (s - m)^2 + eps)^-1/2,
//              y = (s - m) r gamma + beta, total = bf16(s)
//   backward:  h = (s - m) r, q = dy gamma,
//              dx = r (q - mean q - h mean(q h)) + dtotal,
//              dgamma = sum over rows of dy h, dbeta = sum over rows of dy
//
// The variance is the mean of squared differences from the mean, in a second
// pass over the row, which is in registers: the mean square minus the squared
// mean loses all digits of a row that lies far from zero.  The mean of the first
// pass is off by roundings of the size of the row's elements (of 7168 elements of
// 1e5 by 0.008, 1 / 7168 being no fp32 number), which may be many deviations.  The
// second pass therefore sums the differences too: their mean is what the first
// one lacks, to roundings of the size of a difference, and its square is what the
// squares have too much.  Two columns an instruction there: beside what it adds that
// saves the registers of rows above 16384 columns (2048 x 32768: 95 us; 126 by single
// columns), and elsewhere the second sum costs 2 % at most.
//
// Memory bounds both passes.  As in the RMS norm (norm.cu) a warp takes 256
// neighbouring columns a step and each lane copies its elements of the group's
// next row into shared memory while the current one is worked on.  The backward
// pass keeps two rows there: it reads a row twice, once for its sums and once for
// dx, so that registers hold nothing of it but the running dgamma and dbeta of the
// lane's columns.  A CTA adds its groups' sums, and a second kernel the CTAs', in
// their order: results do not depend on timing.
//
// Measured: forward 16384 x 7168 fp32 193 us (6.1 TB/s, DRAM 77 % active), bf16 146,
// 8192 x 2048 bf16 25, 2048 x 32768 bf16 95.  Backward 16384 x 7168 bf16 155 us (6.1
// TB/s with dtotal; 122 registers, 16 warps an SM: issue 50 %, DRAM 55 %), 8192 x 2048
// 27.6 us, of which start, ramp and the joining kernel are about 8; 2048 x 32768, whose
// rows no CTA can keep the sums of, 284 us for two passes over dy and x.
#include <algorithm>

#include "ckpt8.cuh"
#include "internal.h"
#include "norm_rows.cuh"
#include "train.h"
#include "ufp4_device.cuh"

namespace ufp4 {
namespace {

constexpr int kForwardThreads = 1024;   // threads that an SM's registers should hold
constexpr int kBackwardThreads = 512;
constexpr size_t kMostSmem = 232448 - 1024;

struct LnParams {
    const void* x;             // forward: x; backward: the normalised rows
    const void* dy;
    const __nv_bfloat16* add;  // residual, or dtotal
    const void* gamma;
    const void* beta;
    int64_t ldx, ld_dy, ld_add;
    int x_f32, dy_f32, gamma_f32;  // x and dy: where they are read without copies
    int vec;                       // the same: all rows are aligned to their vectors
    int vec_weights;               // gamma and beta are
    int64_t rows;
    int cols;
    int group_warps, groups;       // warps a row, rows a CTA works on at once
    float inv_cols, eps;
    __nv_bfloat16* y;
    __nv_bfloat16* out;            // total, or dx
    int64_t ldy, ld_out;
    float* mean;
    float* rstd;
    float* partials;               // backward, [part][2][partials_pitch(cols)]
};
__host__ __device__ constexpr int partials_pitch(int cols) { return (cols + kVec - 1) / kVec * kVec; }

__device__ __forceinline__ void load8_any(const void* p, int64_t at, int f32, int vec, int n, float v[kVec]) {
    const char* src = (const char*)p + at * (f32 ? 4 : 2);
    if (vec) {
        if (f32) load8<true, true>(src, n, v);
        else load8<false, true>(src, n, v);
    } else {
        if (f32) load8<true, false>(src, n, v);
        else load8<false, false>(src, n, v);
    }
}
// gamma or beta of eight columns; they stay in L1.
__device__ __forceinline__ void load_weight8(const void* p, int f32, int vec, int c, int n, float v[kVec]) {
    if (!vec) {
        load8_any(p, c, f32, 0, n, v);
    } else if (f32) {
        const float4* q = (const float4*)((const float*)p + c);
        widen8(__ldg(q), __ldg(q + 1), v);
    } else {
        widen8(__ldg((const uint4*)((const __nv_bfloat16*)p + c)), v);
    }
}
// Whether they are aligned to vectors and the row has all eight.
template <bool SHIFTED>
__device__ __forceinline__ int weight_vec(const LnParams& p, int n) {
    return SHIFTED ? p.vec_weights && n >= kVec : 1;
}
__device__ __forceinline__ void store8_any(__nv_bfloat16* p, int vec, int n, const float v[kVec]) {
    if (vec) store8_bf16<true>(p, n, v);
    else store8_bf16<false>(p, n, v);
}

// A warp's share of a row in shared memory: one matrix, ITER steps of 256
// columns.  Copied 16 consecutive bytes a lane, so that every 32-byte sector is
// fetched once; read as a lane's 8 elements.  SHIFTED: rows may start anywhere.
// The 16-byte units of memory that hold the share are copied as they are, and a
// lane's elements taken out of two or three of them; what lies beside the share
// in its first unit, which belongs to the matrix too or is left out, is not
// looked at.  (8192 x 4999 bf16: forward 116 us, backward 154; 222 and 311 with the
// elements loaded and stored one by one, 59 and 79 of 5000 columns.)
template <bool F32, int ITER, bool SHIFTED>
struct Copy {
    static constexpr int kElem = F32 ? 4 : 2;
    static constexpr int kStepBytes = kStepCols * kElem;
    static constexpr int kBytes = ITER * kStepBytes + (SHIFTED ? 16 : 0);
    // Bytes of the first unit in front of a row's share: shares start at multiples of 16 bytes of the row.
    static __device__ __forceinline__ int shift(const void* base, int64_t ld, int64_t row) {
        return SHIFTED ? (int)((uint32_t)(uintptr_t)base + (uint32_t)row * (uint32_t)ld * kElem) & 15 : 0;
    }
    static __device__ __forceinline__ void fetch(uint32_t dst, const void* base, int64_t ld, int64_t row, int c0, int cols) {
        const int lane = threadIdx.x & 31;
        const char* src = (const char*)base + (row * ld + c0) * kElem + lane * 16;
        if constexpr (SHIFTED) {
            if (cols <= c0) return;
            const int before = shift(base, ld, row), bytes = before + min(cols - c0, ITER * kStepCols) * kElem;
            src -= before;
#pragma unroll
            for (int k = 0; k <= ITER * kStepBytes / 512; ++k) {
                const int left = bytes - k * 512 - lane * 16;
                if (left <= 0) break;
                if (src + k * 512 < (const char*)base) {  // the matrix starts within this unit
                    for (int i = before; i < min(left, 16); i += kElem) {
                        if (F32) asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + i), "r"(*(const uint32_t*)(src + i)) : "memory");
                        else asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst + i), "h"(*(const uint16_t*)(src + i)) : "memory");
                    }
                } else {
                    copy16_part(dst + k * 512 + lane * 16, src + k * 512, min(left, 16));
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < ITER; ++k) {
                const int left = cols - c0 - k * kStepCols;
                if (left <= 0) break;
                if (lane * (F32 ? 4 : 8) < left) copy16(dst + k * kStepBytes + lane * 16, src + k * kStepBytes);
                if (F32 && 128 + lane * 4 < left) copy16(dst + k * kStepBytes + 512 + lane * 16, src + k * kStepBytes + 512);
            }
        }
    }
    // Step k's elements of the lane, of which n (SHIFTED: or none) exist; `rest` after.
    static __device__ __forceinline__ void read(const uint8_t* src, int k, int shift, int n, float v[kVec], float rest = 0.0f) {
        const uint8_t* p = src + k * kStepBytes + (threadIdx.x & 31) * (kVec * kElem);
        if (!SHIFTED) {
            if (F32) widen8(*(const float4*)p, *(const float4*)(p + 16), v);
            else widen8(*(const uint4*)p, v);
            return;
        }
        constexpr int kWords = kVec * kElem / 4;
        uint32_t w[kWords + 4];
#pragma unroll
        for (int i = 0; i < kWords + 4; i += 4) {
            const uint4 u = *(const uint4*)(p + i * 4);
            w[i] = u.x;
            w[i + 1] = u.y;
            w[i + 2] = u.z;
            w[i + 3] = u.w;
        }
#pragma unroll
        for (int i = 0; i < kWords + 3; ++i) w[i] = shift & 4 ? w[i + 1] : w[i];
#pragma unroll
        for (int i = 0; i < kWords + 1; ++i) w[i] = shift & 8 ? w[i + 2] : w[i];
        if (F32) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) v[i] = __uint_as_float(w[i]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], (shift & 2) * 8);
            widen8(make_uint4(w[0], w[1], w[2], w[3]), v);
        }
        if (n < kVec) {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (i >= n) v[i] = rest;
        }
    }
};

// Stores a warp's share of a bf16 row that may start anywhere, step by step: the 16-byte units of memory are put together from
// neighbouring lanes' elements and stored whole, those at either end of the share by elements.  All lanes call it.
struct ShiftedRow {
    char* first;        // of the lane: its unit of step 0
    int shift, bytes;   // in front of the share, in its first unit; of the share
    uint32_t last[4];   // lane 0: what the step before left of its last lane
    __device__ __forceinline__ ShiftedRow(__nv_bfloat16* share, int cols) {
        shift = (int)(uintptr_t)share & 15;
        bytes = cols * 2;
        first = (char*)share - shift + (threadIdx.x & 31) * 16;
    }
    __device__ __forceinline__ void units(int k, const uint32_t before[4], const uint32_t w[4]) const {
        const int at = k * 512 + (int)(threadIdx.x & 31) * 16 - shift;  // of the unit, in the share
        if (at >= bytes) return;
        uint32_t t[8] = {before[0], before[1], before[2], before[3], w[0], w[1], w[2], w[3]};
        const int from = 16 - shift;  // where the unit starts in the two lanes' bytes
        // from a multiple of 4: words from / 4; otherwise half a word further on
#pragma unroll
        for (int i = 0; i < 7; ++i) t[i] = from & 4 ? t[i + 1] : t[i];
#pragma unroll
        for (int i = 0; i < 6; ++i) t[i] = from & 8 ? t[i + 2] : t[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = from & 16 ? t[i + 4] : t[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) t[i] = __funnelshift_r(t[i], t[i + 1], (from & 2) * 8);
        char* d = first + k * 512;
        if (at >= 0 && at + 16 <= bytes) {
            __stcs(reinterpret_cast<uint4*>(d), make_uint4(t[0], t[1], t[2], t[3]));
            return;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (at + 2 * i >= 0 && at + 2 * i < bytes) *reinterpret_cast<uint16_t*>(d + 2 * i) = (uint16_t)(t[i / 2] >> (16 * (i & 1)));
    }
    __device__ __forceinline__ void step(int k, const float v[kVec]) {
        const int lane = threadIdx.x & 31;
        uint32_t w[4], before[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
            const uint32_t o = __shfl_sync(0xFFFFFFFFu, w[i], (lane + 31) & 31);
            before[i] = lane ? o : last[i];
            last[i] = o;
        }
        units(k, before, w);
    }
    // What is left after `steps` steps.
    __device__ __forceinline__ void finish(int steps) const {
        const uint32_t none[4] = {0, 0, 0, 0};
        if ((threadIdx.x & 31) == 0) units(steps, last, none);
    }
};

// SHIFTED: some row is not aligned to 16 bytes or no whole number of lanes'
// elements.  THREADS: the most a CTA has.
template <bool F32, bool SHIFTED, int ITER, int THREADS>
__global__ void __launch_bounds__(THREADS, kForwardThreads / THREADS) layer_norm_kernel(const LnParams p) {
    using X = Copy<F32, ITER, SHIFTED>;
    using A = Copy<false, ITER, SHIFTED>;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(8) float slots[64];
    griddep_wait();
    griddep_launch();
    const Group<true> g(p.group_warps);
    const int first = g.template first<ITER>();
    const int c0 = first - g.lane * kVec;  // the warp's first column
    const uint8_t* mine = smem + (threadIdx.x >> 5) * (X::kBytes + A::kBytes);
    const uint32_t saddr = (uint32_t)__cvta_generic_to_shared(mine);
    auto fetch = [&](int64_t row) {
        if (row >= p.rows) return;
        X::fetch(saddr, p.x, p.ldx, row, c0, p.cols);
        if (p.add) A::fetch(saddr + X::kBytes, p.add, p.ld_add, row, c0, p.cols);
    };
    fetch(blockIdx.x);
    for (int64_t row = blockIdx.x; row < p.rows; row += gridDim.x) {
        float s[ITER][kVec];
        float sum = 0.0f;
        const int of_x = X::shift(p.x, p.ldx, row), of_add = A::shift(p.add, p.ld_add, row);
        asm volatile("cp.async.wait_all;" ::: "memory");
        __syncwarp();
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int n = p.cols - (first + k * kStepCols);
#pragma unroll
            for (int i = 0; i < kVec; ++i) s[k][i] = 0.0f;
            if (n > 0) {
                X::read(mine, k, of_x, n, s[k]);
                if (p.add) {
                    float r[kVec];
                    A::read(mine + X::kBytes, k, of_add, n, r);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) s[k][i] += r[i];
                }
            }
#pragma unroll
            for (int i = 0; i < kVec; ++i) sum += s[k][i];
        }
        __syncwarp();  // the warp's copies are in registers
        fetch(row + gridDim.x);
        const float mean = g.sum(sum, slots) * p.inv_cols;
        uint64_t d2 = 0, q2 = 0;  // differences from the first mean and their squares, two columns each
        const uint64_t minus = pk2(-mean, -mean);
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int n = p.cols - (first + k * kStepCols);
            if (n < kVec) {  // what is missing lies at the mean
#pragma unroll
                for (int i = 0; i < kVec; ++i)
                    if (i >= n) s[k][i] = mean;
            }
#pragma unroll
            for (int i = 0; i < kVec; i += 2) {
                const uint64_t t = add2(pk2(s[k][i], s[k][i + 1]), minus);
                d2 = add2(t, d2);
                q2 = fma2(t, t, q2);
            }
        }
        float2 d, q;
        up2(d2, d.x, q.x);
        up2(q2, d.y, q.y);
        d = g.sum2(make_float2(d.x + q.x, d.y + q.y), slots);
        const float rest = d.x * p.inv_cols;  // of the mean
        const float v = fmaf(-rest, rest, d.y * p.inv_cols);
        const float r = rsqrtf((v < 0.0f ? 0.0f : v) + p.eps);  // a NaN stays
        const float less = -rest * r;  // (s - mean - rest) r = (s - mean) r + less
        if (g.warp == 0 && g.lane == 0) {
            if (p.mean) p.mean[row] = mean + rest;
            if (p.rstd) p.rstd[row] = r;
        }
        auto result = [&](int k, int n, float w[kVec]) {
            const int c = first + k * kStepCols;
            float b[kVec];
            load_weight8(p.gamma, p.gamma_f32, weight_vec<SHIFTED>(p, n), c, n, w);
            if (p.beta) {
                load_weight8(p.beta, p.gamma_f32, weight_vec<SHIFTED>(p, n), c, n, b);
#pragma unroll
                for (int i = 0; i < kVec; ++i) w[i] = fmaf(fmaf(s[k][i] - mean, r, less), w[i], b[i]);
            } else {
#pragma unroll
                for (int i = 0; i < kVec; ++i) w[i] = fmaf(s[k][i] - mean, r, less) * w[i];
            }
        };
        if (SHIFTED) {
            const int share = min(p.cols - c0, ITER * kStepCols);
            if (share <= 0) continue;
            const int steps = (share + kStepCols - 1) / kStepCols;
            if (p.out) {
                ShiftedRow to(p.out + row * p.ld_out + c0, share);
#pragma unroll
                for (int k = 0; k < ITER; ++k)
                    if (k < steps) to.step(k, s[k]);
                to.finish(steps);
            }
            ShiftedRow to(p.y + row * p.ldy + c0, share);
#pragma unroll
            for (int k = 0; k < ITER; ++k) {
                if (k >= steps) break;
                float w[kVec];
                result(k, p.cols - (first + k * kStepCols), w);
                to.step(k, w);
            }
            to.finish(steps);
            continue;
        }
        __nv_bfloat16* y = p.y + row * p.ldy + first;
        __nv_bfloat16* out = p.out + row * p.ld_out + first;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int n = p.cols - (first + k * kStepCols);
            if (n <= 0) break;
            if (p.out) store8_bf16<true>(out + k * kStepCols, n, s[k]);
            float w[kVec];
            result(k, n, w);
            store8_bf16<true>(y + k * kStepCols, n, w);
        }
    }
}

// How the backward pass gets at its rows.
enum Rows {
    kInPlace,   // read where they are, by vectors or by elements: what is too wide for two rows' copies
    kAligned,   // copied ahead
    kShifted    // the same, of rows that start anywhere
};
// The types of dy and x are given for copied rows (DY32, X32) and looked up
// otherwise.  SUMS: dgamma and dbeta are summed.
template <bool DY32, bool X32, Rows ROWS, bool SUMS, int ITER, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS > kBackwardThreads ? 1 : kBackwardThreads / THREADS)
layer_norm_backward_kernel(const LnParams p) {
    constexpr bool COPIED = ROWS != kInPlace, SHIFTED = ROWS == kShifted;
    using D = Copy<DY32, ITER, SHIFTED>;
    using X = Copy<X32, ITER, SHIFTED>;
    using A = Copy<false, ITER, SHIFTED>;
    constexpr int kWarp = D::kBytes + X::kBytes + A::kBytes;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(8) float slots[64];
    griddep_wait();
    griddep_launch();
    const Group<false> g(p.group_warps);
    const int first = g.template first<ITER>();
    const int c0 = first - g.lane * kVec;
    const int64_t stride = (int64_t)gridDim.x * p.groups;
    const int other = (blockDim.x >> 5) * kWarp;  // from one of the two rows to the other
    const uint8_t* mine = smem + (threadIdx.x >> 5) * kWarp;
    const uint32_t saddr = (uint32_t)__cvta_generic_to_shared(mine);
    auto fetch = [&](int64_t row, int at) {
        if (row < p.rows) {
            D::fetch(saddr + at, p.dy, p.ld_dy, row, c0, p.cols);
            X::fetch(saddr + at + D::kBytes, p.x, p.ldx, row, c0, p.cols);
            if (p.add) A::fetch(saddr + at + D::kBytes + X::kBytes, p.add, p.ld_add, row, c0, p.cols);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int64_t row = (int64_t)blockIdx.x * p.groups + g.index;
    float mean_next = 0.0f, rstd_next = 0.0f;
    auto stats = [&](int64_t r) {
        if (r >= p.rows) return;
        mean_next = p.mean[r];
        rstd_next = p.rstd[r];
    };
    if (COPIED) fetch(row, 0);
    stats(row);
    uint64_t dgamma[SUMS ? ITER : 1][4], dbeta[SUMS ? ITER : 1][4];
    if (SUMS) {
#pragma unroll
        for (int k = 0; k < ITER; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) dgamma[k][i] = dbeta[k][i] = 0;
    }
    // gamma of the lane's columns, as long as registers hold it (16384 x 7168: 155 us; read again for each row 45 more)
    constexpr bool kKept = ITER <= 2;
    auto weights = [&](int k, uint64_t w[4]) {
        const int c = first + k * kStepCols;
        float v[kVec] = {};
        const int n = p.cols - c;
        if (n > 0) load_weight8(p.gamma, p.gamma_f32, COPIED ? weight_vec<SHIFTED>(p, n) : p.vec, c, n, v);
        pair8(v, w);
    };
    uint64_t gamma[kKept ? ITER : 1][4];
    if (kKept) {
#pragma unroll
        for (int k = 0; k < ITER; ++k) weights(k, gamma[k]);
    }
    int at = 0;
    for (; row < p.rows; row += stride) {
        const float mean = mean_next, r = rstd_next;
        const uint64_t minus = pk2(-mean, -mean), r2 = pk2(r, r);
        if (COPIED) {
            fetch(row + stride, at ^ other);
            asm volatile("cp.async.wait_group 1;" ::: "memory");
            __syncwarp();
        }
        stats(row + stride);
        const uint8_t* src = mine + at;
        const int of_dy = D::shift(p.dy, p.ld_dy, row), of_x = X::shift(p.x, p.ldx, row);
        // dy and the normalised row, step k; past the row's end x is the mean, so that h is 0 there as dy is (0 times a mean rstd
        // beyond fp32 is no 0)
        auto load = [&](int k, int c, int n, uint64_t dy[4], uint64_t h[4]) {
            float v[kVec];
            if (COPIED) D::read(src, k, of_dy, n, v);
            else load8_any(p.dy, row * p.ld_dy + c, p.dy_f32, p.vec, n, v);
            pair8(v, dy);
            if (COPIED) {
                X::read(src + D::kBytes, k, of_x, n, v, mean);
            } else {
                load8_any(p.x, row * p.ldx + c, p.x_f32, p.vec, n, v);
                if (n < kVec) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        if (i >= n) v[i] = mean;
                }
            }
            pair8(v, h);
#pragma unroll
            for (int i = 0; i < 4; ++i) h[i] = mul2(add2(h[i], minus), r2);
        };
        uint64_t sq = 0, sqh = 0;
#pragma unroll
        for (int k = 0; k < ITER; ++k) {
            const int c = first + k * kStepCols;
            const int n = p.cols - c;
            if (n <= 0) break;
            uint64_t dy[4], h[4], other_w[4];
            load(k, c, n, dy, h);
            if (!kKept) weights(k, other_w);
            const uint64_t* w = kKept ? gamma[k] : other_w;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (SUMS) {
                    dgamma[k][i] = fma2(dy[i], h[i], dgamma[k][i]);
                    dbeta[k][i] = add2(dy[i], dbeta[k][i]);
                }
                const uint64_t q = mul2(dy[i], w[i]);
                sq = add2(q, sq);
                sqh = fma2(q, h[i], sqh);
            }
        }
        float2 t, u;
        up2(sq, t.x, t.y);
        up2(sqh, u.x, u.y);
        const float2 sums = g.sum2(make_float2(t.x + t.y, u.x + u.y), slots);
        const float mq = -sums.x * p.inv_cols, mqh = -sums.y * p.inv_cols;
        const uint64_t mq2 = pk2(mq, mq), mqh2 = pk2(mqh, mqh);
        const int of_add = A::shift(p.add, p.ld_add, row);
        auto result = [&](int k, float v[kVec]) {
            const int c = first + k * kStepCols, n = p.cols - c;
            uint64_t dy[4], h[4], other_w[4], add[4] = {0, 0, 0, 0};
            load(k, c, n, dy, h);
            if (!kKept) weights(k, other_w);
            const uint64_t* w = kKept ? gamma[k] : other_w;
            if (p.add) {
                if (COPIED) A::read(src + D::kBytes + X::kBytes, k, of_add, n, v);
                else load8_any(p.add, row * p.ld_add + c, 0, p.vec, n, v);
                pair8(v, add);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                up2(fma2(r2, fma2(h[i], mqh2, fma2(dy[i], w[i], mq2)), add[i]), v[2 * i], v[2 * i + 1]);
        };
        if (SHIFTED) {
            const int share = min(p.cols - c0, ITER * kStepCols);
            if (share > 0) {
                const int steps = (share + kStepCols - 1) / kStepCols;
                ShiftedRow to(p.out + row * p.ld_out + c0, share);
#pragma unroll
                for (int k = 0; k < ITER; ++k) {
                    if (k >= steps) break;
                    float v[kVec];
                    result(k, v);
                    to.step(k, v);
                }
                to.finish(steps);
            }
        } else {
            __nv_bfloat16* out = p.out + row * p.ld_out + first;
#pragma unroll
            for (int k = 0; k < ITER; ++k) {
                const int n = p.cols - (first + k * kStepCols);
                if (n <= 0) break;
                float v[kVec];
                result(k, v);
                store8_any(out + k * kStepCols, COPIED ? 1 : p.vec, n, v);
            }
        }
        if (COPIED) {
            __syncwarp();  // the warp is done with this row's copies
            at ^= other;
        }
    }
    if (!SUMS) return;
    // the groups' sums, added in their order by the last one, whole lanes' elements (8192 x 2048: 27.7 us; element by element,
    // 32 bytes apart, 32.1); no copy is in flight (those past the last row copy nothing), and their memory is free once every
    // group is here
    __syncthreads();
    float* sums = reinterpret_cast<float*>(smem);
    const int pitch = partials_pitch(p.cols);
    for (int j = 0; j < p.groups; ++j) {
        if (j) __syncthreads();
        if (g.index != j) continue;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
            float* dst = (j == p.groups - 1 ? p.partials + (int64_t)blockIdx.x * 2 * pitch : sums) + which * pitch;
            const float* before = sums + which * pitch;
#pragma unroll
            for (int k = 0; k < ITER; ++k) {
                const int c = first + k * kStepCols;
                if (c >= p.cols) break;
                float v[kVec];
#pragma unroll
                for (int i = 0; i < 4; ++i) up2(which ? dbeta[k][i] : dgamma[k][i], v[2 * i], v[2 * i + 1]);
#pragma unroll
                for (int i = 0; i < kVec; i += 4) {
                    float4 t = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                    if (j) {
                        const float4 o = *reinterpret_cast<const float4*>(before + c + i);
                        t = make_float4(o.x + t.x, o.y + t.y, o.z + t.z, o.w + t.w);
                    }
                    *reinterpret_cast<float4*>(dst + c + i) = t;
                }
            }
        }
    }
}

// Rows too wide for a CTA's registers to hold their sums: partial sums of
// dgamma and dbeta of 256 columns over a share of the rows.
__global__ void __launch_bounds__(256) layer_norm_columns_kernel(const LnParams p) {
    griddep_wait();
    griddep_launch();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= p.cols) return;
    float dgamma = 0.0f, dbeta = 0.0f;
#pragma unroll 4
    for (int64_t row = blockIdx.y; row < p.rows; row += gridDim.y) {
        const int64_t i = row * p.ld_dy + c, j = row * p.ldx + c;
        const float dy = p.dy_f32 ? ((const float*)p.dy)[i] : __bfloat162float(((const __nv_bfloat16*)p.dy)[i]);
        const float x = p.x_f32 ? ((const float*)p.x)[j] : __bfloat162float(((const __nv_bfloat16*)p.x)[j]);
        dgamma = fmaf(dy, (x - p.mean[row]) * p.rstd[row], dgamma);
        dbeta += dy;
    }
    const int pitch = partials_pitch(p.cols);
    float* dst = p.partials + (int64_t)blockIdx.y * 2 * pitch + c;
    dst[0] = dgamma;
    dst[pitch] = dbeta;
}

// dgamma and dbeta: sums over the parts, in their order.  A CTA takes 32 of the 2 pitch columns, a 128-byte line of a part a warp,
// 32 slices of the parts, then the slices.  (With 8 columns a CTA, a sector of a part each: 4096 x 16384 142 us in all, 129 so.)
__global__ void __launch_bounds__(1024) layer_norm_join_kernel(const float* partials, int parts, int cols, float* dgamma,
                                                               float* dbeta) {
    __shared__ float slice[32][32 + 1];
    griddep_wait();
    griddep_launch();
    const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x * 32 + lane;
    float s = 0.0f;
    const int pitch = partials_pitch(cols);
    if (c < 2 * pitch) {
#pragma unroll 4
        for (int q = w; q < parts; q += 32) s += partials[(int64_t)q * 2 * pitch + c];
    }
    slice[w][lane] = s;
    __syncthreads();
    s = slice[lane][w];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    const int at = blockIdx.x * 32 + w;
    if (lane) return;
    if (at < cols) dgamma[at] = s;
    else if (at >= pitch && at < pitch + cols) dbeta[at - pitch] = s;
}

// ------------------------------------------------------------------- shapes
// Forward, a lane takes up to two steps (up to 16384 columns: 32 warps); with four its 64 registers do not hold the row and what
// two sums and beta take besides (16384 x 7168: 210 us, 190 with two).
Shape row_shape(int64_t cols) {
    const int64_t steps = (cols + kStepCols - 1) / kStepCols;
    const int iter = steps == 1 ? 1 : (steps <= 64 ? 2 : 4);
    return {iter, (int)((steps + iter - 1) / iter), 1};
}
// Backward, a lane takes up to two steps (up to 8192 columns: 512 threads hold
// their sums without a spill), then four (up to 16384); wider rows' sums are
// the columns kernel's.
constexpr int kMostSummed = 16384;
Shape backward_shape(int64_t cols) {
    Shape s;
    s.iter = cols <= kStepCols ? 1 : (cols <= 32 * kStepCols ? 2 : 4);
    s.warps = (int)((cols + s.iter * kStepCols - 1) / (s.iter * kStepCols));
    s.groups = std::max(1, 8 / s.warps);
    return s;
}

template <bool F32, bool SHIFTED, int ITER>
constexpr int forward_smem(int warps) {
    return warps * (Copy<F32, ITER, SHIFTED>::kBytes + Copy<false, ITER, SHIFTED>::kBytes);
}
// Two rows, and at least the sums that the groups but the last leave there.
template <bool DY32, bool X32, Rows ROWS, int ITER>
constexpr int backward_smem(int warps, int groups, int cols) {
    constexpr bool s = ROWS == kShifted;
    const int rows = ROWS == kInPlace ? 0 : 2 * warps * groups * (Copy<DY32, ITER, s>::kBytes + Copy<X32, ITER, s>::kBytes +
                                                                  Copy<false, ITER, s>::kBytes);
    const int sums = groups > 1 ? 2 * partials_pitch(cols) * 4 : 0;
    return rows > sums ? rows : sums;
}
// Of a warp's two rows, shifted ones.
size_t warp_bytes(const Shape& s, bool dy_f32, bool x_f32) {
    return 2 * (size_t)(s.iter * kStepCols * ((dy_f32 ? 4 : 2) + (x_f32 ? 4 : 2) + 2) + 3 * 16);
}
bool copies_fit(const Shape& s, bool dy_f32, bool x_f32) {
    return s.warps * s.groups * warp_bytes(s, dy_f32, x_f32) <= kMostSmem;
}

template <bool F32, bool SHIFTED, int ITER, int THREADS>
struct Fwd {
    static cudaError_t run(const LnParams& p, const Shape& s, int num_sms, cudaStream_t st) {
        const size_t smem = forward_smem<F32, SHIFTED, ITER>(s.warps * s.groups);
        const int64_t grid = std::min<int64_t>(p.rows, (int64_t)num_sms * ctas_per_sm(s, kForwardThreads, smem));
        return launch_pdl(layer_norm_kernel<F32, SHIFTED, ITER, THREADS>, dim3((unsigned)grid), dim3(s.threads()), smem, st, p);
    }
    // Loads the kernel and lets it have what the widest row it serves takes: the limit belongs to the kernel, which
    // calls of other widths use at the same time.
    static cudaError_t load() {
        constexpr int smem = forward_smem<F32, SHIFTED, ITER>(THREADS / 32);
        static_assert(smem <= (int)kMostSmem, "shared memory overflow");
        cudaFuncAttributes at;
        cudaFuncGetAttributes(&at, layer_norm_kernel<F32, SHIFTED, ITER, THREADS>);
        return cudaFuncSetAttribute(layer_norm_kernel<F32, SHIFTED, ITER, THREADS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    smem);
    }
};
template <bool F32, bool SHIFTED, typename F>
cudaError_t forward_by_shape(const Shape& s, F&& f) {
    if (s.iter == 1) return f(Fwd<F32, SHIFTED, 1, 256>());
    if (s.iter == 4) return f(Fwd<F32, SHIFTED, 4, 1024>());
    return s.threads() > 512 ? f(Fwd<F32, SHIFTED, 2, 1024>()) : f(Fwd<F32, SHIFTED, 2, 512>());
}
template <typename F>
cudaError_t forward_kernel(bool f32, bool shifted, const Shape& s, F&& f) {
    if (f32) return shifted ? forward_by_shape<true, true>(s, f) : forward_by_shape<true, false>(s, f);
    return shifted ? forward_by_shape<false, true>(s, f) : forward_by_shape<false, false>(s, f);
}

template <bool DY32, bool X32, Rows ROWS, bool SUMS, int ITER, int THREADS>
struct Bwd {
    static cudaError_t run(const LnParams& p, const Shape& s, int parts, cudaStream_t st) {
        const size_t smem = backward_smem<DY32, X32, ROWS, ITER>(s.warps, s.groups, p.cols);
        return launch_pdl(layer_norm_backward_kernel<DY32, X32, ROWS, SUMS, ITER, THREADS>, dim3((unsigned)parts),
                          dim3(s.threads()), smem, st, p);
    }
    static cudaError_t load() {
        cudaFuncAttributes at;
        cudaFuncGetAttributes(&at, layer_norm_backward_kernel<DY32, X32, ROWS, SUMS, ITER, THREADS>);
        return cudaFuncSetAttribute(layer_norm_backward_kernel<DY32, X32, ROWS, SUMS, ITER, THREADS>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, ROWS == kInPlace ? 64 * 1024 : (int)kMostSmem);
    }
};
template <bool DY32, bool X32, Rows ROWS, typename F>
cudaError_t backward_by_shape(const Shape& s, F&& f) {
    if (s.iter == 1) return f(Bwd<DY32, X32, ROWS, true, 1, 256>());
    if (s.iter == 2)
        return s.threads() > 256 ? f(Bwd<DY32, X32, ROWS, true, 2, 512>()) : f(Bwd<DY32, X32, ROWS, true, 2, 256>());
    return f(Bwd<DY32, X32, ROWS, true, 4, 512>());
}
template <Rows ROWS, typename F>
cudaError_t backward_by_type(bool dy_f32, bool x_f32, const Shape& s, F&& f) {
    if (dy_f32) return x_f32 ? backward_by_shape<true, true, ROWS>(s, f) : backward_by_shape<true, false, ROWS>(s, f);
    return x_f32 ? backward_by_shape<false, true, ROWS>(s, f) : backward_by_shape<false, false, ROWS>(s, f);
}
template <typename F>
cudaError_t backward_kernel(bool dy_f32, bool x_f32, Rows rows, const Shape& s, F&& f) {
    if (s.threads() > kBackwardThreads) return f(Bwd<false, false, kInPlace, false, 4, 1024>());
    if (rows == kInPlace) return f(Bwd<false, false, kInPlace, true, 4, 512>());
    return rows == kAligned ? backward_by_type<kAligned>(dy_f32, x_f32, s, f) : backward_by_type<kShifted>(dy_f32, x_f32, s, f);
}

LnParams common(const LayerNormArgs& a) {
    LnParams p = {};
    p.x = a.x;
    p.ldx = a.ldx;
    p.x_f32 = a.x_f32;
    p.gamma = a.gamma;
    p.beta = a.beta;
    p.gamma_f32 = a.gamma_f32;
    p.rows = a.rows;
    p.cols = (int)a.cols;
    p.inv_cols = 1.0f / (float)a.cols;
    p.eps = a.eps;
    p.mean = a.mean;
    p.rstd = a.rstd;
    return p;
}

}  // namespace

size_t layer_norm_part_bytes(int64_t cols) { return 2 * sizeof(float) * (size_t)partials_pitch((int)cols); }

int layer_norm_parts(int64_t rows, int64_t cols, int num_sms) {
    const Shape s = backward_shape(cols);
    if (cols > kMostSummed) {
        // Shares of the rows, for about eight CTAs an SM, and more where a share would have more than kMostAdded rows: a thread adds
        // them one by one, with as many roundings.  (9 shares at 32768 columns; the partial sums of 256 rows are 1 / 128 of their dy
        // and x in bf16.  Adding a share's rows 64 at a time instead cost 5 % of 2048 x 32768
        // at best, with the types as template parameters.)
        constexpr int64_t kMostAdded = 256, kMostShares = 65535;
        const int64_t chunks = (cols + 255) / 256;
        const int64_t shares = std::max(8 * (int64_t)num_sms / chunks, std::min((rows + kMostAdded - 1) / kMostAdded, kMostShares));
        return (int)std::max<int64_t>(1, std::min(rows, shares));
    }
    const size_t smem = s.warps * s.groups * warp_bytes(s, true, true);  // narrower types take as many
    return (int)std::max<int64_t>(1, std::min<int64_t>((rows + s.groups - 1) / s.groups,
                                                       (int64_t)num_sms * ctas_per_sm(s, kBackwardThreads, smem)));
}

cudaError_t launch_layer_norm(const LayerNormArgs& a, int num_sms, cudaStream_t st) {
    if (a.rows == 0) return cudaSuccess;
    LnParams p = common(a);
    p.add = (const __nv_bfloat16*)a.residual;
    p.ld_add = a.ld_residual;
    p.y = (__nv_bfloat16*)a.y;
    p.ldy = a.ldy;
    p.out = (__nv_bfloat16*)a.total;
    p.ld_out = a.ld_total;
    p.vec = a.cols % kVec == 0 && vec_ok(a.x, a.ldx, a.x_f32 ? 4 : 2, 16) && vec_ok(a.gamma, 0, 1, 16) &&
            (!a.beta || vec_ok(a.beta, 0, 1, 16)) && vec_ok(a.y, a.ldy, 2, 16) &&
            (!a.residual || vec_ok(a.residual, a.ld_residual, 2, 16)) && (!a.total || vec_ok(a.total, a.ld_total, 2, 16));
    const Shape s = row_shape(a.cols);
    p.group_warps = s.warps;
    p.groups = s.groups;
    p.vec_weights = vec_ok(a.gamma, 0, 1, 16) && (!a.beta || vec_ok(a.beta, 0, 1, 16));
    return forward_kernel(a.x_f32, !p.vec, s, [&](auto k) { return k.run(p, s, num_sms, st); });
}

cudaError_t launch_layer_norm_backward(const LayerNormArgs& a, int num_sms, cudaStream_t st) {
    LnParams p = common(a);
    p.dy = a.dy;
    p.ld_dy = a.ld_dy;
    p.dy_f32 = a.dy_f32;
    p.add = (const __nv_bfloat16*)a.dtotal;
    p.ld_add = a.ld_dtotal;
    p.out = (__nv_bfloat16*)a.dx;
    p.ld_out = a.ld_dx;
    p.partials = a.partials;
    p.vec = a.cols % kVec == 0 && vec_ok(a.dy, a.ld_dy, a.dy_f32 ? 4 : 2, 16) && vec_ok(a.x, a.ldx, a.x_f32 ? 4 : 2, 16) &&
            vec_ok(a.gamma, 0, 1, 16) && vec_ok(a.dx, a.ld_dx, 2, 16) && (!a.dtotal || vec_ok(a.dtotal, a.ld_dtotal, 2, 16));
    p.vec_weights = vec_ok(a.gamma, 0, 1, 16);
    const Shape s = backward_shape(a.cols);
    p.group_warps = s.warps;
    p.groups = s.groups;
    const int parts = layer_norm_parts(a.rows, a.cols, num_sms);  // with no rows: one part of zeros
    cudaError_t e = cudaSuccess;
    if (a.cols > kMostSummed) {  // the sums first: dx may lie where dy does
        e = launch_pdl(layer_norm_columns_kernel, dim3((unsigned)((a.cols + 255) / 256), (unsigned)parts), dim3(256), 0, st, p);
        const int64_t grid = std::min<int64_t>(a.rows, num_sms);
        if (e == cudaSuccess && grid)
            e = backward_kernel(a.dy_f32, a.x_f32, kInPlace, s, [&](auto k) { return k.run(p, s, (int)grid, st); });
    } else {
        // (what does not fit has four steps a lane)
        const Rows how = !copies_fit(s, a.dy_f32, a.x_f32) ? kInPlace : (p.vec ? kAligned : kShifted);
        e = backward_kernel(a.dy_f32, a.x_f32, how, s, [&](auto k) { return k.run(p, s, parts, st); });
    }
    if (e != cudaSuccess) return e;
    return launch_pdl(layer_norm_join_kernel, dim3((unsigned)((2 * partials_pitch((int)a.cols) + 31) / 32)), dim3(1024), 0, st,
                      (const float*)a.partials, parts, (int)a.cols, a.dgamma, a.dbeta);
}

cudaError_t preload_layer_norm_kernels() {
    const Shape fwd[] = {{1, 1, 1}, {2, 16, 1}, {2, 32, 1}, {4, 32, 1}};
    const Shape bwd[] = {{1, 1, 8}, {2, 8, 1}, {2, 16, 1}, {4, 16, 1}, {4, 32, 1}};
    for (const Shape& s : fwd)
        for (int i = 0; i < 4; ++i) forward_kernel(i & 1, i & 2, s, [](auto k) { return k.load(); });
    for (const Shape& s : bwd)
        for (int i = 0; i < 12; ++i) backward_kernel(i & 1, i & 2, (Rows)(i / 4), s, [](auto k) { return k.load(); });
    cudaFuncAttributes at;
    cudaFuncGetAttributes(&at, layer_norm_columns_kernel);
    return cudaFuncGetAttributes(&at, layer_norm_join_kernel);
}

}  // namespace ufp4
