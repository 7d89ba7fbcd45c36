// What the two norms (norm.cu, layer_norm.cu) share: a group of warps that
// works on one row, its sums, and the shapes of their launches.
#pragma once

#include <algorithm>
#include <cstdint>
#include <cuda_runtime.h>

#include "ckpt8.cuh"
#include "ufp4_device.cuh"

namespace ufp4 {
namespace {

// A group of warps works on one row: a whole CTA (ALONE) or a share of it,
// with a barrier of its own.  Step k of a lane covers the 8 columns from first
// + k * kStepCols.
constexpr int kStepCols = 32 * kVec;
template <bool ALONE>
struct Group {
    int warps;   // of a group
    int index;   // in the CTA
    int warp;    // in the group
    int lane;
    __device__ __forceinline__ explicit Group(int warps_) : warps(warps_) {
        const int w = threadIdx.x >> 5;
        index = ALONE ? 0 : w / warps;
        warp = w - index * warps;
        lane = threadIdx.x & 31;
    }
    template <int ITER>
    __device__ __forceinline__ int first() const {
        return (warp * ITER * 32 + lane) * kVec;
    }
    __device__ __forceinline__ void sync() const {
        if (ALONE)
            __syncthreads();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(index + 1), "r"(warps * 32) : "memory");
    }
    // Sum over the group, the same value in every lane.  `slots`: 32 floats of the CTA.
    __device__ __forceinline__ float sum(float v, float* slots) const {
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        if (warps == 1) return v;
        slots += index * warps;
        sync();  // the slots' last readers are done
        if (lane == 0) slots[warp] = v;
        sync();
        v = lane < warps ? slots[lane] : 0.0f;
#pragma unroll
        for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
        return v;
    }
    // Two sums at once.  `slots`: 64 floats of the CTA, 8-byte aligned.
    __device__ __forceinline__ float2 sum2(float2 v, float* slots) const {
        auto all = [](float2 t) {
#pragma unroll
            for (int o = 16; o; o >>= 1) {
                t.x += __shfl_xor_sync(0xFFFFFFFFu, t.x, o);
                t.y += __shfl_xor_sync(0xFFFFFFFFu, t.y, o);
            }
            return t;
        };
        v = all(v);
        if (warps == 1) return v;
        float2* s = reinterpret_cast<float2*>(slots) + index * warps;
        sync();  // the slots' last readers are done
        if (lane == 0) s[warp] = v;
        sync();
        return all(lane < warps ? s[lane] : make_float2(0.0f, 0.0f));
    }
};

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The first `bytes` of them, zeros after.
__device__ __forceinline__ void copy16_part(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// fp32 pairs (two elements an instruction) of 8 floats.
__device__ __forceinline__ void pair8(const float v[kVec], uint64_t o[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = pk2(v[2 * i], v[2 * i + 1]);
}

bool vec_ok(const void* p, int64_t ld, int64_t bytes_per_elem, int64_t align) {
    return (uintptr_t)p % align == 0 && (ld * bytes_per_elem) % align == 0;
}

// Steps a lane takes for a row, warps of a group and groups of a CTA.
struct Shape {
    int iter, warps, groups;
    int threads() const { return 32 * warps * groups; }
};
Shape forward_shape(int64_t cols) {
    const int iter = cols <= kStepCols ? 1 : (cols <= 2 * kStepCols ? 2 : 4);
    const int warps = (int)((cols + iter * kStepCols - 1) / (iter * kStepCols));
    return {iter, warps, 1};
}
// CTAs an SM holds, with registers for `threads` threads.
int ctas_per_sm(const Shape& s, int threads, size_t smem) {
    constexpr size_t kSmSmem = 228 * 1024, kReserved = 1024 + 128;  // per SM; per CTA, beside its dynamic memory
    return std::max(1, std::min<int>(std::min(32, threads / s.threads()), (int)(kSmSmem / (smem + kReserved))));
}

}  // namespace
}  // namespace ufp4
