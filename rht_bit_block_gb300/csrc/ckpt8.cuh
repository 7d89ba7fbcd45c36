// The 8-bit checkpoint of a row of fp32 values, and the loads and stores that
// the operators around it share.
//
// A checkpoint is stored in the MXFP8 container of the quantizer (E4M3 byte
// codes, one E8M0 scale byte per 32 elements of a row; 2D-block tutorial, the
// format kept for the Query and Key projections), with the truncation-free
// scale rule of the UE8M0 formats (same page, S = 2^ceil(log2(M / qmax))):
// e is the least integer with M <= 448 * 2^e, M the block's largest magnitude.
// Nothing saturates then: with MXFP8's floor(log2 M) - 8 an element in
// (448, 512) * 2^e would lose up to an eighth of its value, a bias on exactly
// the outliers that a backward pass depends on most.  Eight bits are the
// point of a checkpoint: it halves (bf16) or quarters (fp32) what a layer
// keeps between its forward and its backward pass.  Its error is at most 2^-4
// of an element of at least 2^(e-6); smaller ones, below M 2^-14 or so, are
// off by up to 2^(e-10), half of E4M3's smallest step, and can become 0.
//
// A block that holds a NaN or an infinity stores scale byte 255 and 0x7F
// codes: it reads back as NaN, so an overflow is still seen in the gradients.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "train.h"
#include "ufp4_device.cuh"

namespace ufp4 {

constexpr int kCkptBlock = 32;  // elements per scale
constexpr int kVec = 8;         // elements a thread carries; four threads share a block

// max(|a|, |b|, |c|), NaN if one of them is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// E8M0 byte of a block whose largest magnitude has bit pattern m (an
// infinity's or a NaN's is 0x7F800000 or more).  For a
// normal M = f * 2^k (1 <= f < 2), 448 = 1.75 * 2^8 gives e = k - 8, plus one
// when f > 1.75; the carry of the mantissa plus 0x1FFFFF into the exponent is
// that plus one.
__device__ __forceinline__ uint32_t ckpt_scale_byte(uint32_t m) {
    if (m >= 0x7F800000u) return 255u;
    const uint32_t f = (m + 0x1FFFFFu) >> 23;
    return f > 8u ? f - 8u : 0u;
}
// 2^-e and 2^e of the scale byte e + 127 (bytes 0..247, or 255 in ckpt_unit:
// an infinity, which a 0x7F code turns into NaN).
__device__ __forceinline__ float ckpt_inv_unit(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }
__device__ __forceinline__ float ckpt_unit(uint32_t byte) { return __uint_as_float(byte ? byte << 23 : 0x00400000u); }

// Four E4M3 bytes (round to nearest even) of two fp32 pairs; zeros as +0.
__device__ __forceinline__ uint32_t ckpt_pack4(uint64_t a, uint64_t b) {
    float v0, v1, v2, v3;
    up2(a, v0, v1);
    up2(b, v2, v3);
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v1), "f"(v0));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v3), "f"(v2));
    const uint32_t c = (uint32_t)lo | ((uint32_t)hi << 16);
    const uint32_t mag = (c & 0x7F7F7F7Fu) + 0x7F7F7F7Fu;  // a byte's top bit: it has a magnitude bit
    return c & (mag | 0x7F7F7F7Fu);                        // the sign only there
}

// The values of four codes, without their block's unit.
__device__ __forceinline__ void ckpt_unpack4(uint32_t c, float* v) {
    uint32_t a, b;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(a) : "h"((uint16_t)(c & 0xFFFFu)));
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(b) : "h"((uint16_t)(c >> 16)));
    const float2 fa = __half22float2(*reinterpret_cast<const __half2*>(&a));
    const float2 fb = __half22float2(*reinterpret_cast<const __half2*>(&b));
    v[0] = fa.x;
    v[1] = fa.y;
    v[2] = fb.x;
    v[3] = fb.y;
}

__device__ __forceinline__ void widen8(const uint4& a, float v[kVec]) {  // 8 bf16
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}
__device__ __forceinline__ void widen8(const float4& a, const float4& b, float v[kVec]) {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

// The 8 elements at p (bf16 or fp32) as fp32.  VEC: p is aligned to the
// vector and all 8 exist; otherwise the first n of them, zeros after.
template <bool F32, bool VEC>
__device__ __forceinline__ void load8(const void* p, int n, float v[kVec]) {
    if (VEC) {
        if (F32) {
            const float4* q = reinterpret_cast<const float4*>(p);
            widen8(__ldcs(q), __ldcs(q + 1), v);
        } else {
            widen8(__ldcs(reinterpret_cast<const uint4*>(p)), v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            v[i] = i < n ? (F32 ? reinterpret_cast<const float*>(p)[i]
                                : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]))
                         : 0.0f;
    }
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

template <bool VEC>
__device__ __forceinline__ void store8_bf16(__nv_bfloat16* p, int n, const float v[kVec]) {
    if (VEC) {
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                                       pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])));
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < n) p[i] = __float2bfloat16_rn(v[i]);
    }
}

// Writes elements c .. c + 7 of a row; the four lanes of a quad hold one
// block of 32 and call this together (n = 0 past the end of the row).
template <bool VEC>
__device__ __forceinline__ void ckpt_store8(const Ckpt& k, int64_t row, int c, int n, const float v[kVec]) {
    float m = max_abs3(v[0], v[1], v[2]);
    m = max_abs3(m, v[3], v[4]);
    m = max_abs3(m, v[5], v[6]);
    m = max_abs3(m, v[7], __shfl_xor_sync(0xFFFFFFFFu, max_abs3(m, v[7], v[7]), 1));
    m = max_abs3(m, m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    const uint32_t byte = ckpt_scale_byte(__float_as_uint(m));
    const float inv = ckpt_inv_unit(byte);  // unused where the block is not finite
    const uint64_t inv2 = pk2(inv, inv);
    uint64_t t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = mul2(pk2(v[2 * i], v[2 * i + 1]), inv2);
    uint2 q = make_uint2(ckpt_pack4(t[0], t[1]), ckpt_pack4(t[2], t[3]));
    if (byte == 255u) q = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    if (n <= 0) return;
    uint8_t* dst = k.codes + row * k.codes_ld + c;
    if (VEC) {
        __stcs(reinterpret_cast<uint2*>(dst), q);
    } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < n) dst[i] = (uint8_t)((i < 4 ? q.x : q.y) >> (8 * (i & 3)));
    }
    if ((c & (kCkptBlock - 1)) == 0) k.scales[row * k.scales_ld + c / kCkptBlock] = (uint8_t)byte;
}

// The values of elements c .. c + 7 of a row (zeros past n).
template <bool VEC>
__device__ __forceinline__ void ckpt_load8(const Ckpt& k, int64_t row, int c, int n, float v[kVec]) {
    uint2 q = make_uint2(0u, 0u);
    uint32_t byte = 0;
    if (n > 0) {
        byte = k.scales[row * k.scales_ld + c / kCkptBlock];
        const uint8_t* src = k.codes + row * k.codes_ld + c;
        if (VEC) {
            q = __ldcs(reinterpret_cast<const uint2*>(src));
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i) {
                const uint32_t b = i < n ? (uint32_t)src[i] << (8 * (i & 3)) : 0u;
                if (i < 4) q.x |= b; else q.y |= b;
            }
        }
    }
    const float unit = ckpt_unit(byte);
    ckpt_unpack4(q.x, v);
    ckpt_unpack4(q.y, v + 4);
    const uint64_t unit2 = pk2(unit, unit);
#pragma unroll
    for (int i = 0; i < 4; ++i) up2(mul2(pk2(v[2 * i], v[2 * i + 1]), unit2), v[2 * i], v[2 * i + 1]);
    if (!VEC && byte == 255u) {  // the zeros past the end of a row stay zeros beside a NaN block
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i >= n) v[i] = 0.0f;
    }
}

}  // namespace ufp4
