// Quantization to E4M3 bytes with one fp32 scale for each block of 128
// elements of a row (1 x 128), or each square block of 128 x 128: the operands
// of the block-scaled 8-bit product (fp8_gemm.cu), for the layers that keep
// more precision than 4 bits (2D-block tutorial, 混合精度取舍).  It follows the
// fp32 scale of the codebooks (UFP4 summary, section 数据集: s_B = block amax /
// largest level):
//
//   s = max(fp32(M / 448), 2^-126),  code = E4M3, nearest even, of fp32(x fp32(1/s))
//
// M the block's largest magnitude.  A transposed copy (the operand of WGRAD,
// and of DGRAD for a weight) has its blocks along the other dimension; a square
// block has the same scale and codes either way.  A block that holds a NaN or an
// infinity gets the scale M / 448 (NaN or infinity) and codes 0x7F, so that it
// reads back as NaN.
//
// Memory bounds it: 2 or 4 bytes in and 1 out for each output of an element.
// Rows alone are read as they are written, eight elements a lane, half a warp a
// block.  With a transposed or square output a CTA takes a tile of 128 x 128,
// which it reads once: a warp reads 16 rows, a lane four columns of them, so the
// row's maximum is one warp reduction on the bit patterns (magnitudes order like
// integers) and a column's is 16 of a lane's own values, joined over the warps in
// shared memory; the transposed codes, 16 rows of a column a lane, are turned
// around in shared memory and leave as whole 128-byte rows.
//
// Measured: rows of 16384 x 7168 bf16 64 us (5.5 TB/s, DRAM 63 % active, issue 73
// %); both ways of it 93 us; 8192 x 5632 fp32 both ways 55 us (5.1 TB/s; DRAM 57 %,
// 16 loads a thread in flight, 118 registers, two CTAs an SM); a square-blocked 7168 x
// 7168 fp32 both ways 49 us, bf16 35.  Loads and stores take turns within a CTA, and
// the few CTAs of an SM do not hide it all; with the elements widened to fp32 on
// arrival (twice the registers) the bf16 square took 127 us.
#include "ckpt8.cuh"
#include "internal.h"
#include "train.h"

namespace ufp4 {
namespace {

constexpr int kBlock = 128;  // elements a scale, and rows of a square one

struct Q8Params {
    const void* x;
    int64_t ld, rows, cols;
    Fp8Operand row, col;  // codes null: not wanted
    int64_t col_blocks;   // along the columns
};

struct Scale {
    float s, inv;
    bool bad;  // not finite
};
// The scale of a block whose largest magnitude has bit pattern m.  M / 448 is M / 7 (div_known_rn, correctly rounded) times
// 2^-6, which is exact down to the least scale.
__device__ __forceinline__ Scale make_scale(uint32_t m) {
    Scale q;
    q.bad = m >= 0x7F800000u;
    q.s = q.bad ? __uint_as_float(m) : fmaxf(div_known_rn(__uint_as_float(m), 7.0f, 0x1.24924ap-3f) * 0.015625f, 0x1p-126f);
    q.inv = __frcp_rn(q.s);  // of a block that is not finite unused
    return q;
}
// Four codes of values times the reciprocal scale; zeros as +0.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, uint64_t inv2) {
    return ckpt_pack4(mul2(pk2(a, b), inv2), mul2(pk2(c, d), inv2));
}

// N neighbouring elements of a row as they are read (two bf16 a word, or an fp32).  Magnitudes order like integers, a NaN's
// above an infinity's, so that maxima are taken of the bit patterns, of two bf16 at once.
template <bool F32, int N>
struct Elems {
    static constexpr int kWords = F32 ? N : N / 2;
    uint32_t w[kWords];
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = 0;
    }
    __device__ __forceinline__ void load(const void* p) {  // aligned to the vector
        if (kWords == 2) {
            const uint2 a = __ldg((const uint2*)p);
            w[0] = a.x;
            w[1] = a.y;
        } else {
#pragma unroll
            for (int i = 0; i < kWords; i += 4) {
                const uint4 a = __ldg((const uint4*)p + i / 4);
                w[i] = a.x;
                w[i + 1] = a.y;
                w[i + 2] = a.z;
                w[i + 3] = a.w;
            }
        }
    }
    __device__ __forceinline__ void load(const void* p, int n) {  // the first n, zeros after
        zero();
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < n) {
                if (F32) w[i] = ((const uint32_t*)p)[i];
                else w[i / 2] |= (uint32_t)((const uint16_t*)p)[i] << (16 * (i & 1));
            }
    }
    __device__ __forceinline__ void load_each(const void* p) {  // all of them, unaligned
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            w[i] = F32 ? ((const uint32_t*)p)[i] : __byte_perm(((const uint16_t*)p)[2 * i], ((const uint16_t*)p)[2 * i + 1], 0x5410);
    }
    __device__ __forceinline__ float at(int i) const {
        if (F32) return __uint_as_float(w[i]);
        return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
    }
    __device__ __forceinline__ uint32_t codes(int i, uint64_t inv2) const { return codes4(at(i), at(i + 1), at(i + 2), at(i + 3), inv2); }
    static constexpr uint32_t kMagnitude = F32 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
    static __device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b) { return F32 ? max(a, b) : __vmaxu2(a, b); }
    // The largest magnitude of all, as a float's bit pattern.
    __device__ __forceinline__ uint32_t top() const {
        uint32_t m = w[0] & kMagnitude;
#pragma unroll
        for (int i = 1; i < kWords; ++i) m = larger(m, w[i] & kMagnitude);
        return F32 ? m : max(m << 16, m & 0xFFFF0000u);
    }
};

// Rows alone, blocks of 1 x 128: half a warp a block, kUnroll of them apart by the CTA's 16.
constexpr int kUnroll = 4;
template <bool F32, bool VEC>
__global__ void __launch_bounds__(256, F32 ? 3 : 6) fp8_rows_kernel(const Q8Params p) {
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 15;
    const int64_t first = (int64_t)blockIdx.x * (16 * kUnroll);
    const int64_t row0 = first / p.col_blocks;
    const uint32_t at = (uint32_t)(first - row0 * p.col_blocks) + (threadIdx.x >> 4);
    const uint32_t blocks = (uint32_t)p.col_blocks;
    Elems<F32, kVec> v[kUnroll];
    int64_t row[kUnroll];
    int blk[kUnroll], n[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t i = at + u * 16;
        row[u] = row0 + i / blocks;
        blk[u] = (int)(i % blocks);
        const int64_t c = (int64_t)blk[u] * kBlock + lane * kVec;
        n[u] = row[u] < p.rows ? (int)min(p.cols - c, (int64_t)kVec) : 0;
        v[u].zero();
        const char* src = (const char*)p.x + (row[u] * p.ld + c) * (F32 ? 4 : 2);
        if (n[u] > 0) {
            if (VEC) v[u].load(src);
            else v[u].load(src, n[u]);
        }
    }
    // The blocks' maxima: lanes 4 u to 4 u + 3 end with block u's, and the scales are computed once for four lanes.
    uint32_t m[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) m[u] = v[u].top();
#pragma unroll
    for (int u = 0; u < 2; ++u) {
        const uint32_t give = lane & 8 ? m[u] : m[u + 2];
        m[u] = max(lane & 8 ? m[u + 2] : m[u], __shfl_xor_sync(0xFFFFFFFFu, give, 8));
    }
    const uint32_t give = lane & 4 ? m[0] : m[1];
    uint32_t top = max(lane & 4 ? m[1] : m[0], __shfl_xor_sync(0xFFFFFFFFu, give, 4));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    const Scale mine = make_scale(top);
    const uint32_t lost = __ballot_sync(0xFFFFFFFFu, mine.bad) >> (threadIdx.x & 16);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const float inv = __shfl_sync(0xFFFFFFFFu, mine.inv, 4 * u, 16);
        if (n[u] <= 0) continue;  // half-warps past the rows, or lanes past a short block
        const uint64_t inv2 = pk2(inv, inv);
        uint2 c = make_uint2(v[u].codes(0, inv2), v[u].codes(4, inv2));
        if (lost >> (4 * u) & 1u) c = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        uint8_t* dst = p.row.codes + row[u] * p.row.codes_ld + (int64_t)blk[u] * kBlock + lane * kVec;
        if (VEC || n[u] == kVec) {
            __stcs(reinterpret_cast<uint2*>(dst), c);
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (i < n[u]) dst[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
        }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
        if (lane == 4 * u && row[u] < p.rows) p.row.scales[row[u] * p.row.scales_ld + blk[u]] = mine.s;
}

// Tiles of 128 x 128.
template <bool F32, bool SQUARE>
__global__ void __launch_bounds__(256, F32 ? (SQUARE ? 3 : 2) : 4) fp8_tile_kernel(const Q8Params p, int vec) {
    __shared__ __align__(16) uint32_t tops[8][kBlock];        // columns' maxima by warp; a square block's by warp
    __shared__ __align__(16) uint8_t turned[kBlock * kBlock];  // transposed codes: 16-byte unit w of column c at w ^ (c / 4 % 8)
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tr = blockIdx.x / p.col_blocks, tc = blockIdx.x - tr * p.col_blocks;
    const int64_t r0 = tr * kBlock + warp * 16, c0 = tc * kBlock + lane * 4;
    const int rows = (int)max((int64_t)0, min(p.rows - r0, (int64_t)16));
    const int cols = (int)max((int64_t)0, min(p.cols - c0, (int64_t)4));
    Elems<F32, 4> v[16];
    const char* x = (const char*)p.x + (r0 * p.ld + c0) * (F32 ? 4 : 2);
    const int64_t pitch = p.ld * (F32 ? 4 : 2);
    if (vec && rows == 16 && cols == 4) {  // sixteen loads in flight
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r].load(x + r * pitch);
    } else if (!F32 && rows == 16 && cols == 4) {  // (8192 x 4999 square both ways: 40 us, with a test of each element 63)
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r].load_each(x + r * pitch);
    } else {
#pragma unroll
        for (int r = 0; r < 16; ++r) v[r].load(x + r * pitch, r < rows ? cols : 0);
    }
    uint32_t top[4];  // of the lane's columns
    {
        constexpr int kW = Elems<F32, 4>::kWords;
        constexpr uint32_t kMagnitude = Elems<F32, 4>::kMagnitude;
        uint32_t m[kW];
#pragma unroll
        for (int i = 0; i < kW; ++i) m[i] = v[0].w[i] & kMagnitude;
#pragma unroll
        for (int r = 1; r < 16; ++r)
#pragma unroll
            for (int i = 0; i < kW; ++i) m[i] = Elems<F32, 4>::larger(m[i], v[r].w[i] & kMagnitude);
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = F32 ? m[i % kW] : (i & 1 ? m[i / 2] & 0xFFFF0000u : m[i / 2] << 16);
    }
    // the reciprocal scales of the lane's columns; of a square block in all four
    float inv[4];
    bool bad[4];
    if (SQUARE) {
        const uint32_t m = __reduce_max_sync(0xFFFFFFFFu, max(max(top[0], top[1]), max(top[2], top[3])));
        if (lane == 0) tops[0][warp] = m;
        __syncthreads();
        uint32_t all = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) all = max(all, tops[0][w]);
        const Scale q = make_scale(all);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            inv[i] = q.inv;
            bad[i] = q.bad;
        }
        if (threadIdx.x == 0) {
            if (p.row.codes) p.row.scales[tr * p.row.scales_ld + tc] = q.s;
            if (p.col.codes) p.col.scales[tc * p.col.scales_ld + tr] = q.s;
        }
    } else {
        *reinterpret_cast<uint4*>(&tops[warp][lane * 4]) = make_uint4(top[0], top[1], top[2], top[3]);
    }
    if (p.row.codes) {
        // lane r computes the scale of the warp's row r
        Scale mine = {0.0f, inv[0], bad[0]};
        if (!SQUARE) {
            uint32_t m = 0;
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const uint32_t t = __reduce_max_sync(0xFFFFFFFFu, v[r].top());
                if (lane == r) m = t;
            }
            mine = make_scale(m);
            if (lane < rows) p.row.scales[(r0 + lane) * p.row.scales_ld + tc] = mine.s;
        }
        const uint32_t lost = __ballot_sync(0xFFFFFFFFu, mine.bad);
        uint8_t* dst = p.row.codes + r0 * p.row.codes_ld + c0;
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            const float f = SQUARE ? mine.inv : __shfl_sync(0xFFFFFFFFu, mine.inv, r);
            uint32_t c = v[r].codes(0, pk2(f, f));
            if (lost >> r & 1u) c = 0x7F7F7F7Fu;
            if (r >= rows) continue;
            uint8_t* d = dst + r * p.row.codes_ld;
            if (cols == 4) {
                *reinterpret_cast<uint32_t*>(d) = c;
            } else {
#pragma unroll
                for (int i = 0; i < 3; ++i)
                    if (i < cols) d[i] = (uint8_t)(c >> (8 * i));
            }
        }
    }
    if (!p.col.codes) return;
    if (!SQUARE) {
        __syncthreads();
        uint4 t = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const uint4 o = *reinterpret_cast<const uint4*>(&tops[w][lane * 4]);
            t = make_uint4(max(t.x, o.x), max(t.y, o.y), max(t.z, o.z), max(t.w, o.w));
        }
        const uint32_t m[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const Scale q = make_scale(m[i]);
            inv[i] = q.inv;
            bad[i] = q.bad;
            if (warp == 0 && i < cols) p.col.scales[(c0 + i) * p.col.scales_ld + tr] = q.s;
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t inv2 = pk2(inv[i], inv[i]);
        uint32_t c[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            c[k] = codes4(v[4 * k].at(i), v[4 * k + 1].at(i), v[4 * k + 2].at(i), v[4 * k + 3].at(i), inv2);
            if (bad[i]) c[k] = 0x7F7F7F7Fu;
        }
        const int col = lane * 4 + i;
        *reinterpret_cast<uint4*>(&turned[col * kBlock + ((warp ^ (lane & 7)) << 4)]) = make_uint4(c[0], c[1], c[2], c[3]);
    }
    __syncthreads();
    // 128-byte rows of the transposed tile: eight lanes a row, four rows a warp at a time
    const int unit = lane & 7;
    const int64_t k0 = tr * kBlock + unit * 16;
    const int left = (int)max((int64_t)0, min(p.rows - k0, (int64_t)16));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int col = warp * 16 + j * 4 + (lane >> 3);
        const int64_t c = tc * kBlock + col;
        if (c >= p.cols || left == 0) continue;
        const uint8_t* src = &turned[col * kBlock + ((unit ^ (col >> 2 & 7)) << 4)];
        uint8_t* d = p.col.codes + c * p.col.codes_ld + k0;
        if (left == 16) {
            *reinterpret_cast<uint4*>(d) = *reinterpret_cast<const uint4*>(src);
        } else {
            for (int i = 0; i < left; ++i) d[i] = src[i];
        }
    }
}

}  // namespace

cudaError_t launch_fp8_quantize(const Fp8QuantArgs& a, cudaStream_t st) {
    Q8Params p = {};
    p.x = a.x;
    p.ld = a.ld;
    p.rows = a.rows;
    p.cols = a.cols;
    p.row = a.row;
    p.col = a.col;
    p.col_blocks = (a.cols + kBlock - 1) / kBlock;
    const int64_t bytes = a.f32 ? 4 : 2;
    if (!a.square && !a.col.codes) {
        const bool vec = a.cols % kVec == 0 && (uintptr_t)a.x % 16 == 0 && a.ld * bytes % 16 == 0;
        const int64_t grid = (a.rows * p.col_blocks + 16 * kUnroll - 1) / (16 * kUnroll);
        if (grid > 0x7FFFFFFF) return cudaErrorNotSupported;
        const dim3 g((unsigned)grid), b(256);
        if (a.f32)
            return vec ? launch_pdl(fp8_rows_kernel<true, true>, g, b, 0, st, p)
                       : launch_pdl(fp8_rows_kernel<true, false>, g, b, 0, st, p);
        return vec ? launch_pdl(fp8_rows_kernel<false, true>, g, b, 0, st, p)
                   : launch_pdl(fp8_rows_kernel<false, false>, g, b, 0, st, p);
    }
    const int64_t vector = 4 * bytes;  // a lane's four elements
    const int vec = (uintptr_t)a.x % vector == 0 && a.ld % 4 == 0;
    const int64_t grid = (a.rows + kBlock - 1) / kBlock * p.col_blocks;
    if (grid > 0x7FFFFFFF) return cudaErrorNotSupported;
    const dim3 g((unsigned)grid), b(256);
    if (a.f32)
        return a.square ? launch_pdl(fp8_tile_kernel<true, true>, g, b, 0, st, p, vec)
                        : launch_pdl(fp8_tile_kernel<true, false>, g, b, 0, st, p, vec);
    return a.square ? launch_pdl(fp8_tile_kernel<false, true>, g, b, 0, st, p, vec)
                    : launch_pdl(fp8_tile_kernel<false, false>, g, b, 0, st, p, vec);
}

cudaError_t preload_fp8_quantize_kernels() {
    cudaFuncAttributes at;
    cudaFuncGetAttributes(&at, fp8_rows_kernel<true, true>);
    cudaFuncGetAttributes(&at, fp8_rows_kernel<true, false>);
    cudaFuncGetAttributes(&at, fp8_rows_kernel<false, true>);
    cudaFuncGetAttributes(&at, fp8_rows_kernel<false, false>);
    cudaFuncGetAttributes(&at, fp8_tile_kernel<true, true>);
    cudaFuncGetAttributes(&at, fp8_tile_kernel<true, false>);
    cudaFuncGetAttributes(&at, fp8_tile_kernel<false, true>);
    return cudaFuncGetAttributes(&at, fp8_tile_kernel<false, false>);
}

}  // namespace ufp4
