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
// The scale of a block whose largest magnitude has bit pattern m.
__device__ __forceinline__ Scale make_scale(uint32_t m) {
    Scale q;
    q.s = __fdiv_rn(__uint_as_float(m), 448.0f);
    q.bad = m >= 0x7F800000u;
    if (!q.bad) q.s = fmaxf(q.s, 1.17549435e-38f);
    q.inv = q.bad ? __uint_as_float(0x7FFFFFFFu) : __frcp_rn(q.s);  // NaN: every code of the block becomes 0x7F or 0xFF
    return q;
}
// Four codes of values times the reciprocal scale; zeros as +0, NaN as 0x7F.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d, uint64_t inv2) {
    return ckpt_pack4(mul2(pk2(a, b), inv2), mul2(pk2(c, d), inv2));
}
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Rows alone, blocks of 1 x 128: half a warp a block, kUnroll of them apart by the CTA's 16.
constexpr int kUnroll = 4;
template <bool F32, bool VEC>
__global__ void __launch_bounds__(256) fp8_rows_kernel(const Q8Params p) {
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 15;
    const int64_t first = (int64_t)blockIdx.x * (16 * kUnroll);
    const int64_t row0 = first / p.col_blocks;
    const uint32_t at = (uint32_t)(first - row0 * p.col_blocks) + (threadIdx.x >> 4);
    const uint32_t blocks = (uint32_t)p.col_blocks;
    float v[kUnroll][kVec];
    int64_t row[kUnroll];
    int blk[kUnroll], n[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        const uint32_t i = at + u * 16;
        row[u] = row0 + i / blocks;
        blk[u] = (int)(i % blocks);
        const int64_t c = (int64_t)blk[u] * kBlock + lane * kVec;
        n[u] = row[u] < p.rows ? (int)min(p.cols - c, (int64_t)kVec) : 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[u][i] = 0.0f;
        if (n[u] > 0) load8<F32, VEC>((const char*)p.x + (row[u] * p.ld + c) * (F32 ? 4 : 2), n[u], v[u]);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i) m = max(m, magnitude(v[u][i]));
#pragma unroll
        for (int o = 8; o; o >>= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
        if (n[u] <= 0) continue;  // whole half-warps past the rows, or lanes past a short block
        const Scale q = make_scale(m);
        const uint64_t inv2 = pk2(q.inv, q.inv);
        uint2 c = make_uint2(codes4(v[u][0], v[u][1], v[u][2], v[u][3], inv2), codes4(v[u][4], v[u][5], v[u][6], v[u][7], inv2));
        if (q.bad) c = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
        uint8_t* dst = p.row.codes + row[u] * p.row.codes_ld + (int64_t)blk[u] * kBlock + lane * kVec;
        if (VEC) {
            __stcs(reinterpret_cast<uint2*>(dst), c);
        } else {
#pragma unroll
            for (int i = 0; i < kVec; ++i)
                if (i < n[u]) dst[i] = (uint8_t)((i < 4 ? c.x : c.y) >> (8 * (i & 3)));
        }
        if (lane == 0) p.row.scales[row[u] * p.row.scales_ld + blk[u]] = q.s;
    }
}

// Tiles of 128 x 128.
template <bool F32, bool SQUARE>
__global__ void __launch_bounds__(256, 2) fp8_tile_kernel(const Q8Params p, int vec) {
    __shared__ __align__(16) uint32_t tops[8][kBlock];        // columns' maxima by warp; a square block's by warp
    __shared__ __align__(16) uint8_t turned[kBlock * kBlock];  // transposed codes: 16-byte unit w of column c at w ^ (c / 4 % 8)
    griddep_wait();
    griddep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t tr = blockIdx.x / p.col_blocks, tc = blockIdx.x - tr * p.col_blocks;
    const int64_t r0 = tr * kBlock + warp * 16, c0 = tc * kBlock + lane * 4;
    const int rows = (int)max((int64_t)0, min(p.rows - r0, (int64_t)16));
    const int cols = (int)max((int64_t)0, min(p.cols - c0, (int64_t)4));
    float v[16][4];
    const char* x = (const char*)p.x + (r0 * p.ld + c0) * (F32 ? 4 : 2);
    const int64_t pitch = p.ld * (F32 ? 4 : 2);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[r][i] = 0.0f;
        if (r >= rows || cols <= 0) continue;
        const char* src = x + r * pitch;
        if (vec && cols == 4) {
            if (F32) {
                const float4 t = __ldcs(reinterpret_cast<const float4*>(src));
                v[r][0] = t.x; v[r][1] = t.y; v[r][2] = t.z; v[r][3] = t.w;
            } else {
                const uint2 t = __ldcs(reinterpret_cast<const uint2*>(src));
                v[r][0] = __uint_as_float(t.x << 16);
                v[r][1] = __uint_as_float(t.x & 0xFFFF0000u);
                v[r][2] = __uint_as_float(t.y << 16);
                v[r][3] = __uint_as_float(t.y & 0xFFFF0000u);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (i < cols)
                    v[r][i] = F32 ? reinterpret_cast<const float*>(src)[i]
                                  : __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(src)[i]);
        }
    }
    uint32_t top[4] = {0, 0, 0, 0};  // of the lane's columns
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = max(top[i], magnitude(v[r][i]));
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
                const uint32_t t = __reduce_max_sync(
                    0xFFFFFFFFu, max(max(magnitude(v[r][0]), magnitude(v[r][1])), max(magnitude(v[r][2]), magnitude(v[r][3]))));
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
            uint32_t c = codes4(v[r][0], v[r][1], v[r][2], v[r][3], pk2(f, f));
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
            c[k] = codes4(v[4 * k][i], v[4 * k + 1][i], v[4 * k + 2][i], v[4 * k + 3][i], inv2);
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
