// C ABI of the 8-bit operands with a scale for each block of 128, and of their
// product (declared in include/ufp4.h): argument checks and dispatch.  Nothing
// is launched when an argument is rejected, and nothing here allocates device
// memory.
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/ufp4.h"
#include "api_checks.h"
#include "train.h"

using namespace ufp4;

namespace {

constexpr int64_t kBlock = 128;

bool is_block(int32_t rows) { return rows == 1 || rows == kBlock; }

// A rows x cols operand whose blocks have block_rows rows.
ufp4_status check_operand(const ufp4_qtensor* q, int64_t rows, int64_t cols, Fp8Operand* out) {
    if (!q->codes || !q->scales || q->rows != rows || q->cols != cols) return UFP4_ERR_INVALID_ARG;
    if (q->codes_ld < cols || q->scales_ld < (cols + kBlock - 1) / kBlock) return UFP4_ERR_INVALID_ARG;
    if ((uintptr_t)q->codes % 16 || q->codes_ld % 16 || (uintptr_t)q->scales % 4) return UFP4_ERR_ALIGNMENT;
    *out = {(uint8_t*)q->codes, (float*)q->scales, q->codes_ld, q->scales_ld};
    return UFP4_OK;
}

}  // namespace

extern "C" {

ufp4_status ufp4_fp8_quantize(const void* x, int64_t ld, int32_t x_dtype, int64_t rows, int64_t cols, int32_t block_rows,
                              const ufp4_qtensor* rowwise, const ufp4_qtensor* colwise, cudaStream_t stream) {
    if (rows < 0 || cols < 0 || !is_dtype(x_dtype) || !is_block(block_rows)) return UFP4_ERR_INVALID_ARG;
    if (!rowwise && !colwise) return UFP4_ERR_INVALID_ARG;
    if (rows == 0 || cols == 0) return UFP4_OK;
    if (rows > kMaxExtent || cols > kMaxExtent) return UFP4_ERR_UNSUPPORTED;
    Fp8QuantArgs a = {};
    UFP4_CHECK(check_matrix(x, cols, ld, size_of(x_dtype), false));
    if (rowwise) UFP4_CHECK(check_operand(rowwise, rows, cols, &a.row));
    if (colwise) UFP4_CHECK(check_operand(colwise, cols, rows, &a.col));
    a.x = x;
    a.ld = ld;
    a.rows = rows;
    a.cols = cols;
    a.f32 = x_dtype == UFP4_F32;
    a.square = block_rows == kBlock;
    current_num_sms();  // loads the kernels
    return to_status(launch_fp8_quantize(a, stream));
}

ufp4_status ufp4_fp8_gemm(const ufp4_qtensor* A, int32_t a_block_rows, const ufp4_qtensor* B, int32_t b_block_rows, void* D,
                          int64_t ldd, int32_t d_dtype, int32_t accumulate, cudaStream_t stream) {
    if (!A || !B || !is_block(a_block_rows) || !is_block(b_block_rows) || !is_dtype(d_dtype)) return UFP4_ERR_INVALID_ARG;
    if (accumulate < 0 || accumulate > 1) return UFP4_ERR_INVALID_ARG;
    if (accumulate && d_dtype != UFP4_F32) return UFP4_ERR_UNSUPPORTED;
    const int64_t M = A->rows, N = B->rows, K = A->cols;
    if (M < 0 || N < 0 || K < 0 || B->cols != K) return UFP4_ERR_INVALID_ARG;
    if (M == 0 || N == 0) return UFP4_OK;
    if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return UFP4_ERR_UNSUPPORTED;
    if ((M / kBlock + 1) * (N / kBlock + 1) >= 1ll << 27) return UFP4_ERR_UNSUPPORTED;  // tiles, in up to eight shares
    UFP4_CHECK(check_matrix(D, N, ldd, size_of(d_dtype), false));
    if (K == 0) {  // a sum of nothing
        if (accumulate) return UFP4_OK;
        const size_t bytes = size_of(d_dtype);
        return to_status(cudaMemset2DAsync(D, (size_t)ldd * bytes, 0, (size_t)N * bytes, (size_t)M, stream));
    }
    Fp8GemmArgs a = {};
    UFP4_CHECK(check_operand(A, M, K, &a.a));
    UFP4_CHECK(check_operand(B, N, K, &a.b));
    a.a_square = a_block_rows == kBlock;
    a.b_square = b_block_rows == kBlock;
    a.M = M;
    a.N = N;
    a.K = K;
    a.d = D;
    a.ldd = ldd;
    a.d_f32 = d_dtype == UFP4_F32;
    a.accumulate = accumulate;
    current_num_sms();  // loads the kernels
    return to_status(launch_fp8_gemm(a, stream));
}

}  // extern "C"
