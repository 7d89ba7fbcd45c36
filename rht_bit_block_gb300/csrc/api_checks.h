// Argument checks that the C entry points of the training-step operators share.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/ufp4.h"
#include "train.h"

namespace ufp4 {
namespace {

inline ufp4_status to_status(cudaError_t e) {
    if (e == cudaSuccess) return UFP4_OK;
    return e == cudaErrorNotSupported ? UFP4_ERR_UNSUPPORTED : UFP4_ERR_CUDA;
}

inline bool is_dtype(int32_t t) { return t == UFP4_BF16 || t == UFP4_F32; }
inline int size_of(int32_t t) { return t == UFP4_F32 ? 4 : 2; }

// A rows x cols matrix with leading dimension ld, elements of `bytes` bytes.
inline ufp4_status check_matrix(const void* p, int64_t cols, int64_t ld, int bytes, bool optional) {
    if (!p) return optional ? UFP4_OK : UFP4_ERR_INVALID_ARG;
    if (ld < cols) return UFP4_ERR_INVALID_ARG;
    return (uintptr_t)p % bytes ? UFP4_ERR_ALIGNMENT : UFP4_OK;
}

inline ufp4_status check_workspace(const void* workspace, size_t bytes, size_t need) {
    if (!workspace || bytes < need) return UFP4_ERR_INVALID_ARG;
    return (uintptr_t)workspace % 256 ? UFP4_ERR_ALIGNMENT : UFP4_OK;
}

constexpr int64_t kMaxExtent = 1ll << 30;  // 32-bit column indices and tile counts

}  // namespace
}  // namespace ufp4

#define UFP4_CHECK(expr)                          \
    do {                                          \
        const ufp4_status s_ = (expr);            \
        if (s_ != UFP4_OK) return s_;             \
    } while (0)
