// Argument checks shared by the C ABI's files (host only): each returns a status
// and leaves the message behind blockint8_last_error.
#pragma once

#include <cstdint>

#include "../../include/blockint8.h"
#include "internal.hpp"

namespace bi8 {
namespace checks {

constexpr int64_t kMaxRows = 0x7FFFFFFFll;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline int32_t done(const char *fn) { return bi8::call_status(fn, hipSuccess); }

inline int32_t check_rows(const char *fn, const char *what, int64_t rows) {
    if (rows < 0 || rows > kMaxRows)
        return fail_status(BI8_ERR_SHAPE, "%s: %s = %lld out of range", fn, what, (long long)rows);
    return BI8_OK;
}

inline int32_t check_columns(const char *fn, const char *what, int64_t K) {
    if (K <= 0 || K > BI8_MAX_K)
        return fail_status(BI8_ERR_SHAPE, "%s: %s = %lld out of range [1, %d]", fn, what, (long long)K, BI8_MAX_K);
    return BI8_OK;
}

inline int32_t check_pitch(const char *fn, const char *what, int64_t ld, int64_t K) {
    if (ld < K)
        return fail_status(BI8_ERR_SHAPE, "%s: %s = %lld < %lld columns", fn, what, (long long)ld, (long long)K);
    return BI8_OK;
}

inline int32_t check_block(const char *fn, int32_t block_n, int32_t block_k) {
    if (block_n != 128 || block_k != 128)
        return fail_status(BI8_ERR_BLOCK, "%s: only the [128, 128] block is implemented, got [%d, %d]", fn, block_n,
                           block_k);
    return BI8_OK;
}

inline int32_t check_align(const char *fn, const char *what, const void *p, uintptr_t a) {
    if (!aligned(p, a))
        return fail_status(BI8_ERR_ALIGN, "%s: %s must be %d-byte aligned", fn, what, (int)a);
    return BI8_OK;
}

inline int32_t null_pointer(const char *fn) { return fail_status(BI8_ERR_NULL, "%s: NULL tensor pointer", fn); }

inline int32_t check_workspace(const char *fn, const void *workspace, int64_t bytes) {
    if (bytes < 0) return fail_status(BI8_ERR_SHAPE, "%s: workspace_bytes = %lld < 0", fn, (long long)bytes);
    return check_align(fn, "workspace", workspace, 16);
}

}  // namespace checks
}  // namespace bi8

// Returns from the entry point with the status of a failed check.
#define BI8_TRY(expr)               \
    do {                            \
        const int32_t s_ = (expr);  \
        if (s_ != BI8_OK) return s_; \
    } while (0)
