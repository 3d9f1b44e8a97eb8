// tsenor_checks.h -- argument checks that the C entry points of the 8-bit and dense operators share.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "tsenor.h"
#include "tsenor_internal.h"

namespace tsenor {

// Operands of at most this many entries keep every offset and every count of workgroups
// inside int64; whether the workgroups fit one launch is for the launch functions (grid_fits).
constexpr int64_t kMaxEntries = int64_t(1) << 40;

inline bool misaligned(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }
// rows x cols entries, each padded by up to `pad`, without overflow
inline bool too_big(int64_t rows, int64_t cols, int64_t pad = 0) {
    return rows > kMaxEntries || cols > kMaxEntries || (cols > 0 && rows + pad > kMaxEntries / (cols + pad));
}
inline bool float_type(int t) { return t == TSENOR_F32 || t == TSENOR_BF16; }
inline int element_size(int t) { return t == TSENOR_F32 ? 4 : 2; }

// The status of a launch.
inline int status(int e, const char* where) {
    if (e == kGridTooLarge) return TSENOR_ERR_SHAPE;
    return e == hipSuccess ? TSENOR_OK : hip_error(e, where);
}

}  // namespace tsenor
