// Argument checks shared by the C ABI's translation units (host only).
#pragma once
#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>

#include "ttt.h"

namespace ttt {

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

inline bool dtype_ok(int io_dtype)
{
    return io_dtype == TTT_DTYPE_F32 || io_dtype == TTT_DTYPE_BF16;
}

inline int launch_status(hipError_t e) { return e == hipSuccess ? TTT_OK : TTT_ERR_LAUNCH; }

// [p, p + n) and [q, q + m) share a byte
inline bool overlap(const void* p, size_t n, const void* q, size_t m)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + m && b < a + n;
}

}  // namespace ttt
