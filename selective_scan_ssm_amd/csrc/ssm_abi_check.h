// Argument checks shared by the C ABI's translation units (ssm_abi.cpp,
// block_abi.cpp).  Host arithmetic only: nothing here touches the HIP runtime.
#pragma once

#include <hip/hip_runtime.h>

#include <cstddef>
#include <cstdint>
#include <limits>

#include "ssm_scan.h"

namespace ssm {
namespace abi {

constexpr int64_t kMaxGridY = 65535;   // batch rides on gridDim.y in the scan kernels

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// byte range [p, p + bytes) of one tensor, for overlap checks
struct Range {
    uintptr_t lo, hi;
};
inline Range range(const void *p, int64_t elems, size_t esize) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return {lo, lo + static_cast<uintptr_t>(elems) * esize};
}
inline bool overlap(Range a, Range b) {
    if (a.lo == 0 || b.lo == 0 || a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

// a*b*c without int64 overflow; -1 on overflow
inline int64_t mul3(int64_t a, int64_t b, int64_t c) {
    const int64_t big = std::numeric_limits<int64_t>::max() / 16;
    if (a < 0 || b < 0 || c < 0) return -1;
    if (a && b > big / a) return -1;
    const int64_t ab = a * b;
    if (ab && c > big / ab) return -1;
    return ab * c;
}

inline int check_dtype(int io) { return (io == SSM_F32 || io == SSM_BF16) ? SSM_OK : SSM_ERR_DTYPE; }
inline size_t io_size(int io) { return io == SSM_BF16 ? 2 : 4; }

inline int hip_status(hipError_t e) { return e == hipSuccess ? SSM_OK : SSM_ERR_HIP; }

}  // namespace abi
}  // namespace ssm
