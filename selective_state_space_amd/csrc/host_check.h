// Host-side argument checks and error reporting shared by the C entry points
// (defined in ssd_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/ssd.h"

namespace ssd {

// Records the detail of an error for ssd_last_error_detail() and returns st.
ssd_status fail(ssd_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3)));
// Clears the detail and returns SSD_OK.
ssd_status ok();
// SSD_OK, or SSD_ERR_HIP with the launch's error.
ssd_status hip_result(hipError_t e, const char *what, hipStream_t st);

inline bool misaligned(const void *p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u); }
inline size_t align256(size_t v) { return (v + 255) & ~size_t(255); }

constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr uint64_t kMaxGrid = (uint64_t(1) << 31) - 1;

}  // namespace ssd

#define REQUIRE_PTR(p)                                                                    \
    do {                                                                                  \
        if (!(p)) return ssd::fail(SSD_ERR_NULL, "%s is NULL", #p);                       \
        if (ssd::misaligned(p))                                                           \
            return ssd::fail(SSD_ERR_ALIGN, "%s is not 16-byte aligned", #p);             \
    } while (0)
#define OPTIONAL_PTR(p)                                                                   \
    do {                                                                                  \
        if (ssd::misaligned(p))                                                           \
            return ssd::fail(SSD_ERR_ALIGN, "%s is not 16-byte aligned", #p);             \
    } while (0)
