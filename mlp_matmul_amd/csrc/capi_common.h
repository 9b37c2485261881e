// Helpers shared by the C ABI entry points: errors, pointer checks and the
// descriptor of a compressed matrix.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <string>

#include "uw_internal.h"

namespace uw {

inline int hip_fail(hipError_t e, const char* what) {
    return fail(UW_EHIP, std::string(what) + ": " + hipGetErrorString(e));
}

inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

inline uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }

inline void pack_palette(const uint8_t pal[16], uint32_t out[4]) {
    for (int i = 0; i < 4; ++i)
        out[i] = uint32_t(pal[4 * i]) | (uint32_t(pal[4 * i + 1]) << 8) | (uint32_t(pal[4 * i + 2]) << 16) |
                 (uint32_t(pal[4 * i + 3]) << 24);
}

// Shape and size checks of a descriptor (defined with the matmul entry points).
int check_dmat(const uw_dmat* d, const char* who);

// The raw exponents, NULL without verbatim groups: the section is empty then,
// and kernels whose lanes load from its start take another address for NULL.
inline const uint8_t* vexp_of(const uw_dmat* d) { return d->verbatim_groups ? d->vexp : nullptr; }

// Compute units of the current device (256 if it cannot be queried).
int device_cus();

}  // namespace uw
