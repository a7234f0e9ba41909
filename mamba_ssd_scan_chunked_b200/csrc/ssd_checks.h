// Host-side argument checks shared by the entry points (ssd_api.cu, ssd_layer_api.cu).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/ssd.h"

namespace ssd {

inline size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t a0 = (uintptr_t)a, b0 = (uintptr_t)b;
    return a0 < b0 + nb && b0 < a0 + na;
}

inline bool valid_dtype(int32_t d) { return d == SSD_F32 || d == SSD_BF16; }
inline size_t dsize(int32_t d) { return d == SSD_BF16 ? 2 : 4; }

inline bool is_pow2(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }

}  // namespace ssd
