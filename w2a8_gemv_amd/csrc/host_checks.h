// Argument checks shared by the host sides of the entry points on buffers
// that must not meet.
#pragma once

#include <stdint.h>

#include "w2a8_mx4.h"

namespace w2a8 {

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0; }
inline bool type_ok(int t) { return t == W2A8_F32 || t == W2A8_BF16 || t == W2A8_F16; }
inline int64_t type_bytes(int type) { return type == W2A8_F32 ? 4 : 2; }

// Do two buffers share bytes?  A kernel reads what others of its workgroups
// have written by then, so outputs have to be apart from all other buffers.
inline bool meet(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return a && b && x < y + uint64_t(nb) && y < x + uint64_t(na);
}

}  // namespace w2a8
