// Host-side argument checks shared by the C entry points.
#pragma once
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

inline bool dtype_ok(kda_dtype_t t) { return t == KDA_F32 || t == KDA_BF16; }
inline int64_t dtype_size(kda_dtype_t t) { return t == KDA_BF16 ? 2 : 4; }
inline bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

struct range {  // a tensor's bytes; absent ones overlap nothing
    const void *p;
    int64_t bytes;
};
inline bool overlap(const range &a, const range &b) {
    if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// Pools are below 2^48 bytes, so that no product of their sizes leaves 64 bits.
inline bool pool_ok(int64_t slots, int64_t slot_bytes) {
    return slot_bytes == 0 || slots <= ((int64_t)1 << 48) / slot_bytes;
}

}  // namespace kda
