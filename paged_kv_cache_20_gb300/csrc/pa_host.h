// pa_host.h -- host-side helpers shared by the translation units that implement the
// C ABI.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "../../include/pagedattn.h"

namespace pa {

// Device address of the current device's error word (looked up once per device);
// nullptr if it cannot be had.
unsigned *error_word();

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Whether two buffers share a byte.
inline bool overlap(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

// Block sizes the kernels take: a block of 32 tokens is read as two 16-token tiles,
// a 16-token tile spans two blocks of 8
inline bool supported_block(int b) { return b == 8 || b == 16 || b == 32; }
inline bool supported_dtype(pa_dtype d) { return d == PA_FP16 || d == PA_BF16; }

}  // namespace pa
