// Dropout masks from a counter-based generator: nothing is stored, the
// backward draws the same mask again.
//
// Philox4x32 with ten rounds (J. Salmon, M. Moraes, R. Dror, D. Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", SC 2011): four 32-bit words
// from a 128-bit counter under a 64-bit key. Element (r, c) of a matrix takes
// word c % 4 of the counter (c / 4, r, offset low, offset high) under the
// seed, so the mask depends on the element's place alone, not on strides,
// vector widths or the launch. It is kept where the word is at least
// floor(p 2^32), which happens with probability 1 - floor(p 2^32) / 2^32.
#pragma once

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

struct DropoutState {  // a call's key and the upper half of its counters
  uint32_t k0, k1, c2, c3;
};

MOE_DEV DropoutState dropout_state(const DropoutArgs& d) {
  const unsigned long long seed = d.rng[0], at = d.rng[1] + d.offset;
  return {static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(at),
          static_cast<uint32_t>(at >> 32)};
}

MOE_DEV uint4 dropout_words(const DropoutState& s, uint32_t c0, uint32_t c1) {
  uint32_t c2 = s.c2, c3 = s.c3, k0 = s.k0, k1 = s.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c0, b = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(b);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Four neighbouring elements (columns 4 quad .. 4 quad + 3 of row r): the kept
// ones times 1 / (1 - p), the others zero whatever they hold (infinities and
// NaN too).
MOE_DEV void dropout_quad(const DropoutArgs& d, const DropoutState& s, uint32_t quad, uint32_t r, float* v) {
  const uint4 w = dropout_words(s, quad, r);
  v[0] = w.x >= d.cut ? v[0] * d.scale : 0.0f;
  v[1] = w.y >= d.cut ? v[1] * d.scale : 0.0f;
  v[2] = w.z >= d.cut ? v[2] * d.scale : 0.0f;
  v[3] = w.w >= d.cut ? v[3] * d.scale : 0.0f;
}

}  // namespace moe
