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

constexpr uint32_t kPhiloxM0 = 0xD2511F53u, kPhiloxM1 = 0xCD9E8D57u;  // multipliers
constexpr uint32_t kPhiloxW0 = 0x9E3779B9u, kPhiloxW1 = 0xBB67AE85u;  // key increments

// A call's round keys and the upper half of its counters.
struct DropoutState {
  uint32_t key0[10], key1[10], c2, c3;
};

MOE_DEV DropoutState dropout_state(const DropoutArgs& d) {
  const unsigned long long seed = d.rng[0], at = d.rng[1] + d.offset;
  DropoutState s;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    s.key0[r] = static_cast<uint32_t>(seed) + static_cast<uint32_t>(r) * kPhiloxW0;
    s.key1[r] = static_cast<uint32_t>(seed >> 32) + static_cast<uint32_t>(r) * kPhiloxW1;
  }
  s.c2 = static_cast<uint32_t>(at);
  s.c3 = static_cast<uint32_t>(at >> 32);
  return s;
}

// The first rounds mix the column and the row apart: round 1 multiplies the
// column word (c / 4) and a constant of the call, round 2 a value of the row
// and one of the column, and one factor of round 3 is the column's still.
// What depends on the column alone, or on the row alone, is kept.
struct DropoutColumn {
  uint32_t lo_a;    // low word of round 1's first product
  uint32_t c0_mix;  // round 2's second word ^ round 3's first key
  uint32_t c2_mix;  // high word of round 3's first product ^ its second key
  uint32_t c3;      // its low word
};
struct DropoutRow {
  uint32_t c2_mix;  // high word of round 2's first product ^ its second key
  uint32_t c3;      // its low word
};

MOE_DEV uint64_t wide(uint32_t a, uint32_t b) { return static_cast<uint64_t>(a) * b; }
MOE_DEV uint32_t high(uint64_t v) { return static_cast<uint32_t>(v >> 32); }
MOE_DEV uint32_t low(uint64_t v) { return static_cast<uint32_t>(v); }

MOE_DEV DropoutColumn dropout_column(const DropoutState& s, uint32_t quad) {
  const uint64_t a1 = wide(kPhiloxM0, quad), b1 = wide(kPhiloxM1, s.c2);
  const uint64_t b2 = wide(kPhiloxM1, high(a1) ^ s.c3 ^ s.key1[0]);
  const uint64_t a3 = wide(kPhiloxM0, high(b2) ^ low(b1) ^ s.key0[1]);
  return {low(a1), low(b2) ^ s.key0[2], high(a3) ^ s.key1[2], low(a3)};
}

MOE_DEV DropoutRow dropout_row(const DropoutState& s, uint32_t row) {
  const uint64_t a2 = wide(kPhiloxM0, high(wide(kPhiloxM1, s.c2)) ^ row ^ s.key0[0]);
  return {high(a2) ^ s.key1[1], low(a2)};
}

MOE_DEV uint4 dropout_words(const DropoutState& s, const DropoutColumn& col, const DropoutRow& row) {
  const uint64_t b3 = wide(kPhiloxM1, row.c2_mix ^ col.lo_a);
  uint32_t c0 = high(b3) ^ col.c0_mix, c1 = low(b3), c2 = col.c2_mix ^ row.c3, c3 = col.c3;
#pragma unroll
  for (int r = 3; r < 10; ++r) {
    const uint64_t a = wide(kPhiloxM0, c0), b = wide(kPhiloxM1, c2);
    c0 = high(b) ^ c1 ^ s.key0[r];
    c1 = low(b);
    c2 = high(a) ^ c3 ^ s.key1[r];
    c3 = low(a);
  }
  return make_uint4(c0, c1, c2, c3);
}

// Four neighbouring elements (one block of words), in place: add + the kept
// ones times 1 / (1 - p); dropped ones count as zero whatever they hold
// (infinities and NaN too).
MOE_DEV void dropout_quad(const DropoutArgs& d, const DropoutState& s, const DropoutColumn& col, const DropoutRow& row,
                          float* v, const float* add) {
  const uint4 w = dropout_words(s, col, row);
  v[0] = fmaf(w.x >= d.cut ? v[0] : 0.0f, d.scale, add[0]);
  v[1] = fmaf(w.y >= d.cut ? v[1] : 0.0f, d.scale, add[1]);
  v[2] = fmaf(w.z >= d.cut ? v[2] : 0.0f, d.scale, add[2]);
  v[3] = fmaf(w.w >= d.cut ? v[3] : 0.0f, d.scale, add[3]);
}

}  // namespace moe
