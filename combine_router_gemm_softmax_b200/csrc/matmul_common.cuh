// What the kernels of the free products (moe_grouped_gemm, moe_linear and
// their gradients) share: the argument block, the ragged row groups, the
// activations with their derivatives, and the epilogue of one output element.
//
//   rows mode    D[r, n] = fin( sum_k A[r, k] B_e[., .] ), r in group e's rows.
//                Forward: A = x, B_e = W_e [N, K]. Input gradient: A = dy,
//                B_e = W_e read across (its rows are the reduction).
//   weight mode  D_e[m, n] = sum_{r in group e} A[r, m] B[r, n] (A = dy, B = x).
#pragma once

#include "moe_common.cuh"
#include "moe_internal.h"

namespace moe {

// Rows of group e: [offsets[e], offsets[e+1]) held inside [0, rows], so that
// no offset the caller passes leads outside the buffers; one group of all
// rows without offsets. The bounds may be clamped, which the kernels report
// as MOE_STATUS_BAD_OFFSETS.
MOE_DEV int2 group_rows(const int32_t* offsets, int e, int rows, bool* bad = nullptr) {
  if (offsets == nullptr) return make_int2(0, rows);
  const int a = offsets[e], b = offsets[e + 1];
  const int r0 = min(max(a, 0), rows), r1 = min(max(b, r0), rows);
  if (bad != nullptr && (r0 != a || r1 != b)) *bad = true;
  return make_int2(r0, r1);
}

// One warp: s_rows[e] (if wanted) = group e's rows, prefix[e] = row tiles (of 2^tile_shift rows)
// before group e, prefix[E] = all of them. E <= kMaxE (eight groups a lane).
MOE_DEV void build_groups(const int32_t* offsets, int E, int rows, int tile_shift, int2* s_rows, int* prefix,
                          int32_t* status, int lane) {
  int loc[kMaxE / 32];
  int sum = 0;
  bool bad = false;
#pragma unroll
  for (int v = 0; v < kMaxE / 32; ++v) {
    const int e = lane * (kMaxE / 32) + v;
    loc[v] = 0;
    if (e < E) {
      const int2 r = group_rows(offsets, e, rows, &bad);
      if (s_rows != nullptr) s_rows[e] = r;
      loc[v] = (r.y - r.x + (1 << tile_shift) - 1) >> tile_shift;
    }
    sum += loc[v];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  int run = inc - sum;
#pragma unroll
  for (int v = 0; v < kMaxE / 32; ++v) {
    const int e = lane * (kMaxE / 32) + v;
    if (e < E) prefix[e] = run;
    run += loc[v];
  }
  if (lane == 31) prefix[E] = inc;
  if (bad && blockIdx.x == 0) report_status(status, MOE_STATUS_BAD_OFFSETS);
}

// The block of 2^shift rows with index `block`, counted over all groups: its
// group and rows. False if there are fewer. Every warp finds it for itself
// (each lane eight groups), so that nothing waits on a barrier before the
// weights' loads.
struct RowBlock {
  int e, r0, end;
};

MOE_DEV bool find_block(const int32_t* offsets, int E, int rows, int shift, int block, int32_t* status, int lane,
                        RowBlock& out) {
  constexpr int kPer = kMaxE / 32;
  int2 g[kPer];
  int blocks[kPer], sum = 0;
  bool bad = false;
#pragma unroll
  for (int v = 0; v < kPer; ++v) {
    const int e = lane * kPer + v;
    g[v] = e < E ? group_rows(offsets, e, rows, &bad) : make_int2(0, 0);
    blocks[v] = (g[v].y - g[v].x + (1 << shift) - 1) >> shift;
    sum += blocks[v];
  }
  if (bad) report_status(status, MOE_STATUS_BAD_OFFSETS);
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  const uint32_t past = __ballot_sync(0xffffffffu, inc > block);
  if (past == 0) return false;
  int left = block - (inc - sum);  // blocks before it in this lane's groups (if it is this lane's)
  RowBlock mine{};
  bool found = false;
#pragma unroll
  for (int v = 0; v < kPer; ++v) {
    if (!found && left < blocks[v]) {
      mine = {lane * kPer + v, g[v].x + (left << shift), g[v].y};
      found = true;
    }
    left -= blocks[v];
  }
  const int src = __ffs(past) - 1;
  out.e = __shfl_sync(0xffffffffu, mine.e, src);
  out.r0 = __shfl_sync(0xffffffffu, mine.r0, src);
  out.end = __shfl_sync(0xffffffffu, mine.end, src);
  return true;
}

// The group that row tile t belongs to: prefix[e] <= t < prefix[e+1].
MOE_DEV int group_of_tile(const int* prefix, int E, int t) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// ------------------------------------------------------------------ activations
// Two forms of each: for fp32 outputs the IEEE functions, for outputs that are
// rounded to bf16 (kFast) base-2 exponentials and reciprocals by the
// approximate instructions (about 2 ulp) with the constants folded, since the
// activation's issue slots are what bounds an epilogue of a short reduction:
// the slope of GELU's tanh form takes 11 instructions instead of 25.
MOE_DEV float ex2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

MOE_DEV float rcp_fast(float x) {  // 0 for infinity
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

constexpr float kLog2E = 1.4426950408889634f;
constexpr float kGeluTanhC = 0.7978845608028654f;  // sqrt(2 / pi)
constexpr float kGeluTanhA = 0.044715f;

// 1 / (1 + e^-z)
template <bool kFast>
MOE_DEV float sigmoid_of(float z) {
  return kFast ? rcp_fast(1.0f + ex2_fast(-kLog2E * z)) : 1.0f / (1.0f + expf(-z));
}

// sigmoid(2 u) with u = sqrt(2/pi) (z + 0.044715 z^3). The tanh form of GELU is
// z sigmoid(2 u), since (1 + tanh u) / 2 = sigmoid(2 u): no cancellation for
// negative z.
template <bool kFast>
MOE_DEV float gelu_sigmoid(float z) {
  if constexpr (kFast) {
    const float p = fmaf(z * z, -2.0f * kLog2E * kGeluTanhC * kGeluTanhA, -2.0f * kLog2E * kGeluTanhC);
    return rcp_fast(1.0f + ex2_fast(z * p));
  } else {
    return sigmoid_of<false>(2.0f * kGeluTanhC * (z + kGeluTanhA * z * z * z));
  }
}

// The negative tail of Phi, the standard normal distribution function, by fast
// instructions: Phi(-|z|) = gauss s q(s) with gauss = exp(-z^2 / 2),
// s = 1 / (1 + 0.3086339 |z|) and q of degree five, fitted for the least
// relative error of Phi(-|z|) over |z| <= 14.5: 4.1e-6, about 1e-5 with the
// rounding of z^2 / 2. So GELU keeps its bf16 digits down to where gauss
// leaves fp32's normal range (z < -13.2: zero, true values below 1e-37).
struct FastTail {
  float s, q, gauss;
};

MOE_DEV FastTail fast_tail(float z, float abs_z) {
  FastTail t;
  t.s = rcp_fast(fmaf(0.30863391f, abs_z, 1.0f));
  t.gauss = ex2_fast(z * z * (-0.5f * kLog2E));
  t.q = fmaf(-0.07501083f, t.s, 0.18683868f);
  t.q = fmaf(t.q, t.s, 0.00985154f);
  t.q = fmaf(t.q, t.s, 0.13559357f);
  t.q = fmaf(t.q, t.s, 0.11936795f);
  t.q = fmaf(t.q, t.s, 0.12335706f);
  return t;
}

// z Phi(z). Fast: max(z, 0) - |z| Phi(-|z|), which needs no choice by sign;
// |z| is held to 15, where gauss is zero, so that infinity meets no zero.
// Else erfc, which keeps its relative precision in the negative tail.
template <bool kFast>
MOE_DEV float gelu_of(float z) {
  if constexpr (kFast) {
    const float abs_z = fminf(fabsf(z), 15.0f);
    const FastTail t = fast_tail(z, abs_z);
    return fmaf(-(abs_z * t.s * t.gauss), t.q, fmaxf(z, 0.0f));
  } else {
    return z * (0.5f * erfcf(-z * 0.70710678118654752f));
  }
}

// Phi(z) + z gauss / sqrt(2 pi), the slope of it.
template <bool kFast>
MOE_DEV float gelu_slope(float z) {
  float phi, gauss;
  if constexpr (kFast) {
    const FastTail t = fast_tail(z, fabsf(z));
    gauss = t.gauss;
    const float tail = t.q * t.s * gauss;
    phi = z < 0.0f ? tail : 1.0f - tail;
  } else {
    gauss = expf(-0.5f * z * z);
    phi = 0.5f * erfcf(-z * 0.70710678118654752f);
  }
  return fmaf(z * 0.3989422804014327f, gauss, phi);
}

template <int kAct, bool kFast>
MOE_DEV float act_value(float z) {
  if constexpr (kAct == MOE_ACT_RELU) {
    return z > 0.0f ? z : (z != z ? z : 0.0f);
  } else if constexpr (kAct == MOE_ACT_GELU) {
    return gelu_of<kFast>(z);
  } else if constexpr (kAct == MOE_ACT_GELU_TANH) {
    return z * gelu_sigmoid<kFast>(z);
  } else if constexpr (kAct == MOE_ACT_SILU) {
    return z * sigmoid_of<kFast>(z);
  } else {
    return z;
  }
}

template <int kAct, bool kFast>
MOE_DEV float slope_value(float z) {
  if constexpr (kAct == MOE_ACT_RELU) {
    return z > 0.0f ? 1.0f : 0.0f;
  } else if constexpr (kAct == MOE_ACT_GELU) {
    return gelu_slope<kFast>(z);
  } else if constexpr (kAct == MOE_ACT_GELU_TANH) {
    const float s = gelu_sigmoid<kFast>(z);
    // far out s - s^2 is zero, and stays zero times a finite du
    const float du = fmaf(fminf(z * z, 1e30f), 6.0f * kGeluTanhC * kGeluTanhA, 2.0f * kGeluTanhC);
    return fmaf(z * fmaf(-s, s, s), du, s);
  } else if constexpr (kAct == MOE_ACT_SILU) {
    const float s = sigmoid_of<kFast>(z);
    return fmaf(z, fmaf(-s, s, s), s);
  } else {
    return 1.0f;
  }
}

// f(Act<kAct>) for the activation `act`: the branch is taken once around f.
template <int kAct>
struct Act {
  static constexpr int value = kAct;
};

template <typename F>
MOE_DEV void with_act(int act, F&& f) {
  switch (act) {
    case MOE_ACT_RELU:
      return f(Act<MOE_ACT_RELU>{});
    case MOE_ACT_GELU:
      return f(Act<MOE_ACT_GELU>{});
    case MOE_ACT_GELU_TANH:
      return f(Act<MOE_ACT_GELU_TANH>{});
    case MOE_ACT_SILU:
      return f(Act<MOE_ACT_SILU>{});
    default:
      return f(Act<MOE_ACT_NONE>{});
  }
}

template <bool kFast>
MOE_DEV float act_of(float z, int act) {
  float v;
  with_act(act, [&](auto k) { v = act_value<decltype(k)::value, kFast>(z); });
  return v;
}

template <bool kFast>
MOE_DEV float act_slope(float z, int act) {
  float v;
  with_act(act, [&](auto k) { v = slope_value<decltype(k)::value, kFast>(z); });
  return v;
}

// ------------------------------------------------------------------ storage types
template <typename T>
MOE_DEV float to_f32(T v);
template <>
MOE_DEV float to_f32<float>(float v) {
  return v;
}
template <>
MOE_DEV float to_f32<__nv_bfloat16>(__nv_bfloat16 v) {
  return __bfloat162float(v);
}
template <typename T>
MOE_DEV T from_f32(float v);
template <>
MOE_DEV float from_f32<float>(float v) {
  return v;
}
template <>
MOE_DEV __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Up to four neighbouring fp32 outputs of rows mode from their sums (`have`
// exist): forward act(sum + bias) + residual (the pre-activation stored first),
// input gradient sum * act'(z) + residual. kVec: all four exist and every
// matrix can be read and written 16 bytes at a time.
template <bool kVec>
MOE_DEV void load_outputs(const float* p, int have, float (&f)[4]) {
  if constexpr (kVec) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = i < have ? p[i] : 0.0f;
  }
}

template <bool kVec>
MOE_DEV void store_outputs(float* p, int have, const float (&f)[4]) {
  if constexpr (kVec) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < have) p[i] = f[i];
  }
}

template <bool kDgrad, bool kVec>
MOE_DEV void finish_outputs(const MatmulArgs& a, float (&f)[4], int e, long long r, int n, int have) {
  float res[4], z[4], b[4];
  if (a.residual != nullptr) load_outputs<kVec>(static_cast<const float*>(a.residual) + r * a.ldr + n, have, res);
  if constexpr (kDgrad) {
    if (a.z != nullptr) {
      load_outputs<kVec>(static_cast<const float*>(a.z) + r * a.ldz + n, have, z);
      with_act(a.act, [&](auto k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] *= slope_value<decltype(k)::value, false>(z[i]);
      });
    }
  } else {
    if (a.bias != nullptr) {
      load_outputs<false>(a.bias + static_cast<size_t>(e) * a.n + n, have, b);
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] += b[i];
    }
    if (a.preact != nullptr) store_outputs<kVec>(static_cast<float*>(a.preact) + r * a.ldz + n, have, f);
    with_act(a.act, [&](auto k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] = act_value<decltype(k)::value, false>(f[i]);
    });
  }
  if (a.residual != nullptr) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] += res[i];
  }
  store_outputs<kVec>(static_cast<float*>(a.d) + r * a.ldd + n, have, f);
}

}  // namespace moe
