// moe_dropout: y = residual + dropout(x) over a matrix, the mask drawn where
// it is used (dropout.cuh).
//
// Bound: HBM (x and the residual read, y written, once each). The generator
// costs about ten integer multiplies and twenty logic operations for four
// elements, under half of the time that their bytes take. Each thread owns
// 16-byte vectors one grid apart and starts the loads of several before it
// draws any word, so the integer work runs under the loads' latency.
#include "dropout.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Row16;  // 16 bytes of a row as floats

template <>
struct Row16<__nv_bfloat16> {
  static constexpr int N = 8;
  MOE_DEV static void load(const uint4& q, float* f) {
    const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&q);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 x = __bfloat1622float2(p[i]);
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
  MOE_DEV static uint4 store(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  MOE_DEV static float one(const __nv_bfloat16* p) { return __bfloat162float(*p); }
  MOE_DEV static void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
};

template <>
struct Row16<float> {
  static constexpr int N = 4;
  MOE_DEV static void load(const uint4& q, float* f) {
    f[0] = __uint_as_float(q.x);
    f[1] = __uint_as_float(q.y);
    f[2] = __uint_as_float(q.z);
    f[3] = __uint_as_float(q.w);
  }
  MOE_DEV static uint4 store(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
  MOE_DEV static float one(const float* p) { return *p; }
  MOE_DEV static void put(float* p, float v) { *p = v; }
};

struct Matrices {
  const void *x, *residual;
  void* y;
  long long ldx, ldr, ldy;
  int rows, cols;
  int vpr;                 // units (vectors or quads) a row
  int step_rows, step_units;  // one grid of units = step_rows rows and step_units units
};

// Rows that are whole 16-byte vectors on 16-byte boundaries.
template <typename T, bool kDrop, bool kResidual>
__global__ void __launch_bounds__(kThreads) dropout_vec_kernel(const Matrices m, const DropoutArgs d) {
  using V = Row16<T>;
  constexpr int U = 4;
  const long long first = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  long long r = first / m.vpr;
  int u = static_cast<int>(first - r * m.vpr);
  DropoutState s{};
  if constexpr (kDrop) s = dropout_state(d);
  while (r < m.rows) {
    long long rr[U];
    int uu[U];
    uint4 qx[U], qr[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      rr[i] = r;
      uu[i] = u;
      if (r < m.rows) {
        qx[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(m.x) + r * m.ldx) + u);
        if constexpr (kResidual)
          qr[i] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const T*>(m.residual) + r * m.ldr) + u);
      }
      r += m.step_rows;
      u += m.step_units;
      if (u >= m.vpr) {
        u -= m.vpr;
        ++r;
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (rr[i] >= m.rows) break;
      float f[V::N];
      V::load(qx[i], f);
      if constexpr (kDrop) {
#pragma unroll
        for (int j = 0; j < V::N / 4; ++j)
          dropout_quad(d, s, static_cast<uint32_t>(uu[i]) * (V::N / 4) + j, static_cast<uint32_t>(rr[i]), f + 4 * j);
      }
      if constexpr (kResidual) {
        float g[V::N];
        V::load(qr[i], g);
#pragma unroll
        for (int j = 0; j < V::N; ++j) f[j] += g[j];
      }
      __stcs(reinterpret_cast<uint4*>(static_cast<T*>(m.y) + rr[i] * m.ldy) + uu[i], V::store(f));
    }
  }
}

// Any width and stride: four columns (one block of the generator) a step.
template <typename T, bool kDrop, bool kResidual>
__global__ void __launch_bounds__(kThreads) dropout_any_kernel(const Matrices m, const DropoutArgs d) {
  const long long first = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  long long r = first / m.vpr;
  int u = static_cast<int>(first - r * m.vpr);
  DropoutState s{};
  if constexpr (kDrop) s = dropout_state(d);
  while (r < m.rows) {
    const int c = u * 4, have = min(4, m.cols - c);
    const T* px = static_cast<const T*>(m.x) + r * m.ldx + c;
    T* py = static_cast<T*>(m.y) + r * m.ldy + c;
    float f[4], g[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = j < have ? Row16<T>::one(px + j) : 0.f;
    if constexpr (kResidual) {
      const T* pr = static_cast<const T*>(m.residual) + r * m.ldr + c;
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = j < have ? Row16<T>::one(pr + j) : 0.f;
    }
    if constexpr (kDrop) dropout_quad(d, s, static_cast<uint32_t>(u), static_cast<uint32_t>(r), f);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < have) Row16<T>::put(py + j, f[j] + g[j]);
    r += m.step_rows;
    u += m.step_units;
    if (u >= m.vpr) {
      u -= m.vpr;
      ++r;
    }
  }
}

template <typename T, bool kDrop, bool kResidual>
cudaError_t launch_typed(Matrices m, const DropoutArgs& d, cudaStream_t s) {
  constexpr int N = Row16<T>::N;
  const bool vec = m.cols % N == 0 && m.ldx % N == 0 && m.ldy % N == 0 && (!kResidual || m.ldr % N == 0);
  m.vpr = vec ? m.cols / N : (m.cols + 3) / 4;
  const long long units = static_cast<long long>(m.rows) * m.vpr;
  const long long per_block = static_cast<long long>(kThreads) * (vec ? 4 : 1);
  const unsigned grid =
      static_cast<unsigned>(std::max(1LL, std::min((units + per_block - 1) / per_block, device_sm_count() * 8LL)));
  const long long step = static_cast<long long>(grid) * kThreads;
  m.step_rows = static_cast<int>(step / m.vpr);
  m.step_units = static_cast<int>(step % m.vpr);
  return vec ? launch_kernel(dropout_vec_kernel<T, kDrop, kResidual>, dim3(grid), dim3(kThreads), 0, s, false, 1, m, d)
             : launch_kernel(dropout_any_kernel<T, kDrop, kResidual>, dim3(grid), dim3(kThreads), 0, s, false, 1, m, d);
}

template <typename T>
cudaError_t launch_of(const Matrices& m, const DropoutArgs& d, cudaStream_t s) {
  if (d.cut == 0) return m.residual ? launch_typed<T, false, true>(m, d, s) : launch_typed<T, false, false>(m, d, s);
  return m.residual ? launch_typed<T, true, true>(m, d, s) : launch_typed<T, true, false>(m, d, s);
}

}  // namespace

cudaError_t launch_dropout(int dtype, int rows, int cols, const void* x, long long ldx, const void* residual,
                           long long ldr, void* y, long long ldy, const DropoutArgs& d, cudaStream_t s) {
  const Matrices m{x, residual, y, ldx, ldr, ldy, rows, cols, 0, 0, 0};
  return dtype == MOE_DTYPE_F32 ? launch_of<float>(m, d, s) : launch_of<__nv_bfloat16>(m, d, s);
}

}  // namespace moe
