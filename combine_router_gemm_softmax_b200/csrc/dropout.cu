// moe_dropout: y = residual + dropout(x) over a matrix, the mask drawn where
// it is used (dropout.cuh).
//
// Bound: HBM (x and the residual read, y written, once each), with the
// generator's integer work close behind: a thread keeps one column of 16-byte
// vectors and walks down its rows, so that what the generator does to the
// column is done once (15 instead of 20 products a block of four words), and
// starts the loads of several rows before it draws any word.
#include "dropout.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
// Rows of a thread in flight, and CTAs an SM (32768 x 4096 bf16 with a
// residual, 805 MB: 134.8 us; 2 rows at 4 CTAs 140.2, 4 at 3 147.7, 1 at 8
// 135.7, 2 at 5, where registers spill, 170.6).
constexpr int kDropRows = 2;
constexpr int kDropCtas = 3;

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
  int vpr;        // units (vectors or quads) a row
  int step_rows;  // rows from a thread's unit to its next
};

// Rows that are whole 16-byte vectors on 16-byte boundaries.
template <typename T, bool kDrop, bool kResidual>
__global__ void __launch_bounds__(kThreads, kDropCtas) dropout_vec_kernel(const Matrices m, const DropoutArgs d) {
  using V = Row16<T>;
  constexpr int U = kDropRows, Q = V::N / 4;
  const unsigned first = blockIdx.x * kThreads + threadIdx.x;
  const int u = first % m.vpr;
  long long r = first / m.vpr;
  pdl_wait();
  if (r >= m.step_rows) return;  // the grid's remainder
  DropoutState s{};
  DropoutColumn col[Q];
  if constexpr (kDrop) {
    s = dropout_state(d);
#pragma unroll
    for (int j = 0; j < Q; ++j) col[j] = dropout_column(s, static_cast<uint32_t>(u) * Q + j);
  }
  const T* px = static_cast<const T*>(m.x) + u * V::N;
  const T* pr = static_cast<const T*>(m.residual) + u * V::N;
  T* py = static_cast<T*>(m.y) + u * V::N;
  for (; r < m.rows; r += static_cast<long long>(U) * m.step_rows) {
    uint4 qx[U], qr[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const long long ri = r + static_cast<long long>(i) * m.step_rows;
      if (ri < m.rows) {
        qx[i] = __ldcs(reinterpret_cast<const uint4*>(px + ri * m.ldx));
        if constexpr (kResidual) qr[i] = __ldcs(reinterpret_cast<const uint4*>(pr + ri * m.ldr));
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const long long ri = r + static_cast<long long>(i) * m.step_rows;
      if (ri >= m.rows) break;
      float f[V::N];
      V::load(qx[i], f);
      float g[V::N] = {};
      if constexpr (kResidual) V::load(qr[i], g);
      if constexpr (kDrop) {
        const DropoutRow row = dropout_row(s, static_cast<uint32_t>(ri));
#pragma unroll
        for (int j = 0; j < Q; ++j) dropout_quad(d, s, col[j], row, f + 4 * j, g + 4 * j);
      } else {
#pragma unroll
        for (int j = 0; j < V::N; ++j) f[j] += g[j];
      }
      __stcs(reinterpret_cast<uint4*>(py + ri * m.ldy), V::store(f));
    }
  }
}

// Any width and stride: four columns (one block of the generator) a step.
template <typename T, bool kDrop, bool kResidual>
__global__ void __launch_bounds__(kThreads) dropout_any_kernel(const Matrices m, const DropoutArgs d) {
  const unsigned first = blockIdx.x * kThreads + threadIdx.x;
  const int u = first % m.vpr;
  long long r = first / m.vpr;
  pdl_wait();
  if (r >= m.step_rows) return;
  DropoutState s{};
  DropoutColumn col{};
  if constexpr (kDrop) {
    s = dropout_state(d);
    col = dropout_column(s, static_cast<uint32_t>(u));
  }
  const int c = u * 4, have = min(4, m.cols - c);
  for (; r < m.rows; r += m.step_rows) {
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
    if constexpr (kDrop) {
      dropout_quad(d, s, col, dropout_row(s, static_cast<uint32_t>(r)), f, g);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] += g[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < have) Row16<T>::put(py + j, f[j]);
  }
}

template <typename T, bool kDrop, bool kResidual>
cudaError_t launch_typed(Matrices m, const DropoutArgs& d, cudaStream_t s) {
  constexpr int N = Row16<T>::N;
  const bool vec = m.cols % N == 0 && m.ldx % N == 0 && m.ldy % N == 0 && (!kResidual || m.ldr % N == 0);
  m.vpr = vec ? m.cols / N : static_cast<int>((m.cols + 3LL) / 4);  // up to 2^31 - 1 columns
  // Threads for a whole number of rows: every thread keeps its column. Enough
  // for a row at least, and no more than fill the SMs.
  const long long units = static_cast<long long>(m.rows) * m.vpr;
  const long long per_block = static_cast<long long>(kThreads) * (vec ? kDropRows : 1);
  long long grid = std::min((units + per_block - 1) / per_block, device_sm_count() * 8LL);
  grid = std::max(grid, (m.vpr + kThreads - 1LL) / kThreads);
  m.step_rows = static_cast<int>(grid * kThreads / m.vpr);
  const dim3 blocks(static_cast<unsigned>(grid));
  return vec ? launch_kernel(dropout_vec_kernel<T, kDrop, kResidual>, blocks, dim3(kThreads), 0, s, true, 1, m, d)
             : launch_kernel(dropout_any_kernel<T, kDrop, kResidual>, blocks, dim3(kThreads), 0, s, true, 1, m, d);
}

template <typename T>
cudaError_t launch_of(const Matrices& m, const DropoutArgs& d, cudaStream_t s) {
  if (d.cut == 0) return m.residual ? launch_typed<T, false, true>(m, d, s) : launch_typed<T, false, false>(m, d, s);
  return m.residual ? launch_typed<T, true, true>(m, d, s) : launch_typed<T, true, false>(m, d, s);
}

// Which of a 16-byte vector's elements are kept, a bit each.
template <int N>
MOE_DEV uint32_t keep_bits(const DropoutArgs& d, const DropoutState& s, uint32_t v, const DropoutRow& row) {
  uint32_t bits = 0;
#pragma unroll
  for (int j = 0; j < N / 4; ++j) {
    const uint4 w = dropout_words(s, dropout_column(s, v * (N / 4) + j), row);
    bits |= ((w.x >= d.cut ? 1u : 0u) | (w.y >= d.cut ? 2u : 0u) | (w.z >= d.cut ? 4u : 0u) | (w.w >= d.cut ? 8u : 0u))
            << (4 * j);
  }
  return bits;
}

// 16-byte vectors of a row that a lane has in flight, by the rows it adds up:
// 8 to 12 loads, the residual's among them, at three CTAs an SM (45.5 us on the
// case below; up to 16 loads at two CTAs 51.8, one vector at four 70.4).
constexpr int combine_vectors(int rows) { return rows <= 2 ? 4 : rows <= 6 ? 2 : 1; }

// One token from its NK kept rows, in slot order: the loads of U vectors a
// lane go out first, the mask is drawn while they are under way (in a loop, so
// that the generator's code is there once: unrolled over the vectors it ran
// out of the instruction cache), then the sums.
template <typename T, int NK, int K>
MOE_DEV void combine_token(const uint4* __restrict__ y_perm, const int (&dst)[K], const float (&g)[K],
                           const uint4* residual, uint4* y, int vpr, int lane, const DropoutArgs& d,
                           const DropoutState& s, const DropoutRow& row) {
  using V = Row16<T>;
  constexpr int U = combine_vectors(NK);
  static_assert(U * V::N <= 32, "a bit each");
  for (int v0 = lane; v0 < vpr; v0 += 32 * U) {
    uint4 q[NK > 0 ? NK : 1][U], qr[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int v = v0 + u * 32;
#pragma unroll
      for (int j = 0; j < NK; ++j)
        q[j][u] = v < vpr ? __ldg(y_perm + static_cast<size_t>(dst[j]) * vpr + v) : make_uint4(0, 0, 0, 0);
      qr[u] = residual != nullptr && v < vpr ? __ldcs(residual + v) : make_uint4(0, 0, 0, 0);
    }
    uint32_t keep = 0xffffffffu;
    if (d.cut != 0) {
      keep = 0;
#pragma unroll 1
      for (int u = 0; u < U; ++u) keep |= keep_bits<V::N>(d, s, v0 + u * 32, row) << (V::N * u);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float acc[V::N] = {}, f[V::N];
#pragma unroll
      for (int j = 0; j < NK; ++j) {
        V::load(q[j][u], f);
#pragma unroll
        for (int i = 0; i < V::N; ++i) acc[i] = fmaf(g[j], f[i], acc[i]);
      }
      V::load(qr[u], f);
#pragma unroll
      for (int i = 0; i < V::N; ++i) {
        const float kept = (keep >> (V::N * u + i)) & 1u ? acc[i] : 0.0f;
        acc[i] = residual != nullptr ? fmaf(kept, d.scale, f[i]) : kept * d.scale;
      }
      const int v = v0 + u * 32;
      if (v < vpr) y[v] = V::store(acc);
    }
  }
}

// moe_unpermute_combine_dropout: one warp a token, its kept slots listed first
// (in slot order). Bound: HBM (the kept rows and the residual read, y written);
// 16384 tokens of 2048 under a capacity that keeps 27 thousand of 98 thousand
// assignments: 247 MB.
template <typename T, int K>
__global__ void __launch_bounds__(kThreads, 3)
    combine_dropout_kernel(const uint4* __restrict__ y_perm, const int32_t* __restrict__ dest_row,
                           const float* __restrict__ gate, const uint4* residual, uint4* y, int tokens, int rows,
                           int vpr, const DropoutArgs d) {
  const int lane = threadIdx.x & 31;
  pdl_wait();
  DropoutState s{};
  if (d.cut != 0) s = dropout_state(d);
  for (int t = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); t < tokens; t += gridDim.x * (kThreads / 32)) {
    const int my_dest = lane < K ? dest_row[static_cast<size_t>(t) * K + lane] : -1;
    const float my_gate = lane < K ? gate[static_cast<size_t>(t) * K + lane] : 0.f;
    uint32_t rest = __ballot_sync(0xffffffffu, my_dest >= 0 && my_dest < rows);
    const int kept = __popc(rest);
    int dst[K];
    float g[K];
#pragma unroll
    for (int j = 0; j < K; ++j) {
      const int from = rest ? __ffs(rest) - 1 : 0;
      rest &= rest - 1;
      dst[j] = __shfl_sync(0xffffffffu, my_dest, from);
      g[j] = __shfl_sync(0xffffffffu, my_gate, from);
    }
    const DropoutRow row = dropout_row(s, static_cast<uint32_t>(t));
    const size_t at = static_cast<size_t>(t) * vpr;
    const uint4* res = residual != nullptr ? residual + at : nullptr;
    switch (kept) {
#define MOE_COMBINE_NK(NK)                                                                           \
  case NK:                                                                                           \
    if constexpr (NK <= K) combine_token<T, NK, K>(y_perm, dst, g, res, y + at, vpr, lane, d, s, row); \
    break;
      MOE_COMBINE_NK(0)
      MOE_COMBINE_NK(1)
      MOE_COMBINE_NK(2)
      MOE_COMBINE_NK(3)
      MOE_COMBINE_NK(4)
      MOE_COMBINE_NK(5)
      MOE_COMBINE_NK(6)
      MOE_COMBINE_NK(7)
      MOE_COMBINE_NK(8)
#undef MOE_COMBINE_NK
      default:
        break;
    }
  }
}

template <typename T, int K>
cudaError_t launch_combine_k(const uint4* y_perm, const int32_t* dest_row, const float* gate, const uint4* residual,
                             uint4* y, int tokens, int rows, int k, int vpr, const DropoutArgs& d, cudaStream_t s) {
  if constexpr (K < kMaxK) {
    if (k > K) return launch_combine_k<T, K + 1>(y_perm, dest_row, gate, residual, y, tokens, rows, k, vpr, d, s);
  }
  const long long grid = std::min<long long>((tokens + 7LL) / 8, device_sm_count() * 8LL);
  return launch_kernel(combine_dropout_kernel<T, K>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, true, 1,
                       y_perm, dest_row, gate, residual, y, tokens, rows, vpr, d);
}

}  // namespace

cudaError_t launch_combine_dropout(int dtype, const void* y_perm, int rows, const int32_t* dest_row,
                                   const float* gate, const void* residual, const DropoutArgs& drop, void* y, int T, int k, int d,
                                   cudaStream_t s) {
  if (T == 0) return cudaSuccess;
  const uint4* src = static_cast<const uint4*>(y_perm);
  const uint4* res = static_cast<const uint4*>(residual);
  uint4* out = static_cast<uint4*>(y);
  if (dtype == MOE_DTYPE_F32)
    return launch_combine_k<float, 1>(src, dest_row, gate, res, out, T, rows, k, d / 4, drop, s);
  return launch_combine_k<__nv_bfloat16, 1>(src, dest_row, gate, res, out, T, rows, k, d / 8, drop, s);
}

cudaError_t launch_dropout(int dtype, int rows, int cols, const void* x, long long ldx, const void* residual,
                           long long ldr, void* y, long long ldy, const DropoutArgs& d, cudaStream_t s) {
  const Matrices m{x, residual, y, ldx, ldr, ldy, rows, cols, 0, 0};
  return dtype == MOE_DTYPE_F32 ? launch_of<float>(m, d, s) : launch_of<__nv_bfloat16>(m, d, s);
}

}  // namespace moe
