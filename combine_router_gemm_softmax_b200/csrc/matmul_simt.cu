// The free products in fp32 (moe_grouped_gemm, moe_linear and their
// gradients with dtype MOE_DTYPE_F32), on the CUDA cores: products and sums
// stay IEEE fp32, which the tensor cores' reduced input formats would not.
//
// A CTA of 256 threads owns a tile of BT x BT outputs (BT 128 or 64), each
// thread (BT/16)^2 of them in registers as pairs along n, so that one packed
// fma.rn.f32x2 does two multiply-adds. Slices of 16 along the reduction pass
// through two shared-memory buffers, one barrier a slice; the next slices are
// under way in registers (one for 128-wide tiles, whose slice takes a
// microsecond of arithmetic, four for 64-wide ones, whose slice takes a
// quarter of the load latency). Operands are read as they lie: along the
// reduction or across it, by template, so no mode needs a transposed copy.
// Bound: the fp32 pipe (128 multiply-adds a cycle and SM, about 70 TFLOP/s) for
// 128-wide tiles (4099 x 1408 x 2048: forward 592 us, 40 TFLOP/s, dgrad 43,
// wgrad 30, whose 176 tiles leave a part of the SMs one instead of two); for
// 64-wide ones the shared-memory loads, two of 16 bytes for a thread's
// eight packed multiply-adds (333 x 768 x 1000: 26.8 us, L1 73% busy, the fp32
// pipe 22%).
//
// Few tiles leave SMs idle, so a cluster of S CTAs can share one 64 x 64 tile:
// each takes a part of the reduction, and the partial tiles are added through
// distributed shared memory in the order of the CTAs' ranks (the same sum on
// every run).
#include "matmul_common.cuh"

namespace moe {
namespace {

constexpr int kBK = 16;
constexpr int kThreads = 256;

struct Quad {
  float v[4];
};

// Four elements from p, `valid` of them inside the row (the others zero).
// kVec: the row's width is a multiple of four and it starts on four elements'
// alignment, so that all four exist or none; one load under one predicate.
template <typename T, bool kVec>
MOE_DEV Quad load4(const T* p, int valid) {
  Quad q{};
  if constexpr (kVec) {
    if (valid > 0) {
      if constexpr (sizeof(T) == 4) {
        const float4 f = *reinterpret_cast<const float4*>(p);
        q.v[0] = f.x, q.v[1] = f.y, q.v[2] = f.z, q.v[3] = f.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(p);
        const float2 lo = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.x));
        const float2 hi = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u.y));
        q.v[0] = lo.x, q.v[1] = lo.y, q.v[2] = hi.x, q.v[3] = hi.y;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < valid) q.v[j] = to_f32(p[j]);
  }
  return q;
}

// One operand's slice of BT (rows of the tile) x 16 (reduction), in registers.
// kAlong: elements lie along the reduction (row-major tile rows); else across.
template <bool kAlong, bool kVec, int BT>
struct Slice {
  static constexpr int kQuads = BT * kBK / 4 / kThreads;
  Quad q[kQuads];

  // base: element (first row of the tile, reduction index 0); rows and
  // depth: what of the tile and of the reduction [k0, ...) exists.
  MOE_DEV void load(const float* base, long long ld, int rows, int k0, int depth) {
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const int id = threadIdx.x + i * kThreads;
      if constexpr (kAlong) {
        const int r = id >> 2, k = k0 + (id & 3) * 4;
        q[i] = load4<float, kVec>(base + r * ld + k, r < rows ? depth - k : 0);
      } else {
        const int k = k0 + id / (BT / 4), r = (id % (BT / 4)) * 4;
        q[i] = load4<float, kVec>(base + k * ld + r, k < depth ? rows - r : 0);
      }
    }
  }

  MOE_DEV void store(float (*s)[BT + 4]) const {
#pragma unroll
    for (int i = 0; i < kQuads; ++i) {
      const int id = threadIdx.x + i * kThreads;
      if constexpr (kAlong) {
        const int r = id >> 2, k = (id & 3) * 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) s[k + j][r] = q[i].v[j];
      } else {
        const int k = id / (BT / 4), r = (id % (BT / 4)) * 4;
        *reinterpret_cast<float4*>(&s[k][r]) = make_float4(q[i].v[0], q[i].v[1], q[i].v[2], q[i].v[3]);
      }
    }
  }
};

MOE_DEV uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

MOE_DEV void fma2(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

MOE_DEV float2 unpack2(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}

// BT x BT outputs of a thread grid of 16 x 16: row i of thread ty is
// (i / 4) * (BT / 2) + ty * 4 + i % 4 for BT 128 (two groups of four), ty * 4 + i for 64.
template <int BT>
MOE_DEV int at(int t, int i) {
  return BT == 128 ? (i >> 2) * 64 + t * 4 + (i & 3) : t * 4 + i;
}

template <MatmulMode kMode, bool kVec, int BT>
__global__ void __launch_bounds__(kThreads, BT == 128 ? 2 : 3) matmul_simt_kernel(const MatmulArgs a) {
  constexpr int kPer = BT / 16;  // outputs of a thread along each axis
  constexpr bool kWeight = kMode == MatmulMode::kWgrad;
  __shared__ __align__(16) float sA[2][kBK][BT + 4];
  __shared__ __align__(16) float sB[2][kBK][BT + 4];
  __shared__ int2 s_rows[kMaxE];
  __shared__ int prefix[kMaxE + 1];
  // a partial tile for the sum over the cluster (64 x 64 only)
  __shared__ __align__(16) float s_part[BT == 64 ? 64 * 64 : 4];

  uint32_t split, part;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
  part = split > 1 ? cluster_ctarank() : 0;
  pdl_wait();
  if (threadIdx.x < 32)
    build_groups(a.offsets, a.groups, a.rows, BT == 128 ? 7 : 6, s_rows, prefix, a.status, threadIdx.x);
  __syncthreads();
  const int tiles_n = (a.n + BT - 1) / BT;
  const int tiles_m = kWeight ? (a.m + BT - 1) / BT : prefix[a.groups];
  const long long total = static_cast<long long>(tiles_n) * tiles_m * (kWeight ? a.groups : 1);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;

  for (long long tile = blockIdx.x / split; tile < total; tile += gridDim.x / split) {
    const int tn = static_cast<int>(tile % tiles_n);
    const long long rest = tile / tiles_n;
    int e, m0, m_valid, depth, k_first = 0;
    const int n0 = tn * BT, n_valid = min(BT, a.n - n0);
    const float* pa;
    const float* pb;
    if constexpr (kWeight) {
      e = static_cast<int>(rest / tiles_m);
      m0 = static_cast<int>(rest % tiles_m) * BT;
      m_valid = min(BT, a.m - m0);
      depth = s_rows[e].y - s_rows[e].x;
      pa = static_cast<const float*>(a.a) + s_rows[e].x * a.lda + m0;
      pb = static_cast<const float*>(a.b) + s_rows[e].x * a.ldb + n0;
    } else {
      e = group_of_tile(prefix, a.groups, static_cast<int>(rest));
      m0 = s_rows[e].x + (static_cast<int>(rest) - prefix[e]) * BT;
      m_valid = min(BT, s_rows[e].y - m0);
      depth = a.k;
      pa = static_cast<const float*>(a.a) + m0 * a.lda;
      pb = static_cast<const float*>(a.b) + e * a.b_stride + (kMode == MatmulMode::kForward ? n0 * a.ldb : n0);
    }
    if (split > 1) {
      const int slices = (depth + kBK - 1) / kBK;
      k_first = static_cast<int>(static_cast<long long>(slices) * part / split) * kBK;
      depth = min(depth, static_cast<int>(static_cast<long long>(slices) * (part + 1) / split) * kBK);
    }

    uint64_t acc[kPer][kPer / 2];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
#pragma unroll
      for (int j = 0; j < kPer / 2; ++j) acc[i][j] = 0;

    constexpr int kAhead = BT == 128 ? 1 : 4;  // slices in registers
    Slice<!kWeight, kVec, BT> qa[kAhead];
    Slice<kMode == MatmulMode::kForward, kVec, BT> qb[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      qa[i].load(pa, a.lda, m_valid, k_first + i * kBK, depth);
      qb[i].load(pb, a.ldb, n_valid, k_first + i * kBK, depth);
    }
    int buf = 0;
    for (int k1 = k_first; k1 < depth; k1 += kAhead * kBK) {
#pragma unroll
      for (int s = 0; s < kAhead; ++s) {
        const int k0 = k1 + s * kBK;
        if (k0 >= depth) break;
        qa[s].store(sA[buf]);
        qb[s].store(sB[buf]);
        __syncthreads();  // also: everyone is done with the other buffer
        qa[s].load(pa, a.lda, m_valid, k0 + kAhead * kBK, depth);
        qb[s].load(pb, a.ldb, n_valid, k0 + kAhead * kBK, depth);
#pragma unroll(BT == 128 ? 16 : 8)
        for (int k = 0; k < kBK; ++k) {
          float ra[kPer];
          uint64_t rb[kPer / 2];
#pragma unroll
          for (int g = 0; g < kPer / 4; ++g) {
            const float4 f = *reinterpret_cast<const float4*>(&sA[buf][k][at<BT>(ty, g * 4)]);
            ra[4 * g] = f.x, ra[4 * g + 1] = f.y, ra[4 * g + 2] = f.z, ra[4 * g + 3] = f.w;
            const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(&sB[buf][k][at<BT>(tx, g * 4)]);
            rb[2 * g] = u.x, rb[2 * g + 1] = u.y;
          }
#pragma unroll
          for (int i = 0; i < kPer; ++i) {
            const uint64_t d = pack2(ra[i], ra[i]);
#pragma unroll
            for (int j = 0; j < kPer / 2; ++j) fma2(acc[i][j], d, rb[j]);
          }
        }
        buf ^= 1;
      }
    }
    __syncthreads();  // before the next tile's slices overwrite a buffer

    // four neighbouring outputs of the tile: row i, columns j ..
    auto finish = [&](int i, int j, float(&f)[4]) {
      const int have = n_valid - j;
      if (i >= m_valid || have <= 0) return;
      if constexpr (kWeight) {
        float* d = static_cast<float*>(a.d) + (static_cast<long long>(e) * a.m + m0 + i) * a.ldd + n0 + j;
        if (have >= 4 && a.vec_out)
          store_outputs<true>(d, 4, f);
        else
          store_outputs<false>(d, have, f);
      } else if (have >= 4 && a.vec_out) {
        finish_outputs<kMode == MatmulMode::kDgrad, true>(a, f, e, m0 + i, n0 + j, 4);
      } else {
        finish_outputs<kMode == MatmulMode::kDgrad, false>(a, f, e, m0 + i, n0 + j, have);
      }
    };
    if constexpr (BT == 64) {
      // Through shared memory: the tile's rows are finished whole by neighbouring
      // threads in a short loop (unrolled over a thread's own outputs, the
      // activations' code outlasted a small product). With a split, the partial
      // tiles lie side by side in the cluster's shared memory, and each CTA adds
      // and finishes its share of the rows.
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int j = 0; j < kPer / 2; ++j)
          *reinterpret_cast<float2*>(&s_part[at<BT>(ty, i) * 64 + at<BT>(tx, 2 * j)]) = unpack2(acc[i][j]);
      if (split > 1)
        cluster_sync();
      else
        __syncthreads();
      const uint32_t mine = smem_addr(s_part);
      const int first = 64 * 64 / 4 * part / split, last = 64 * 64 / 4 * (part + 1) / split;
#pragma unroll 1
      for (int q = first + threadIdx.x; q < last; q += kThreads) {
        float f[4] = {0.f, 0.f, 0.f, 0.f};
        if (split > 1) {
          for (uint32_t c = 0; c < split; ++c) {
            float g[4];
            ld_shared_cluster_v4(mapa_shared(mine + q * 16, c), g);
#pragma unroll
            for (int x = 0; x < 4; ++x) f[x] += g[x];
          }
        } else {
          const float4 g = *reinterpret_cast<const float4*>(&s_part[q * 4]);
          f[0] = g.x, f[1] = g.y, f[2] = g.z, f[3] = g.w;
        }
        finish(q >> 4, (q & 15) * 4, f);
      }
      // nobody overwrites or leaves while somebody still reads
      if (split > 1)
        cluster_sync();
      else
        __syncthreads();
    } else {
#pragma unroll
      for (int i = 0; i < kPer; ++i)
#pragma unroll
        for (int g = 0; g < kPer / 4; ++g) {
          const float2 lo = unpack2(acc[i][2 * g]), hi = unpack2(acc[i][2 * g + 1]);
          float f[4] = {lo.x, lo.y, hi.x, hi.y};
          finish(at<BT>(ty, i), at<BT>(tx, 4 * g), f);
        }
    }
  }
}

template <MatmulMode kMode, bool kVec>
cudaError_t launch_tiles(const MatmulPlan& plan, const MatmulArgs& a, int sms, cudaStream_t s) {
  if (plan.bn == 128)
    return launch_kernel(matmul_simt_kernel<kMode, kVec, 128>,
                         dim3(static_cast<unsigned>(std::min<long long>(plan.tiles, 2 * sms))), dim3(kThreads), 0, s, true,
                         1, a);
  const long long grid = std::min<long long>(plan.tiles, 3 * sms) * plan.split;
  return launch_kernel(matmul_simt_kernel<kMode, kVec, 64>, dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, true,
                       static_cast<unsigned>(plan.split), a);
}

template <MatmulMode kMode>
cudaError_t launch_mode(const MatmulPlan& plan, const MatmulArgs& a, int sms, cudaStream_t s) {
  return a.vec ? launch_tiles<kMode, true>(plan, a, sms, s) : launch_tiles<kMode, false>(plan, a, sms, s);
}

}  // namespace

MatmulPlan plan_matmul_f32(MatmulMode mode, const MatmulArgs& a, int sms) {
  // no more than these row tiles exist, however the rows fall to the groups
  auto tiles = [&](long long bt) {
    const long long tn = (a.n + bt - 1) / bt;
    const long long tm = mode == MatmulMode::kWgrad ? static_cast<long long>(a.groups) * ((a.m + bt - 1) / bt)
                                                    : a.rows / bt + a.groups;
    return tm * tn;
  };
  if (tiles(128) >= sms) return {Form::kSingle, 128, 1, tiles(128)};
  const long long t = tiles(64);
  const int depth = mode == MatmulMode::kWgrad ? a.rows : a.k;
  int split = 1;
  while (split < 8 && t * split * 2 <= 3 * sms && depth / (split * 2) >= 64) split *= 2;
  return {split > 1 ? Form::kSplit : Form::kSingle, 64, split, t};
}

cudaError_t launch_matmul_f32(MatmulMode mode, const MatmulPlan& plan, const MatmulArgs& a, int sms, cudaStream_t s) {
  switch (mode) {
    case MatmulMode::kForward:
      return launch_mode<MatmulMode::kForward>(plan, a, sms, s);
    case MatmulMode::kDgrad:
      return launch_mode<MatmulMode::kDgrad>(plan, a, sms, s);
    default:
      return launch_mode<MatmulMode::kWgrad>(plan, a, sms, s);
  }
}

// ------------------------------------------------------------------ bias gradient
// db[e, n] = sum of dy[r, n] over group e's rows. A CTA's 16 warps take 128
// columns (four a lane) and every 16th row, eight rows in flight each (two
// CTAs an SM; 16 rows in flight leave room for one, and 134 MB took 79 us
// instead of 31); the cluster's CTAs share the rows, and their sums meet in
// distributed shared memory in rank order. Bound: HBM (dy read once). status
// (or NULL, when a product of the same call looks the offsets over) receives
// MOE_STATUS_BAD_OFFSETS from the first CTA's first warp.
namespace {

constexpr int kSumWarps = 16, kSumRows = 8;

template <typename T, bool kVec>
__global__ void __launch_bounds__(32 * kSumWarps) column_sum_kernel(const T* dy, long long ld, const int32_t* offsets,
                                                                    int rows, int n, float* out, int groups,
                                                                    int32_t* status) {
  __shared__ __align__(16) float s_sum[kSumWarps][128];
  uint32_t split, part;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
  part = split > 1 ? cluster_ctarank() : 0;
  const int e = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n0 = static_cast<int>(blockIdx.x / split) * 128;
  pdl_wait();
  if (status != nullptr && (blockIdx.x | blockIdx.y | warp) == 0) {
    bool bad = false;
    for (int i = lane; i < groups; i += 32) group_rows(offsets, i, rows, &bad);
    if (bad) report_status(status, MOE_STATUS_BAD_OFFSETS);
  }
  const int2 g = group_rows(offsets, e, rows);
  const long long have = g.y - g.x;
  const int r0 = g.x + static_cast<int>(have * part / split), r1 = g.x + static_cast<int>(have * (part + 1) / split);
  const int c = n0 + lane * 4;
  const T* p = dy + c;
  float s[4] = {0.f, 0.f, 0.f, 0.f};
  for (int r = r0 + warp; r < r1; r += kSumRows * kSumWarps) {
    Quad q[kSumRows];
#pragma unroll
    for (int i = 0; i < kSumRows; ++i)
      q[i] = load4<T, kVec>(p + static_cast<long long>(r + i * kSumWarps) * ld, r + i * kSumWarps < r1 ? n - c : 0);
#pragma unroll
    for (int i = 0; i < kSumRows; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += q[i].v[j];
  }
  *reinterpret_cast<float4*>(&s_sum[warp][lane * 4]) = make_float4(s[0], s[1], s[2], s[3]);
  __syncthreads();
  if (threadIdx.x < 128) {
    float t = 0.f;
#pragma unroll
    for (int w = 0; w < kSumWarps; ++w) t += s_sum[w][threadIdx.x];
    s_sum[0][threadIdx.x] = t;
  }
  if (split > 1) cluster_sync();
  if (part == 0 && threadIdx.x < 128 && n0 + static_cast<int>(threadIdx.x) < n) {
    float t = s_sum[0][threadIdx.x];
    for (uint32_t k = 1; k < split; ++k) t += ld_shared_cluster_f32(mapa_shared(smem_addr(&s_sum[0][threadIdx.x]), k));
    out[static_cast<size_t>(e) * n + n0 + threadIdx.x] = t;
  }
  if (split > 1) cluster_sync();
}

template <typename T>
cudaError_t column_sums(const void* dy, long long ld, const int32_t* offsets, int groups, int rows, int n, float* out,
                        int32_t* status, bool vec, cudaStream_t s) {
  const int blocks = (n + 127) / 128;
  int split = 1;
  while (split < 8 && static_cast<long long>(blocks) * groups * split * 2 <= 2LL * device_sm_count() &&
         rows / groups / split > kSumRows * kSumWarps)
    split *= 2;
  return launch_kernel(vec ? column_sum_kernel<T, true> : column_sum_kernel<T, false>, dim3(blocks * split, groups),
                       dim3(32 * kSumWarps), 0, s, true, static_cast<unsigned>(split), static_cast<const T*>(dy), ld,
                       offsets, rows, n, out, groups, status);
}

// dz = dy act'(z), elementwise over [rows, n], four columns a step. Bound: HBM in
// fp32 (16384 x 4096, SiLU: 124 us, 6.5 TB/s; GELU by erfc and exp 179 us); in
// bf16, where a step is 8 bytes of each matrix, the slopes' instructions and the
// short loads: SiLU 88 us, 4.6 TB/s, GELU's tanh form 100, GELU 107.
template <typename T, bool kVec>
__global__ void __launch_bounds__(256) act_backward_kernel(const T* dy, long long ldy, const T* z, long long ldz, T* dz,
                                                           long long ldd, int rows, int n, int act) {
  const unsigned quads = (n + 3) / 4;
  const long long total = static_cast<long long>(rows) * quads;
  pdl_wait();
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const long long r = i / quads;
    const int c = static_cast<int>(i - r * quads) * 4;
    const Quad q = load4<T, kVec>(dy + r * ldy + c, n - c), w = load4<T, kVec>(z + r * ldz + c, n - c);
    T out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = from_f32<T>(q.v[j] * act_slope<sizeof(T) == 2>(w.v[j], act));
    T* p = dz + r * ldd + c;
    if constexpr (kVec) {
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<float4*>(p) = make_float4(out[0], out[1], out[2], out[3]);
      else
        *reinterpret_cast<uint2*>(p) = make_uint2(
            static_cast<uint32_t>(__bfloat16_as_ushort(out[0])) | static_cast<uint32_t>(__bfloat16_as_ushort(out[1])) << 16,
            static_cast<uint32_t>(__bfloat16_as_ushort(out[2])) | static_cast<uint32_t>(__bfloat16_as_ushort(out[3])) << 16);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (c + j < n) p[j] = out[j];
    }
  }
}

template <typename T>
cudaError_t act_backward(const void* dy, long long ldy, const void* z, long long ldz, void* dz, long long ldd, int rows,
                         int n, int act, bool vec, cudaStream_t s) {
  const long long quads = static_cast<long long>(rows) * ((n + 3) / 4);
  const unsigned grid = static_cast<unsigned>(std::min<long long>((quads + 255) / 256, device_sm_count() * 16LL));
  return launch_kernel(vec ? act_backward_kernel<T, true> : act_backward_kernel<T, false>, dim3(grid), dim3(256), 0, s,
                       true, 1, static_cast<const T*>(dy), ldy, static_cast<const T*>(z), ldz, static_cast<T*>(dz), ldd,
                       rows, n, act);
}

}  // namespace

cudaError_t launch_column_sums(int dtype, const void* dy, long long ld, const int32_t* offsets, int groups, int rows,
                               int n, float* out, int32_t* status, bool vec, cudaStream_t s) {
  return dtype == MOE_DTYPE_F32 ? column_sums<float>(dy, ld, offsets, groups, rows, n, out, status, vec, s)
                                : column_sums<__nv_bfloat16>(dy, ld, offsets, groups, rows, n, out, status, vec, s);
}

cudaError_t launch_act_backward(int dtype, const void* dy, long long ldy, const void* z, long long ldz, void* dz,
                                long long ldd, int rows, int n, int act, bool vec, cudaStream_t s) {
  return dtype == MOE_DTYPE_F32 ? act_backward<float>(dy, ldy, z, ldz, dz, ldd, rows, n, act, vec, s)
                                : act_backward<__nv_bfloat16>(dy, ldy, z, ldz, dz, ldd, rows, n, act, vec, s);
}

}  // namespace moe
