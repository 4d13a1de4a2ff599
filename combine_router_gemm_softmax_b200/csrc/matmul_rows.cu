// The free products in bf16 for few rows a group (moe_grouped_gemm and
// moe_linear when tokens are decoded): y[r, j] = fin(sum_i x[r, i] W_e[j, i]).
//
// Bound: HBM, the weights of the groups that have rows, each read once. A
// 128-row tile would leave most of its rows empty and, with one CTA a tile,
// too few SMs with loads in flight. Here a CTA of 8 or 4 warps takes 16 or 32
// output features of one group and 8 of its rows (launch_matmul_rows has the
// rule); its warps share the reduction, and their sums meet in shared memory in
// warp order (the same result on every run).
//
// The weights go from global memory straight into the fragments of mma.sync
// (m16n8k16, W as the 16-row operand, the tokens as the 8 columns): a lane
// reads 16 bytes of a weight row, k = 8 t .. 8 t + 7 of a chunk of 32, and
// uses them as the k pairs of two MMAs; the token operand is read the same
// way, so both operands agree on which k a slot holds and no shuffle or shared
// memory is needed. A warp has 8 KB of weights in flight.
#include "matmul_common.cuh"

namespace moe {
namespace {

constexpr int kChunk = 32;  // reduction elements of a step
// Chunks that a warp adds in one set of accumulators. The tensor cores truncate
// when they add (6e-5 of a sum of 16384 elements of one sign, 7e-4 of 131072);
// after 4096 elements the sums go to shared memory and are added there, rounded
// to nearest. Reductions of up to 16384 never get there.
constexpr int kChainChunks = 128;

// Eight elements of a row from p: all of them, or the first `valid`, or none.
template <bool kStream>
MOE_DEV uint4 load8(const __nv_bfloat16* p, int valid) {
  if (valid >= 8) {
    uint4 q;
    if constexpr (kStream)
      asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                   : "l"(p));
    else
      q = __ldg(reinterpret_cast<const uint4*>(p));
    return q;
  }
  uint32_t h[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < valid) h[i >> 1] |= static_cast<uint32_t>(__bfloat16_as_ushort(p[i])) << (16 * (i & 1));
  return make_uint4(h[0], h[1], h[2], h[3]);
}

MOE_DEV void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// kTiles: 16-feature blocks of a CTA; kWarps: its warps, 16 of which an SM holds.
template <int kTiles, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, 16 / kWarps) matmul_rows_kernel(const MatmulArgs a) {
  constexpr int kThreads = 32 * kWarps;
  constexpr int kFeatures = 16 * kTiles;
  constexpr int kUnroll = 8 / kTiles;  // chunks in flight
  __shared__ float s_sum[kWarps][8][kFeatures + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  RowBlock at{0, static_cast<int>(blockIdx.y) * 8, a.rows};
  if (a.offsets != nullptr &&
      !find_block(a.offsets, a.groups, a.rows, 3, blockIdx.y, (blockIdx.x | blockIdx.y | warp) == 0 ? a.status : nullptr,
                  lane, at))
    return;
  const int e = at.e, r0 = at.r0;
  const int have = min(8, at.end - r0);
  const int n0 = blockIdx.x * kFeatures;
  const int g = lane >> 2, t = lane & 3;

  // this warp's chunks of the reduction
  const int chunks = (a.k + kChunk - 1) / kChunk;
  const int c0 = static_cast<int>(static_cast<long long>(chunks) * warp / kWarps);
  const int c1 = static_cast<int>(static_cast<long long>(chunks) * (warp + 1) / kWarps);
  const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(a.b) + e * a.b_stride + (n0 + g) * a.ldb + t * 8;
  const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.a) + (static_cast<long long>(r0) + g) * a.lda + t * 8;
  float acc[kTiles][4];
  // rows g and g + 8 of the 16 features, tokens 2 t and 2 t + 1
  auto sum_at = [&](int m, int i) -> float& { return s_sum[warp][2 * t + (i & 1)][m * 16 + g + 8 * (i >> 1)]; };
  int from = c0;
  do {
    const int to = min(from + kChainChunks, c1);
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[m][i] = 0.0f;
    for (int c = from; c < to; c += kUnroll) {
      uint4 qw[kUnroll][2 * kTiles], qx[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int k = (c + u) * kChunk;
        const int valid = c + u < c1 ? a.k - k - t * 8 : 0;  // of this lane's eight
#pragma unroll
        for (int i = 0; i < 2 * kTiles; ++i)
          qw[u][i] = load8<true>(w + static_cast<long long>(i) * 8 * a.ldb + k, n0 + g + 8 * i < a.n ? valid : 0);
        qx[u] = load8<false>(x + k, g < have ? valid : 0);
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u)
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
          const uint4 &lo = qw[u][2 * m], &hi = qw[u][2 * m + 1];
          mma(acc[m], lo.x, hi.x, lo.y, hi.y, qx[u].x, qx[u].y);
          mma(acc[m], lo.z, hi.z, lo.w, hi.w, qx[u].z, qx[u].w);
        }
    }
#pragma unroll
    for (int m = 0; m < kTiles; ++m)
#pragma unroll
      for (int i = 0; i < 4; ++i) sum_at(m, i) = from > c0 ? sum_at(m, i) + acc[m][i] : acc[m][i];
    from = to;
  } while (from < c1);
  __syncthreads();
  for (int i = threadIdx.x; i < have * kFeatures; i += kThreads) {
    const int token = i / kFeatures, f = i % kFeatures, n = n0 + f;
    if (n >= a.n) continue;
    float v = 0.0f;
#pragma unroll
    for (int q = 0; q < kWarps; ++q) v += s_sum[q][token][f];
    const long long r = static_cast<long long>(r0) + token;
    if (a.bias != nullptr) v += a.bias[static_cast<size_t>(e) * a.n + n];
    if (a.preact != nullptr) static_cast<__nv_bfloat16*>(a.preact)[r * a.ldz + n] = __float2bfloat16_rn(v);
    v = act_of<true>(v, a.act);
    if (a.residual != nullptr) v += __bfloat162float(static_cast<const __nv_bfloat16*>(a.residual)[r * a.ldr + n]);
    static_cast<__nv_bfloat16*>(a.d)[r * a.ldd + n] = __float2bfloat16_rn(v);
  }
}

// The same in fp32 on the CUDA cores: a warp takes a part of the reduction of
// four features and kTokens of the group's rows (more take further blocks).
constexpr int kF32Features = 4, kF32Warps = 8;

template <int kTokens, bool kVec>
__global__ void __launch_bounds__(32 * kF32Warps) matmul_rows_f32_kernel(const MatmulArgs a) {
  constexpr int kShift = kTokens == 1 ? 0 : kTokens == 2 ? 1 : 2;
  __shared__ float s_sum[kF32Warps][kF32Features * kTokens];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  RowBlock at{0, static_cast<int>(blockIdx.y) * kTokens, a.rows};
  if (a.offsets != nullptr &&
      !find_block(a.offsets, a.groups, a.rows, kShift, blockIdx.y,
                  (blockIdx.x | blockIdx.y | warp) == 0 ? a.status : nullptr, lane, at))
    return;
  const int e = at.e, r0 = at.r0;
  const int have = min(kTokens, at.end - r0), n0 = blockIdx.x * kF32Features;
  const float* w = static_cast<const float*>(a.b) + e * a.b_stride + n0 * a.ldb;
  const float* x = static_cast<const float*>(a.a) + static_cast<long long>(r0) * a.lda;
  float acc[kF32Features][kTokens] = {};
  constexpr int kStep = kVec ? 4 : 1;
#pragma unroll 2
  for (int k = (warp * 32 + lane) * kStep; k < a.k; k += 32 * kF32Warps * kStep) {
    float fw[kF32Features][kStep], fx[kTokens][kStep];
    auto load = [](float(&f)[kStep], const float* p, bool there) {
      if constexpr (kVec) {
        const float4 q = there ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
        f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
      } else {
        f[0] = there ? *p : 0.0f;
      }
    };
#pragma unroll
    for (int i = 0; i < kF32Features; ++i) load(fw[i], w + i * a.ldb + k, n0 + i < a.n);
#pragma unroll
    for (int j = 0; j < kTokens; ++j) load(fx[j], x + j * a.lda + k, j < have);
#pragma unroll
    for (int i = 0; i < kF32Features; ++i)
#pragma unroll
      for (int j = 0; j < kTokens; ++j)
#pragma unroll
        for (int v = 0; v < kStep; ++v) acc[i][j] = fmaf(fw[i][v], fx[j][v], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < kF32Features; ++i)
#pragma unroll
    for (int j = 0; j < kTokens; ++j) {
      float v = acc[i][j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (lane == 0) s_sum[warp][j * kF32Features + i] = v;
    }
  __syncthreads();
  const int token = threadIdx.x / kF32Features, n = n0 + static_cast<int>(threadIdx.x) % kF32Features;
  if (token >= have || n >= a.n) return;
  float v = 0.0f;
#pragma unroll
  for (int q = 0; q < kF32Warps; ++q) v += s_sum[q][threadIdx.x];
  float f[4] = {v, 0.0f, 0.0f, 0.0f};
  finish_outputs<false, false>(a, f, e, static_cast<long long>(r0) + token, n, 1);
}

template <int kTokens>
cudaError_t launch_f32(const MatmulArgs& a, cudaStream_t s) {
  const long long blocks = (a.rows + kTokens - 1LL) / kTokens + std::min(a.groups, a.rows) - 1;
  return launch_kernel(a.vec ? matmul_rows_f32_kernel<kTokens, true> : matmul_rows_f32_kernel<kTokens, false>,
                       dim3((a.n + kF32Features - 1) / kF32Features, static_cast<unsigned>(blocks)),
                       dim3(32 * kF32Warps), 0, s, true, 1, a);
}

template <int kTiles, int kWarps>
cudaError_t launch_features(const MatmulArgs& a, long long blocks, cudaStream_t s) {
  return launch_kernel(matmul_rows_kernel<kTiles, kWarps>,
                       dim3((a.n + 16 * kTiles - 1) / (16 * kTiles), static_cast<unsigned>(blocks)), dim3(32 * kWarps), 0,
                       s, true, 1, a);
}

}  // namespace

// Row blocks: at most, however the rows fall to the groups.
static long long row_blocks(const MatmulArgs& a) { return (a.rows + 7LL) / 8 + std::min(a.groups, a.rows) - 1; }

// Where this kernel measured faster than the tiles (us, here / there):
//  - one block of one group: k 4096, n 14336, 1-8 rows 24.1 / 28.1; k 1408, n 2048
//    3.5 / 8.5;
//  - at most half as many rows as groups, so mostly a group's weights for each
//    row. In captured loops over weights that leave L2, k 2048 (rows of random
//    routes; past the cut in brackets, where the tiles run):
//      groups, n  |  rows 8        16           32           64           128
//      128,  768  |  7.3 / 15.9  11.6 / 26.0  23.8 / 22.6  37.9 / 35.3  [50.4 / 44.2]
//      256,  768  |  8.6 / 19.2  13.4 / 27.8  25.6 / 23.0  39.8 / 36.1   64.8 / 62.4
//      64,  1408  |  9.2 / 21.5  15.9 / 33.6  29.4 / 44.3 [47.8 / 43.0] [66.0 / 60.9]
//    (6, 12, 30, 60 and 126 rows in the last line); k 768, n 2048, 128 groups:
//    8.1 / 17.6, 15.2 / 19.3, 26.0 / 24.3, 43.0 / 35.8, [60.0 / 44.6]. So the cut
//    lies about right for 64 groups (48 rows 39.8 / 40.9, 96 rows 56.0 / 58.6)
//    and too far for 128 and more, by 5 to 20% of a call between a quarter and
//    a half; the crossing follows the tiles' widths more than the rows;
//  - several blocks that read a group's weights again from L2, while all of
//    them run at once: on half of the SMs' warps k = n = 4096, 16 rows
//    11.2 / 13.7, k 2048, n 16, 2048 rows 3.8 / 9.9 (k 128, n 640, 256 rows, more
//    than one wave: 6.3 / 3.6); on all of them if the reads stay small: k 1408,
//    n 2048, 64 rows, 46 MB 8.0 / 8.8 (k = n = 4096, 24 rows, 100 MB 15.5 / 13.9).
bool matmul_few_rows(const MatmulArgs& a, int sms) {
  if (a.rows <= 8 || 2LL * a.rows <= a.groups) return true;
  const long long blocks = row_blocks(a), warps = (a.n + 31) / 32 * 4 * blocks;
  return warps <= 7LL * sms || (warps <= 16LL * sms && blocks * a.n * a.k <= (24LL << 20));
}

cudaError_t launch_matmul_rows(const MatmulArgs& a, int sms, cudaStream_t s) {
  const long long blocks = row_blocks(a);
  // The cut with the most warps that still fit on the SMs at once (16 each):
  // with k 4096, n 4096 and one row 16 features x 8 warps take 8.2 us, 32 x 8
  // 10.1 and 32 x 4 15.5; with n 14336, 26.7, 25.4 and 23.8 us.
  const long long fit = 16LL * sms;
  if ((a.n + 15) / 16 * blocks * 8 <= fit) return launch_features<1, 8>(a, blocks, s);
  if ((a.n + 31) / 32 * blocks * 8 <= fit) return launch_features<2, 8>(a, blocks, s);
  return launch_features<2, 4>(a, blocks, s);
}

bool matmul_few_rows_f32(const MatmulArgs& a) { return a.rows <= 8 || 2LL * a.rows <= a.groups; }

cudaError_t launch_matmul_rows_f32(const MatmulArgs& a, cudaStream_t s) {
  const int each = (a.rows + a.groups - 1) / a.groups;
  return each == 1 ? launch_f32<1>(a, s) : each == 2 ? launch_f32<2>(a, s) : launch_f32<4>(a, s);
}

}  // namespace moe
