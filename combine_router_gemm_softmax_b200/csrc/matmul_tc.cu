// The free products in bf16 (moe_grouped_gemm, moe_linear and their gradients)
// on the tensor cores, over ragged row groups.
//
//   forward   D[r, j] = fin(sum_i x[r, i] W_e[j, i])      A = x, B = W_e
//   dgrad     D[r, i] = fin(sum_j dy[r, j] W_e[j, i])     A = dy, B = W_e read across
//   wgrad     D_e[j, i] = sum_r dy[r, j] x[r, i]          A = dy, B = x, both read across
//
// Nothing is transposed or packed beforehand: an operand whose reduction index
// is the contiguous one enters the MMA K-major, one that lies across it
// MN-major (both 128-byte swizzled tiles as the TMA loads write them, told
// apart by the matrix and instruction descriptors). W is a three-dimensional
// tensor map (k, n, group), so that what lies past a group's last row of W is
// zero and not the next group's.
//
// Persistent CTAs (one an SM) walk a tile list built on the device from the
// offsets. Warp 0 loads a ring of up to 8 stages (192 KB) by TMA, one thread
// of warp 1 issues tcgen05.mma into one of two TMEM accumulators, warps 2..9
// drain the other: bias, activation, slope and residual in fp32, one rounding,
// then stores. Three forms:
//
//   kPair    256 x bn tiles on a cluster of two CTAs (cta_group::2): each loads
//            128 rows of A and half of B, 32 KB for a block of 64 along the
//            reduction at bn = 256, so that the ring covers 3000 cycles of load
//            latency. The form for large products.
//   kSingle  128 x bn tiles, a CTA each (48 KB a block): groups of few rows,
//            whose 256-row tiles would be padding.
//   kSplit   a cluster of CTAs shares one 128 x bn tile's reduction when there
//            are few tiles: the partial tiles lie in the CTAs' own shared
//            memory, and each CTA adds its share of the 32 x 32 blocks over all
//            of them in rank order, then runs the epilogue on it (the same
//            order on every run).
//
// The width bn is chosen per call so that the tiles fill the SMs evenly
// (choose_tiles); the last column tile issues MMAs only as wide as it is.
//
// Bound: the tensor pipe, at the clock that the 1 kW limit leaves (8192 x 4096 x
// 4096: pipe 91-92% active forward and dgrad, 81% wgrad with 512-row
// accumulators; 8192 x 14336 x 4096 forward and dgrad: 1.27-1.35 PFLOP/s in
// loops, a library product 1.32-1.37); for short reductions the epilogue, for
// few rows a group the weights' bytes.
//
// wgrad's reduction is the group's rows: its last 64-row block may run into
// the next group, so warp 1 zeroes those rows of both operands in shared memory
// (a row of a tile is 128 contiguous bytes whatever the swizzle) before the MMA
// reads them. Zeroing one operand would not do: the other may hold NaN.
//
// The tensor cores add into an fp32 accumulator by truncation, which biases a
// long sum towards zero by about 1.1e-9 of it a row (measured: 1.9e-5 over
// 16384 rows, more than in proportion beyond). An accumulator therefore takes
// chain_blocks() of the reduction only, and the epilogue adds these partial
// sums, rounded to nearest, in registers, while the MMAs fill the other
// accumulator. wgrad's fp32 outputs take 512 rows (relative error of normal
// sums, root mean square, and the time of 8192 rows, 4096 x 14336 in loops:
// 256 rows 2.5e-7, 1076 us; 384 3.6e-7, 883; 512 4.8e-7, 801; 768 7.2e-7, 776;
// a plain fp32 product 9.6e-7 at this length, 2.5e-7 at 1000 rows, 1.5e-6 at
// 16384), the bf16 outputs of the rows modes 16384 elements, a hundredth of
// half their step, so that no reduction grows less exact than that. In rows
// mode the adding is an instance of its own (kChained), since its registers
// spill in the others.
#include <cmath>

#include "matmul_common.cuh"

namespace moe {
namespace {

constexpr int kBM = 128;
constexpr int kBN = 256;  // columns of an accumulator: the widest tile
constexpr int kBK = 64;
constexpr int kMaxStages = 8;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 32 * (2 + kEpiWarps);

// Blocks of the reduction added in one accumulator (whole stages of the ring).
constexpr int chain_blocks(MatmulMode m) { return m == MatmulMode::kWgrad ? 8 : 256; }
constexpr uint32_t kABytes = kBM * kBK * 2;  // one CTA's rows of A
constexpr uint32_t kTmemCols = 2 * kBN;
constexpr uint32_t kBoxBytes = 64 * 128;  // an MN-major box: 64 reduction rows of 64 elements

// Blocks of 64 along the reduction that a stage of the ring holds. Two halve
// the barrier traffic of a block, which bounds narrow tiles (pairs of width
// 128: 221 -> 187 ns a block); the 48 KB blocks of wide single tiles leave no
// room for them.
constexpr int blocks_per_stage(Form f) { return f == Form::kPair ? 2 : 1; }

struct TcArgs {
  MatmulArgs p;
  int bn;                // columns of a tile: a multiple of 32 up to kBN
  int stages;            // of the operand ring
  uint32_t block_bytes;  // of one block in one CTA's ring
  int n_tiles, m_tiles;  // column tiles; weight mode: row tiles of one group
  int band;              // row tiles per band of the tile walk
  int stall;             // testing hook: the MMA warp first waits on a barrier that nothing signals
  int align_d, align_p, align_z, align_r;  // bytes that rows of D, preact, z and the residual start on: 32, 16, or less
};

// full, empty, tails and zeroed per stage, two accumulators' full and empty, the drain; even
constexpr int kBarriers = 4 * kMaxStages + 6;

template <MatmulMode kMode>
struct Shape {
  static constexpr bool kWeight = kMode == MatmulMode::kWgrad;
  static constexpr bool kAcrossA = kWeight;                       // A lies across the reduction
  static constexpr bool kAcrossB = kMode != MatmulMode::kForward;  // B does
  static constexpr uint32_t kRingBytes = 192 * 1024;
  static constexpr uint32_t kStgBytes = kWeight ? 32 * 128 : 0;  // a warp's store staging
  static constexpr size_t kSmem = 1024 + kRingBytes + kEpiWarps * kStgBytes + kBarriers * 8 + 16 +
                                  (kWeight ? 0 : (kMaxE + 1) * 4);
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// Matrix descriptor of an MN-major tile: boxes of 64 reduction rows x 64
// elements (128 bytes a row, 128-byte swizzle). Eight reduction rows are 1024
// bytes; the next 64 elements along M or N are the next box. Sixteen reduction
// rows further is 2048 bytes.
MOE_DEV uint64_t sw128_mnmajor_desc(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(kBoxBytes >> 4) << 16;  // leading-dimension offset: 64 elements along M/N
  d |= static_cast<uint64_t>(1024 >> 4) << 32;       // stride: 8 rows along the reduction
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

template <bool kAcross>
MOE_DEV uint64_t operand_desc(uint32_t tile) {
  return kAcross ? sw128_mnmajor_desc(tile) : sw128_kmajor_desc(tile);
}

// A tile: group, row tile, column tile, its blocks of 64 along the reduction,
// and the group's rows.
struct Tile {
  int e, m, n, kb0, kb1;
  int2 rows;
};

// Tile loads completing on the barrier at `bar` (of this CTA, or with kPair of
// the pair's CTA whose address it is).
template <bool kPair>
MOE_DEV void load_2d(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  if constexpr (kPair)
    tma_load_2d_pair(dst, map, bar, x, y);
  else
    tma_load_2d_at(dst, map, bar, x, y);
}

template <bool kPair>
MOE_DEV void load_3d(void* dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  if constexpr (kPair)
    tma_load_3d_pair(dst, map, bar, x, y, z);
  else
    tma_load_3d_at(dst, map, bar, x, y, z);
}

// 32 bf16 of a row from column n0 (n columns in all), as they are; columns
// past n, and all of them where the lane has no row, are zero.
struct Row32 {
  uint4 q[4];
};

MOE_DEV Row32 load_row(const void* base, long long at, int n0, int n, int align, bool valid) {
  Row32 r;
  const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(base) + at;
  if (n0 + 32 <= n && align >= 32) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.q[i] = make_uint4(0, 0, 0, 0);
    if (valid) {
#pragma unroll
      for (int i = 0; i < 4; i += 2)
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r.q[i].x), "=r"(r.q[i].y), "=r"(r.q[i].z), "=r"(r.q[i].w), "=r"(r.q[i + 1].x),
                       "=r"(r.q[i + 1].y), "=r"(r.q[i + 1].z), "=r"(r.q[i + 1].w)
                     : "l"(p + 8 * i)
                     : "memory");
    }
  } else if (n0 + 32 <= n) {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.q[i] = valid ? reinterpret_cast<const uint4*>(p)[i] : make_uint4(0, 0, 0, 0);
  } else {
    uint32_t h[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t lo = valid && n0 + 2 * i < n ? __bfloat16_as_ushort(p[2 * i]) : 0;
      const uint32_t hi = valid && n0 + 2 * i + 1 < n ? __bfloat16_as_ushort(p[2 * i + 1]) : 0;
      h[i] = lo | (hi << 16);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) r.q[i] = make_uint4(h[4 * i], h[4 * i + 1], h[4 * i + 2], h[4 * i + 3]);
  }
  return r;
}

MOE_DEV float2 pair_of(const Row32& r, int i) {  // elements 2 i and 2 i + 1
  const uint4& q = r.q[i >> 2];
  const uint32_t w = (i & 3) == 0 ? q.x : (i & 3) == 1 ? q.y : (i & 3) == 2 ? q.z : q.w;
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

// Rows mode: a lane's 32 bf16 columns of the output, `have` of which exist,
// straight from its registers: whole 32-byte sectors where rows start on them
// (`align`), else 16 bytes, else single elements. Staged through shared
// memory, whose bandwidth the MMA operands and the ring's loads use up, or
// stored by TMA, a proxy fence a block, a short reduction's blocks took longer
// (k 512, single tiles: 3.8 us a tile against 4.5).
MOE_DEV void store_rows(const float (&f)[32], void* base, long long at, int have, int align, bool valid) {
  if (!valid) return;
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = pack_bf16x2(f[2 * i], f[2 * i + 1]);
  __nv_bfloat16* p = static_cast<__nv_bfloat16*>(base) + at;
  if (have >= 32 && align >= 32) {
#pragma unroll
    for (int i = 0; i < 16; i += 8)
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p + 2 * i), "r"(w[i]), "r"(w[i + 1]),
                   "r"(w[i + 2]), "r"(w[i + 3]), "r"(w[i + 4]), "r"(w[i + 5]), "r"(w[i + 6]), "r"(w[i + 7])
                   : "memory");
  } else if (have >= 32) {  // 16 bytes: what the entry points demand
#pragma unroll
    for (int i = 0; i < 16; i += 4)
      *reinterpret_cast<uint4*>(p + 2 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (i < have) p[i] = __float2bfloat16_rn(f[i]);
  }
}

// Weight mode: a warp's 32 x 32 block of fp32, a row a lane, through shared
// memory (16-byte chunk j of row r at j ^ (r & 7)), so that a store instruction
// writes 4 whole rows of 128 bytes. With many short groups the stores are what
// bounds the kernel, and 32-byte pieces of 32 rows an instruction cost 17%
// there (2051 tokens in 128 groups: 322 us against 275, both gradients).
MOE_DEV void store_block(uint8_t* stg, const float (&f)[32], float* out, long long ld, int rows, int cols, bool vec,
                         int lane) {
  auto place = [](int r, int j) { return r * 128 + ((j ^ (r & 7)) << 4); };
  __syncwarp();
#pragma unroll
  for (int j = 0; j < 8; ++j)
    *reinterpret_cast<float4*>(stg + place(lane, j)) = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
  __syncwarp();
  const int j = lane & 7, have = cols - j * 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = i * 4 + (lane >> 3);
    const float4 q = *reinterpret_cast<const float4*>(stg + place(r, j));
    if (r >= rows) continue;
    float* p = out + r * ld + j * 4;
    if (have >= 4 && vec) {
      *reinterpret_cast<float4*>(p) = q;
    } else {
      if (have > 0) p[0] = q.x;
      if (have > 1) p[1] = q.y;
      if (have > 2) p[2] = q.z;
      if (have > 3) p[3] = q.w;
    }
  }
}

// What the epilogue of a rows-mode block reads besides the sums, loaded ahead
// of them: z (dgrad, if any) or else the residual.
template <bool kDgrad>
MOE_DEV Row32 load_ahead(const TcArgs& a, long long r, int n0, bool valid) {
  const MatmulArgs& p = a.p;
  if (kDgrad && p.z != nullptr) return load_row(p.z, r * p.ldz + n0, n0, p.n, a.align_z, valid);
  if (p.residual != nullptr) return load_row(p.residual, r * p.ldr + n0, n0, p.n, a.align_r, valid);
  return Row32{};
}

// The epilogue of one 32 x 32 block of rows mode: rows row0 .. of which the
// group has `left`, this lane's the lane-th; columns n0 ..; sums in f.
template <bool kDgrad>
MOE_DEV void finish_rows(const TcArgs& a, float (&f)[32], const Row32& ahead, int e, long long row0, int left, int n0,
                         int lane) {
  const MatmulArgs& p = a.p;
  const long long r = row0 + lane;
  const bool valid = lane < left;
  if constexpr (kDgrad) {
    if (p.z != nullptr) {
      with_act(p.act, [&](auto k) {
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float2 z = pair_of(ahead, i);
          f[2 * i] *= slope_value<decltype(k)::value, true>(z.x);
          f[2 * i + 1] *= slope_value<decltype(k)::value, true>(z.y);
        }
      });
    }
  } else {
    if (p.bias != nullptr) {
      const float b = n0 + lane < p.n ? p.bias[static_cast<size_t>(e) * p.n + n0 + lane] : 0.0f;
#pragma unroll
      for (int i = 0; i < 32; ++i) f[i] += __shfl_sync(0xffffffffu, b, i);
    }
    if (p.preact != nullptr) store_rows(f, p.preact, r * p.ldz + n0, p.n - n0, a.align_p, valid);
    if (p.act != MOE_ACT_NONE)
      with_act(p.act, [&](auto k) {
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = act_value<decltype(k)::value, true>(f[i]);
      });
  }
  if (p.residual != nullptr) {
    const Row32 res = kDgrad && p.z != nullptr
                          ? load_row(p.residual, r * p.ldr + n0, n0, p.n, a.align_r, valid)
                          : ahead;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 t = pair_of(res, i);
      f[2 * i] += t.x;
      f[2 * i + 1] += t.y;
    }
  }
  store_rows(f, p.d, r * p.ldd + n0, p.n - n0, a.align_d, valid);
}

// One 32 x 32 block to its epilogue (weight mode: fp32 rows of group e's gradient).
template <MatmulMode kMode>
MOE_DEV void finish_block(const TcArgs& a, float (&f)[32], const Row32& ahead, const Tile& c, int row0, int left, int n0,
                          uint8_t* stg, int lane) {
  if constexpr (Shape<kMode>::kWeight) {
    const MatmulArgs& p = a.p;
    store_block(stg, f, static_cast<float*>(p.d) + (static_cast<long long>(c.e) * p.m + row0) * p.ldd + n0, p.ldd, left,
                p.n - n0, a.align_d >= 16, lane);
  } else {
    finish_rows<kMode == MatmulMode::kDgrad>(a, f, ahead, c.e, row0, left, n0, lane);
  }
}

// kChained: reductions may be longer than an accumulator takes (always, in weight mode).
template <MatmulMode kMode, Form kForm, bool kChained>
__global__ void __launch_bounds__(kThreads, 1)
    matmul_tc_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                     const TcArgs a) {
  using S = Shape<kMode>;
  constexpr bool kPair = kForm == Form::kPair, kSplit = kForm == Form::kSplit;
  constexpr int kTileM = kPair ? 2 * kBM : kBM, kPerStage = blocks_per_stage(kForm);
  constexpr int kChain = chain_blocks(kMode);
  static_assert(kChain % kPerStage == 0, "an accumulator takes whole stages");
  static_assert(kChained || !S::kWeight, "a group may have any number of rows, none too");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_1024(smem_raw);  // the ring: per stage A, then B
  uint8_t* stg_all = smem + S::kRingBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(stg_all + kEpiWarps * S::kStgBytes);
  uint64_t* empty = full + kMaxStages;
  // kPair, weight mode, a block with rows to zero: the second CTA's loads
  // complete on its own tails[s], and its zeroing on the leader's zeroed[s]
  uint64_t* tails = empty + kMaxStages;
  uint64_t* zeroed = tails + kMaxStages;
  uint64_t* tfull = zeroed + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(full + kBarriers);  // 16-byte aligned, and what follows it
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* consumed_slot = reinterpret_cast<int*>(tmem_slot + 2);
  int* prefix = reinterpret_cast<int*>(tmem_slot + 4);  // rows modes: row tiles before each group

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const MatmulArgs& p = a.p;
  uint32_t split = 1, rank = 0;  // CTAs of the cluster, this one's place
  if constexpr (kForm != Form::kSingle) {
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(split));
    rank = cluster_ctarank();
  }
  const bool leader = rank == 0;
  auto raise_abort = [&]() {
    *abort_flag = 1;
    if constexpr (kPair) st_shared_cluster_u32(mapa_shared(smem_addr(const_cast<int*>(abort_flag)), rank ^ 1u), 1u);
  };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tails[s], 1);
      mbar_init(&zeroed[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&tfull[i], 1);
      mbar_init(&tempty[i], kPair ? 2 * kEpiWarps : kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *consumed_slot = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  pdl_wait();  // everything before this runs beside the end of the stream's previous kernel
  if (warp == 0) {
    if constexpr (S::kWeight) {
      bool bad = false;
      for (int e = lane; e < p.groups; e += 32) group_rows(p.offsets, e, p.rows, &bad);
      if (bad && blockIdx.x == 0) report_status(p.status, MOE_STATUS_BAD_OFFSETS);
    } else {
      build_groups(p.offsets, p.groups, p.rows, kPair ? 8 : 7, nullptr, prefix, p.status, lane);
    }
  } else if (warp == 1) {
    if constexpr (kPair) {
      tmem_alloc_pair(tmem_slot, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_slot, kTmemCols);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (kPair) cluster_sync();  // both CTAs' barriers are initialised before any cross-CTA signal
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int m_total = S::kWeight ? p.groups * a.m_tiles : prefix[p.groups];
  const uint32_t total = static_cast<uint32_t>(m_total) * a.n_tiles;  // below 2^31 (plan_product)
  const uint32_t first_tile = blockIdx.x / split;
  const uint32_t step = kSplit ? 1u << 31 : gridDim.x / split;  // a split cluster has one tile (or none)

  // Bands of row tiles, each swept over all column tiles, so that a wave of
  // CTAs shares A and B in L2; in weight mode the bands stay inside a group.
  auto tile_at = [&](uint32_t t) {
    Tile c;
    if constexpr (S::kWeight) {
      const uint32_t per = a.m_tiles * a.n_tiles, band_tiles = a.band * a.n_tiles;
      c.e = t / per;
      const uint32_t rem = t - c.e * per, b = rem / band_tiles, within = rem - b * band_tiles;
      const uint32_t rows = min(a.band, static_cast<int>(a.m_tiles - b * a.band));
      c.m = b * a.band + within % rows;
      c.n = within / rows;
      c.rows = group_rows(p.offsets, c.e, p.rows);
      c.kb0 = 0;
      c.kb1 = (c.rows.y - c.rows.x + kBK - 1) / kBK;
    } else {
      const uint32_t band_tiles = a.band * a.n_tiles, b = t / band_tiles, within = t - b * band_tiles;
      const uint32_t rows = min(a.band, static_cast<int>(m_total - b * a.band));
      const int gm = b * a.band + within % rows;
      c.n = within / rows;
      c.e = group_of_tile(prefix, p.groups, gm);
      c.m = gm - prefix[c.e];
      c.rows = group_rows(p.offsets, c.e, p.rows);
      c.kb0 = 0;
      c.kb1 = (p.k + kBK - 1) / kBK;
    }
    if constexpr (kSplit) {
      const int blocks = c.kb1;
      c.kb0 = static_cast<int>(static_cast<long long>(blocks) * rank / split);
      c.kb1 = static_cast<int>(static_cast<long long>(blocks) * (rank + 1) / split);
    }
    return c;
  };
  // Columns the MMAs of a tile compute; each CTA of a pair loads half of them,
  // and both halves are multiples of 16.
  auto width_of = [&](const Tile& c) {
    constexpr int kUnit = kPair ? 32 : 16;
    return min(a.bn, (p.n - c.n * a.bn + kUnit - 1) & ~(kUnit - 1));
  };
  // Rows of the group in block kb of the reduction (weight mode). Of a last
  // block the MMAs take them in steps of 16; the rest of such a step is zeroed.
  auto rows_in = [&](const Tile& c, int kb) { return min(c.rows.y - c.rows.x - kb * kBK, kBK); };
  const int b_cols = kPair ? a.bn / 2 : a.bn;  // columns of B in this CTA's ring
  const int b_boxes = (b_cols + 63) / 64;       // of a B that lies across

  int issued = 0;
  uint32_t tail_seen = 0, tail_last = 0;  // kPair's second CTA: stages whose tails[] was used, and the last phase's parity
  if (warp == 0) {
    // ---------------------------------------------------------------- TMA producer
    int s = 0;
    uint32_t phase = 0, tail_next = 0;
    bool stop = false;
    const uint32_t full_leader = kPair ? mapa_shared(smem_addr(&full[0]), 0) : smem_addr(&full[0]);
    for (uint32_t t = first_tile; t < total && !stop; t += step) {
      const Tile c = tile_at(t);
      const int n0 = c.n * a.bn + (kPair ? static_cast<int>(rank) * (width_of(c) / 2) : 0);
      const int m0 = c.m * kTileM + (kPair ? static_cast<int>(rank) * kBM : 0);
      for (int kb = c.kb0; kb < c.kb1; kb += kPerStage) {
        if (!mbar_wait(&empty[s], phase ^ 1, abort_flag)) {
          raise_abort();
          stop = true;
          break;
        }
        const int blocks = min(kPerStage, c.kb1 - kb);
        const bool tail = kPair && S::kWeight && rows_in(c, kb + blocks - 1) % 16 != 0;
        const bool own_tail = tail && !leader;
        if (elect_one()) {
          const uint32_t bar = own_tail ? smem_addr(&tails[s]) : full_leader + s * 8;
          if (own_tail)
            mbar_expect_tx(&tails[s], blocks * a.block_bytes);
          else if (leader || !kPair)
            mbar_expect_tx(&full[s], (kPair && !tail ? 2 : 1) * blocks * a.block_bytes);
          for (int i = 0; i < blocks; ++i) {
            uint8_t* da = smem + (s * kPerStage + i) * a.block_bytes;
            uint8_t* db = da + kABytes;
            const int k = kb + i;
            if constexpr (S::kWeight) {
              const int r = c.rows.x + k * kBK;
#pragma unroll
              for (int j = 0; j < kBM / 64; ++j) load_2d<kPair>(da + j * kBoxBytes, &tm_a, bar, m0 + j * 64, r);
              for (int j = 0; j < b_boxes; ++j) load_2d<kPair>(db + j * kBoxBytes, &tm_b, bar, n0 + j * 64, r);
            } else {
              load_2d<kPair>(da, &tm_a, bar, k * kBK, c.rows.x + m0);
              if constexpr (S::kAcrossB) {
                for (int j = 0; j < b_boxes; ++j) load_3d<kPair>(db + j * kBoxBytes, &tm_b, bar, n0 + j * 64, k * kBK, c.e);
              } else {
                load_3d<kPair>(db, &tm_b, bar, k * kBK, n0, c.e);
              }
            }
          }
        }
        __syncwarp();
        if (own_tail) {
          tail_seen |= 1u << s;
          tail_last = (tail_last & ~(1u << s)) | (tail_next & (1u << s));
          tail_next ^= 1u << s;
        }
        ++issued;
        if (++s == a.stages) {
          s = 0;
          phase ^= 1;
        }
      }
    }
  } else if (warp == 1) {
    // ---------------------------------------------------------------- MMA issuer
    // The whole warp walks the ring; one lane issues (the leader's, of a pair),
    // and in weight mode all lanes zero the rows of a group's last block that
    // belong to no one (the second CTA's warp does only that).
    int s = 0, consumed = 0, filled = 0;  // ring stage, blocks taken, accumulators filled
    uint32_t phase = 0, tail_next = 0;
    bool stop = false;
    const uint64_t ring_a = operand_desc<S::kAcrossA>(smem_addr(smem));
    const uint64_t ring_b = operand_desc<S::kAcrossB>(smem_addr(smem) + kABytes);
    if (a.stall && !mbar_wait(drain, 0, abort_flag)) stop = true;  // nothing arrives on `drain` before the end
    auto zero_rows = [&](int block, int have) {
      const int chunks = (16 - have % 16) * 8;  // 16-byte chunks of one box
      uint8_t* base = smem + (s * kPerStage + block) * a.block_bytes + have * 128;
#pragma unroll 1
      for (int box = 0; box < kBM / 64 + b_boxes; ++box)
        for (int i = lane; i < chunks; i += 32)
          *reinterpret_cast<uint4*>(base + box * kBoxBytes + i * 16) = make_uint4(0, 0, 0, 0);
      fence_proxy_async_shared();
      __syncwarp();
    };
    for (uint32_t t = first_tile; t < total && !stop; t += step) {
      const Tile c = tile_at(t);
      const uint32_t idesc =
          idesc_bf16_f32(kTileM, width_of(c)) | (S::kAcrossA ? 1u << 15 : 0u) | (S::kAcrossB ? 1u << 16 : 0u);
      for (int k0 = c.kb0; k0 < c.kb1 && !stop; k0 += kChained ? kChain : c.kb1 - c.kb0, ++filled) {
        const int acc = filled & 1;
        if (leader || !kPair) {
          if (!mbar_wait(&tempty[acc], ((filled >> 1) & 1) ^ 1, abort_flag)) {
            stop = true;
            break;
          }
          tc_fence_after();
        }
        const uint32_t d_tmem = tmem + acc * kBN;
        const int k1 = kChained ? min(k0 + kChain, c.kb1) : c.kb1;
        for (int kb = k0; kb < k1; kb += kPerStage) {
          const int blocks = min(kPerStage, k1 - kb);
          const int have = S::kWeight ? rows_in(c, kb + blocks - 1) : kBK;  // of the stage's last block
          bool ok = true;
          if (kPair && !leader) {
            if (have % 16 != 0) {
              ok = mbar_wait(&tails[s], (tail_next >> s) & 1, abort_flag);
              if (ok) {
                zero_rows(blocks - 1, have);
                if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_addr(&zeroed[s]), 0));
              }
              tail_next ^= 1u << s;
            }
          } else {
            ok = mbar_wait(&full[s], phase, abort_flag);
            if (ok && have % 16 != 0) {
              zero_rows(blocks - 1, have);
              if constexpr (kPair) {
                ok = mbar_wait(&zeroed[s], (tail_next >> s) & 1, abort_flag);
                fence_acq_rel_cluster();
                tail_next ^= 1u << s;
              }
            }
            if (ok && elect_one()) {
              // descriptors hold addresses in 16-byte units, and no sum of them leaves its field
              uint32_t at = s * kPerStage * (a.block_bytes >> 4);
              for (int i = 0; i < blocks; ++i, at += a.block_bytes >> 4) {
#pragma unroll
                for (int kk = 0; kk < kBK / 16; ++kk) {
                  if (S::kWeight && i == blocks - 1 && kk * 16 >= have) break;
                  const uint64_t da = ring_a + (at + kk * (S::kAcrossA ? 2048 >> 4 : 32 >> 4));
                  const uint64_t db = ring_b + (at + kk * (S::kAcrossB ? 2048 >> 4 : 32 >> 4));
                  const uint32_t add = (kb != k0) || (i != 0) || (kk != 0);
                  if constexpr (kPair)
                    umma_bf16_pair(d_tmem, da, db, idesc, add);
                  else
                    umma_bf16(d_tmem, da, db, idesc, add);
                }
              }
              if constexpr (kPair)
                umma_commit_pair_all(&empty[s], 0x3);
              else
                umma_commit(&empty[s]);
            }
            __syncwarp();
          }
          if (!ok) {
            stop = true;
            break;
          }
          ++consumed;
          if (++s == a.stages) {
            s = 0;
            phase ^= 1;
          }
        }
        if (!stop && elect_one()) {
          if constexpr (kPair) {
            if (leader) umma_commit_pair_all(&tfull[acc], 0x3);
          } else {
            umma_commit(&tfull[acc]);
          }
        }
        __syncwarp();
      }
    }
    __syncwarp();
    if (elect_one()) {
      if (stop) raise_abort();
      *consumed_slot = consumed;
      if (leader || !kPair) {
        if constexpr (kPair)
          umma_commit_pair(drain);
        else
          umma_commit(drain);
        mbar_wait(drain, 0, nullptr);
      }
    }
  } else {
    // ---------------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quadrant this warp may read
    // its 32-column blocks of the tile: the first or the second half
    const int blocks = a.bn / 32, half = (warp - 2) >> 2;
    const int b_first = half * ((blocks + 1) / 2), b_end = half ? blocks : (blocks + 1) / 2;
    uint8_t* stg = stg_all + (warp - 2) * S::kStgBytes;
    const uint32_t lanes = static_cast<uint32_t>(q * 32) << 16;
    int filled = 0;
    auto wait_acc = [&]() {
      if (!mbar_wait(&tfull[filled & 1], (filled >> 1) & 1, abort_flag)) {
        raise_abort();
        return false;
      }
      tc_fence_after();
      return true;
    };
    auto free_acc = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (kPair)
          mbar_arrive_cluster(mapa_shared(smem_addr(&tempty[filled & 1]), 0));
        else
          mbar_arrive(&tempty[filled & 1]);
      }
      ++filled;
    };
    // a partial tile into the operand ring, which nothing reads any more:
    // block (q, c32) of 32 rows x 128 bytes, 16-byte chunks swizzled
    auto keep_partial = [&](int c32, const float (&f)[32]) {
      uint8_t* row = smem + (c32 * 4 + q) * 4096 + lane * 128;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<float4*>(row + ((j ^ (lane & 7)) << 4)) =
            make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
    };
    for (uint32_t t = first_tile; t < total; t += step) {
      const Tile c = tile_at(t);
      const int m0 = c.m * kTileM + (kPair ? static_cast<int>(rank) * kBM : 0) + q * 32;
      const int row0 = S::kWeight ? m0 : c.rows.x + m0;
      const int left = S::kWeight ? p.m - row0 : c.rows.y - row0;  // rows from row0 to the end
      const bool whole = !kChained || (c.kb1 > c.kb0 && c.kb1 - c.kb0 <= kChain);  // one accumulator holds the sums
      if (kChained && !whole) {
        float f[4][32];
#pragma unroll
        for (int b = 0; b < 4; ++b)
#pragma unroll
          for (int i = 0; i < 32; ++i) f[b][i] = 0.0f;
        bool ok = true;
        for (int k0 = c.kb0; k0 < c.kb1; k0 += kChain) {
          if (!(ok = wait_acc())) break;
          const uint32_t tbase = tmem + (filled & 1) * kBN + lanes + b_first * 32;
#pragma unroll
          for (int b = 0; b < 8; ++b) {
            if (b_first + (b >> 1) >= b_end) break;
            uint32_t v[16];
            tmem_ld16(tbase + b * 16, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 16; ++i) f[b >> 1][(b & 1) * 16 + i] += __uint_as_float(v[i]);
          }
          free_acc();
        }
        if (!ok) break;
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const int c32 = b_first + b, n0 = c.n * a.bn + c32 * 32;
          if (c32 >= b_end) break;
          if constexpr (kSplit) {
            keep_partial(c32, f[b]);
          } else {
            if (n0 >= p.n || left <= 0) continue;
            Row32 ahead{};
            if constexpr (!S::kWeight)
              ahead = load_ahead<kMode == MatmulMode::kDgrad>(a, row0 + lane, n0, lane < left);
            finish_block<kMode>(a, f[b], ahead, c, row0, left, n0, stg, lane);
          }
        }
      } else {
        constexpr bool kDgrad = kMode == MatmulMode::kDgrad, kAhead = !kSplit && !S::kWeight;
        Row32 next{};
        if constexpr (kAhead) next = load_ahead<kDgrad>(a, row0 + lane, c.n * a.bn + b_first * 32, lane < left);
        if (!wait_acc()) break;
        const uint32_t tbase = tmem + (filled & 1) * kBN + lanes;
#pragma unroll 1
        for (int c32 = b_first; c32 < b_end; ++c32) {
          const int n0 = c.n * a.bn + c32 * 32;
          if (n0 >= p.n || left <= 0) break;
          uint32_t v[32];
          float f[32];
          tmem_ld32(tbase + c32 * 32, v);
          const Row32 ahead = next;
          if constexpr (kAhead) next = load_ahead<kDgrad>(a, row0 + lane, n0 + 32, c32 + 1 < b_end && lane < left);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
          if constexpr (kSplit)
            keep_partial(c32, f);
          else
            finish_block<kMode>(a, f, ahead, c, row0, left, n0, stg, lane);
        }
        free_acc();
      }
    }
  }
  __syncwarp();
  if constexpr (kSplit) {
    cluster_sync();  // every partial tile is in place
    if (warp >= 2 && first_tile < total && !*abort_flag) {
      const Tile c = tile_at(first_tile);
      uint8_t* stg = stg_all + (warp - 2) * S::kStgBytes;
      // the tile's blocks of 32 x 32 shared out over the cluster's epilogue warps
#pragma unroll 1
      for (int b = rank * kEpiWarps + warp - 2; b < (a.bn / 32) * 4; b += split * kEpiWarps) {
        const int q = b & 3, c32 = b >> 2;
        const int n0 = c.n * a.bn + c32 * 32;
        const int row0 = (S::kWeight ? 0 : c.rows.x) + c.m * kBM + q * 32;
        const int left = S::kWeight ? p.m - row0 : c.rows.y - row0;
        if (n0 >= p.n || left <= 0) continue;
        const uint32_t row = smem_addr(smem) + b * 4096 + lane * 128;
        Row32 ahead{};
        if constexpr (!S::kWeight)
          ahead = load_ahead<kMode == MatmulMode::kDgrad>(a, row0 + lane, n0, lane < left);
        float f[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) f[i] = 0.0f;
#pragma unroll 1
        for (uint32_t k = 0; k < split; ++k) {
          const uint32_t peer = mapa_shared(row, k);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float g[4];
            ld_shared_cluster_v4(peer + ((j ^ (lane & 7)) << 4), g);
#pragma unroll
            for (int i = 0; i < 4; ++i) f[4 * j + i] += g[i];
          }
        }
        finish_block<kMode>(a, f, ahead, c, row0, left, n0, stg, lane);
      }
    }
    cluster_sync();  // nobody leaves while a peer reads its shared memory
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (*abort_flag) {
    if (threadIdx.x == 0) report_status(p.status, MOE_STATUS_TIMEOUT);
    // loads issued but never consumed must land before the CTA leaves
    if (warp == 0 && lane == 0) {
      if (leader || !kPair)
        for (int i = *consumed_slot; i < issued; ++i) mbar_wait(&full[i % a.stages], (i / a.stages) & 1, nullptr);
      for (int s = 0; s < a.stages; ++s)
        if ((tail_seen >> s) & 1) mbar_wait(&tails[s], (tail_last >> s) & 1, nullptr);
    }
  }
  if constexpr (kPair)
    cluster_sync();  // neither CTA leaves while the pair's MMAs or signals may still touch it
  else
    __syncthreads();
  if (warp == 1) {
    if constexpr (kPair)
      tmem_dealloc_pair(tmem, kTmemCols);
    else
      tmem_dealloc(tmem, kTmemCols);
  }
}

// The tensor map of an operand: cols contiguous, rows ld apart, and with
// groups > 0 a third axis of `stride` elements; boxes of 64 columns, 128-byte
// swizzle. False if the driver refuses it.
bool load_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t ld, uint64_t groups,
              uint64_t stride, uint32_t box_rows) {
  const cuuint64_t dims[3] = {cols, rows, groups}, strides[2] = {ld * 2, stride * 2};
  const cuuint32_t box[3] = {64, box_rows, 1}, one[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, groups ? 3 : 2, const_cast<void*>(base), dims, strides, box,
                     one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <MatmulMode kMode, Form kForm, bool kChained>
cudaError_t launch_chained(const CUtensorMap& ta, const CUtensorMap& tb, const TcArgs& t, long long grid, int cluster,
                         cudaStream_t s) {
  using S = Shape<kMode>;
  auto* kernel = matmul_tc_kernel<kMode, kForm, kChained>;
  const cudaError_t err =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(S::kSmem));
  if (err != cudaSuccess) return err;
  return launch_kernel(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), S::kSmem, s, true,
                       static_cast<unsigned>(cluster), ta, tb, t);
}

// blocks: along the reduction, of the CTA that has most of them (rows modes).
template <MatmulMode kMode, Form kForm>
cudaError_t launch_tiles(const CUtensorMap& ta, const CUtensorMap& tb, const TcArgs& t, int blocks, long long grid,
                         int cluster, cudaStream_t s) {
  if constexpr (!Shape<kMode>::kWeight)
    if (blocks <= chain_blocks(kMode)) return launch_chained<kMode, kForm, false>(ta, tb, t, grid, cluster, s);
  return launch_chained<kMode, kForm, true>(ta, tb, t, grid, cluster, s);
}

struct Problem {
  bool weight, across;  // weight mode; B lies across the reduction
  long long rows;  // tiled rows: of D in all groups, or of one group's D (weight mode)
  int groups, n, blocks;
};

// Row tiles of `tile` rows: as many as there can be, however the rows fall to
// the groups, and as many as expected (half a tile of padding a group).
long long most_tiles(const Problem& q, int tile) {
  const long long t = (q.rows + tile - 1) / tile;
  return q.weight ? t * q.groups : t + q.groups - 1;
}
double expected_tiles(const Problem& q, int tile) {
  if (q.weight || q.groups == 1) return static_cast<double>(most_tiles(q, tile));
  return q.rows / static_cast<double>(tile) + 0.5 * static_cast<double>(std::min<long long>(q.groups, q.rows));
}

// The cut with the least estimated time on the busiest SM, in nanoseconds: a
// block of 64 along the reduction costs what it measured on B200 with all SMs
// busy (2048 rows, 9 column tiles, k 4096 to 8192; forward, wgrad):
//            bn 256     128
//   kPair    370, 433   187, 310
//   kSingle  422, 437   250, 328
// (narrow tiles are bound by the issue of loads and MMAs, wide ones by the
// tensor pipe at the clock that the power limit leaves). A tile costs about
// 500 more, in weight mode no less than its fp32 stores (13 bn), with pairs
// and ragged groups 1700 for the zeroed rows' handshake (2051 tokens in 128
// groups: 256-wide single tiles 170 us, pairs 240); a pair's start 2000, a
// split's exchange 1500 a CTA (clusters of 8 measured 25 us slower than their
// share: few fit beside one another).
//
// Many ragged groups in rows mode take the widest tiles, in pairs from 1024 rows
// a group on: their sizes are not known here, so neither is how the tiles
// fill the last wave (skewed layer, 64 groups of 0 to 1920 rows out of 98304:
// 256-wide pairs and single tiles 187 and 183 us, 192-wide pairs 217; 8 groups
// of about 1000 rows 52, 57 and 61).
MatmulPlan choose_tiles(const Problem& q, int sms) {
  MatmulPlan best{Form::kSingle, kBN, 1, 0};
  if (!q.weight && q.groups > 1 && q.n > kBN / 2 && expected_tiles(q, 256) * ((q.n + kBN - 1) / kBN) > sms) {
    if (q.rows >= 1024LL * q.groups) best.form = Form::kPair;
    return best;
  }
  double least = 1e300;
  auto consider = [&](Form form, int bn, int split, double tiles, int units, double block, double once) {
    const double waves = std::ceil(tiles / units - 1e-9);
    double tile = (q.blocks + split - 1) / split * block + 500;
    if (q.weight) tile = std::max(tile, 13.0 * bn) + (form == Form::kPair && q.groups > 1 ? 1700 : 0);
    const double time = waves * tile + once;
    if (time < least) {
      least = time;
      best = {form, bn, split, 0};
    }
  };
  for (int bn = kBN; bn >= 64; bn -= 32) {
    if (bn - 32 >= q.n && bn > 64) continue;  // wider than the matrix
    const double n_tiles = (q.n + bn - 1) / bn;
    const double pair = q.weight ? 190 + 0.95 * bn : std::max(1.44 * bn, 130 + 0.45 * bn);
    const double single = q.weight ? 217 + 0.86 * bn : std::max(77 + 1.35 * bn, 150 + 0.78 * bn);
    // a B that lies across is loaded in whole boxes of 64 columns
    if (!q.across || bn % 128 == 0) consider(Form::kPair, bn, 1, expected_tiles(q, 256) * n_tiles, sms / 2, pair, 2000);
    if (q.across && bn % 64 != 0) continue;
    consider(Form::kSingle, bn, 1, expected_tiles(q, 128) * n_tiles, sms, single, 0);
    for (int split = 2; split <= 4; split *= 2)
      if (most_tiles(q, 128) * n_tiles * split <= sms && q.blocks >= 2 * split)
        consider(Form::kSplit, bn, split, 1, 1, single, 1500 * split);
  }
  return best;
}

Problem problem_of(MatmulMode mode, const MatmulArgs& a) {
  const bool weight = mode == MatmulMode::kWgrad;
  const int depth = weight ? (a.rows + a.groups - 1) / a.groups : a.k;
  return {weight, mode != MatmulMode::kForward, weight ? a.m : a.rows, a.groups, a.n, (depth + kBK - 1) / kBK};
}

template <MatmulMode kMode>
cudaError_t launch_mode(const MatmulPlan& choice, const MatmulArgs& a, int sms, cudaStream_t s) {
  using S = Shape<kMode>;
  if (encode_fn() == nullptr) return cudaErrorNotSupported;
  const int blocks = problem_of(kMode, a).blocks;
  const bool pair = choice.form == Form::kPair;
  const int tile_m = pair ? 256 : 128, b_cols = pair ? choice.bn / 2 : choice.bn;
  CUtensorMap ta, tb;
  TcArgs t{};
  t.p = a;
  t.bn = choice.bn;
  t.n_tiles = (a.n + t.bn - 1) / t.bn;
  t.stall = take_gemm_stall();
  t.m_tiles = S::kWeight ? (a.m + tile_m - 1) / tile_m : 0;
  t.block_bytes = kABytes + (S::kAcrossB ? (b_cols + 63) / 64 * kBoxBytes : b_cols * kBK * 2);
  t.stages = std::min<int>(kMaxStages, S::kRingBytes / (blocks_per_stage(choice.form) * t.block_bytes));
  const int bytes = S::kWeight ? 4 : 2;
  auto align_of = [&](const void* p, long long ld) {
    const uint64_t u = reinterpret_cast<uintptr_t>(p) | static_cast<uint64_t>(ld) * bytes;
    return u % 32 == 0 ? 32 : u % 16 == 0 ? 16 : bytes;
  };
  t.align_d = align_of(a.d, a.ldd);
  t.align_p = align_of(a.preact, a.ldz);
  t.align_z = align_of(a.z, a.ldz);
  t.align_r = align_of(a.residual, a.ldr);
  bool ok;
  if constexpr (S::kWeight) {
    t.band = 16;
    ok = load_map(&ta, a.a, a.m, a.rows, a.lda, 0, 0, 64) && load_map(&tb, a.b, a.n, a.rows, a.ldb, 0, 0, 64);
  } else {
    // a band of row tiles holds about 64 MB of A, so that it stays in L2 while the weights stream past it
    const long long tile_bytes = 2LL * tile_m * a.k;
    t.band = pair ? 4 : 8;
    while (t.band < (pair ? 16 : 32) && t.band * 2 * tile_bytes <= (64LL << 20)) t.band *= 2;
    constexpr bool fwd = kMode == MatmulMode::kForward;
    ok = load_map(&ta, a.a, a.k, a.rows, a.lda, 0, 0, kBM) &&
         load_map(&tb, a.b, fwd ? a.k : a.n, fwd ? a.n : a.k, a.ldb, a.groups, a.b_stride, fwd ? b_cols : 64);
  }
  if (!ok) return cudaErrorInvalidValue;
  const long long tiles = choice.tiles;
  switch (choice.form) {
    case Form::kPair:
      return launch_tiles<kMode, Form::kPair>(ta, tb, t, blocks, 2 * std::min<long long>(tiles, sms / 2), 2, s);
    case Form::kSplit:
      return launch_tiles<kMode, Form::kSplit>(ta, tb, t, (blocks + choice.split - 1) / choice.split, tiles * choice.split,
                                               choice.split, s);
    default:
      return launch_tiles<kMode, Form::kSingle>(ta, tb, t, blocks, std::min<long long>(tiles, sms), 1, s);
  }
}

}  // namespace

MatmulPlan plan_matmul_tc(MatmulMode mode, const MatmulArgs& a, int sms) {
  const Problem q = problem_of(mode, a);
  MatmulPlan plan = choose_tiles(q, sms);
  plan.tiles = most_tiles(q, plan.form == Form::kPair ? 256 : 128) * ((a.n + plan.bn - 1) / plan.bn);
  return plan;
}

cudaError_t launch_matmul_tc(MatmulMode mode, const MatmulPlan& plan, const MatmulArgs& a, int sms, cudaStream_t s) {
  switch (mode) {
    case MatmulMode::kForward:
      return launch_mode<MatmulMode::kForward>(plan, a, sms, s);
    case MatmulMode::kDgrad:
      return launch_mode<MatmulMode::kDgrad>(plan, a, sms, s);
    default:
      return launch_mode<MatmulMode::kWgrad>(plan, a, sms, s);
  }
}

}  // namespace moe
