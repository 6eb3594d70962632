// linear.cu - matrix product with bias, activation and residual in its epilogue,
// and its gradients.
//   z = x w^T + bias;  y = act(z) + residual
//   dz = dy act'(z);  db = sum over rows of dz;  dx = dz w;  dw = dz^T x
// 16-bit operands, fp32 sums (tcgen05, accumulators in TMEM), each output rounded once.
//
// Two kernels: persistent CTA pairs on 256 x 256 tiles, and single tiles of 128 x 128 or
// 128 x 64 (the weight on the 128 rows where x has few) with the depth of each split
// over a cluster.  Measured (device us; a library's product of the same sizes in
// brackets; 1645.8 TFLOP/s is the measured peak):
//   16384 x 6144 x 4096           535  1.54 PFLOP/s  [546]    in short runs; 620 call after call, at the
//                                                             power limit
//   dx, dw of 16384 x 4096 x 4096 350, 381           [350, 352]  dw: 3.5 waves of tiles
//   777 x 4096 x 4096              28  0.92 PFLOP/s           64 tiles on 74 pairs, start and end of the tile
//   one row, 6144 x 4096         11.8  4.3 TB/s      [11.9]   latency of start and join
//   777 x 1000 x 1112            10.2                [6.2]    latency of start and join
// Tried and slower: the last wave's tiles shared out along the depth over all pairs, the
// parts joined through L2 (dw 433: pairs at different depths share no rows in L2, and
// the join adds 15 us); the last tiles in halves of 128 columns (dw 407, with the
// boxes of 64 rows that takes); tiles of 256 x 128 and 256 x 64.
#include <algorithm>
#include <atomic>

#include "attn_common.cuh"
#include "host_status.h"
#include "layer.cuh"

namespace opr {
namespace {

// The activations bound the epilogues of short products, so they take the fast
// exponential and quotient (a few steps of the last place; 0 and 1 at the ends).
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }

// gelu with tanh: z/2 (1 + tanh u) = z sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3)
constexpr float kGeluC = 0.79788456080286536f, kGeluA = 0.044715f, kSqrtHalf = 0.70710678118654752f,
                kInvSqrt2Pi = 0.39894228040143268f;

// Phi(z), the normal distribution function, and e = exp(-z^2 / 2): with x = |z| / sqrt 2,
// 1 - erf(x) = (a1 t + ... + a5 t^5) e, t = 1 / (1 + p x) (Abramowitz and Stegun 7.1.26,
// within 1.5e-7 of 1: GELU of -3 is off by 5e-5 of its value, of -4 by 5e-4, where 1 + erff
// makes 1e-6 and 3e-4; further out it is the better of the two).  With erff the products
// with this activation took up to 1.2 times as long (dz of 2377 x 4096: 22 against 18 us).
__device__ __forceinline__ float normal(float z, float& e) {
  const float x = fabsf(z) * kSqrtHalf;
  const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
  e = __expf(-x * x);
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  const float tail = 0.5f * p * t * e;  // of the side beyond |z|
  return z < 0.f ? tail : 1.f - tail;
}

__device__ __forceinline__ float activate(float z, int32_t act) {
  if (act == OPR_ACT_SILU) return z * sigmoid(z);
  if (act == OPR_ACT_GELU) {
    float e;
    return z * normal(z, e);
  }
  if (act == OPR_ACT_GELU_TANH) return z * sigmoid(2.f * kGeluC * (z + kGeluA * z * z * z));
  return z;
}

// The slopes have reached 0 or 1 at |z| = 128 in fp32, and further out their terms
// overflow (z^3 from 2^43 on, the infinities at once) and would meet those zeros as NaN:
// z is held to +-128; NaN stays.
__device__ __forceinline__ float activate_slope(float z, int32_t act) {
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(z), "f"(-128.f));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(z) : "f"(z), "f"(128.f));
  if (act == OPR_ACT_SILU) {
    const float s = sigmoid(z);
    return s * (1.f + z * (1.f - s));
  }
  if (act == OPR_ACT_GELU) {
    float e;
    const float phi = normal(z, e);
    return phi + z * kInvSqrt2Pi * e;
  }
  if (act == OPR_ACT_GELU_TANH) {
    const float s = sigmoid(2.f * kGeluC * (z + kGeluA * z * z * z));
    return s * (1.f + 2.f * z * (1.f - s) * kGeluC * (1.f + 3.f * kGeluA * z * z));
  }
  return 1.f;
}

__device__ __forceinline__ bool store_typed(void* p, int32_t dtype, int64_t i, float v) {
  if (dtype == OPR_DTYPE_BF16) {
    static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
  } else if (dtype == OPR_DTYPE_FP16) {
    static_cast<__half*>(p)[i] = __float2half_rn(v);
    return beyond_f16(v);
  } else {
    static_cast<float*>(p)[i] = v;
  }
  return false;
}

// ---------------------------------------------------------------- tiles
// A product is C(p, q) = sum_k P(p, k) Q(q, k): P fills the 128 rows (TMEM lanes)
// of a tile, Q its BN columns.  An operand is K-major (k contiguous) or MN-major
// (its rows contiguous); a 64-deep slice of R rows is staged as
//   K-major   R rows of 128 bytes (64 k), one box
//   MN-major  R / 64 chunks of 64 k-rows of 128 bytes (64 rows of the operand)
// with the 128-byte swizzle.  Boxes past the ends read zeros.
constexpr int kRowsP = 128;
constexpr int kDepth = 64;
constexpr int kChunk = kDepth * 128;  // bytes of an MN-major chunk

// Loads a 64-deep slice of `rows` rows from row0 into dst; PAIR: for a CTA pair, `bar`
// (a shared::cluster address) may be the peer's.  A K-major slice is one box.  An
// MN-major one is a box of all its chunks where the map is of chunks (`folded`, rows a
// multiple of 64), else a box a chunk: every box more in a slice costs the copy engine
// time (a pair's products with four boxes a slice took 1.09 times as long as with two).
template <bool MN, bool PAIR>
__device__ __forceinline__ void load_slice(const CUtensorMap* map, uint32_t bar, uint8_t* dst, int row0, int k0, int rows,
                                           bool folded) {
  auto box = [&](uint8_t* to, int c0, int c1) {
    if constexpr (PAIR)
      asm volatile(
          "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
          " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(to)),
          "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
          : "memory");
    else
      asm volatile(
          "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
          " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(to)),
          "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1)
          : "memory");
  };
  if constexpr (!MN) {
    box(dst, k0, row0);
  } else if (folded) {
    if constexpr (PAIR)
      asm volatile(
          "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
          " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
          "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(k0), "r"(row0 / 64)
          : "memory");
    else
      asm volatile(
          "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
          " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
          "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(0), "r"(k0), "r"(row0 / 64)
          : "memory");
  } else {
    for (int c = 0; c < rows / 64; ++c) box(dst + c * kChunk, row0 + 64 * c, k0);
  }
}

// Descriptor of a staged slice, and its step from 16 k to the next 16 k.
template <bool MN>
__device__ __forceinline__ uint64_t slice_desc(uint32_t saddr) {
  return MN ? smem_desc_sw128(saddr, kChunk, 1024) : smem_desc_sw128(saddr, 16, 1024);
}
template <bool MN>
__device__ __forceinline__ constexpr uint64_t slice_step(int kk) {
  return static_cast<uint64_t>((MN ? kk * 2048 : kk * 32) >> 4);
}

struct ProductArgs {
  int64_t rows_p;
  int32_t rows_q;
  int64_t depth;
  int32_t f16;
  int32_t folded_p, folded_q;  // MN-major operands: the map is of chunks (load_slice)
  int32_t tiles_p, tiles_q;    // tiles along P and, product_pair_kernel only, Q
  int32_t vec;  // the rows of y, z and the residual allow vector accesses
  LinearEpilogue e;
  int32_t* dev_status;
  uint32_t wait_ns;
};

// One output: bias, z, activation, residual, rounding.  Returns whether an fp16
// value overflowed.
__device__ __forceinline__ bool finish(const LinearEpilogue& e, bool f16, int64_t m, int64_t n, float z) {
  bool bad = false;
  if (e.bias != nullptr) z += load_typed(e.bias, e.bias_dtype, n);
  if (e.z != nullptr) bad |= store_typed(e.z, f16 ? OPR_DTYPE_FP16 : OPR_DTYPE_BF16, m * e.ldz + n, z);
  z = activate(z, e.activation);
  if (e.residual != nullptr) z += load_typed(e.residual, e.residual_dtype, m * e.ld_residual + n);
  return store_typed(e.y, e.y_dtype, m * e.ldy + n, z) || bad;
}

// W = 4 or 8 neighbours of a row of type dtype, aligned to W entries of 16 bits (16
// bytes for fp32).
template <int W>
__device__ __forceinline__ void load_row(const void* p, int32_t dtype, int64_t i, float (&v)[W]) {
  if (dtype == OPR_DTYPE_FP32) {
    const float4* f = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int q = 0; q < W / 4; ++q) {
      const float4 x = f[q];
      v[4 * q] = x.x;
      v[4 * q + 1] = x.y;
      v[4 * q + 2] = x.z;
      v[4 * q + 3] = x.w;
    }
    return;
  }
  using Words = std::conditional_t<W == 8, uint4, uint2>;
  const Words u = *reinterpret_cast<const Words*>(static_cast<const uint16_t*>(p) + i);
  const uint32_t* w = reinterpret_cast<const uint32_t*>(&u);
#pragma unroll
  for (int k = 0; k < W / 2; ++k) {
    if (dtype == OPR_DTYPE_BF16) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[k]));
      v[2 * k] = f.x;
      v[2 * k + 1] = f.y;
    }
  }
}

template <int W>
__device__ __forceinline__ bool store_row(void* p, int32_t dtype, int64_t i, const float (&v)[W]) {
  if (dtype == OPR_DTYPE_FP32) {
    float4* f = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
#pragma unroll
    for (int q = 0; q < W / 4; ++q) f[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
    return false;
  }
  using Words = std::conditional_t<W == 8, uint4, uint2>;
  Words u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
  bool bad = false;
#pragma unroll
  for (int k = 0; k < W / 2; ++k) {
    if (dtype == OPR_DTYPE_BF16) {
      w[k] = pack_bf16x2(v[2 * k], v[2 * k + 1]);
    } else {
      w[k] = pack_f16x2(v[2 * k], v[2 * k + 1]);
      bad |= beyond_f16(v[2 * k]) || beyond_f16(v[2 * k + 1]);
    }
  }
  *reinterpret_cast<Words*>(static_cast<uint16_t*>(p) + i) = u;
  return bad;
}

template <int W>
__device__ __forceinline__ void activate_row(float (&v)[W], int32_t act) {
  if (act == OPR_ACT_NONE) return;
  auto each = [&](auto f) {
#pragma unroll
    for (int k = 0; k < W; ++k) v[k] = f(v[k]);
  };
  if (act == OPR_ACT_SILU)
    each([](float z) { return activate(z, OPR_ACT_SILU); });
  else if (act == OPR_ACT_GELU)
    each([](float z) { return activate(z, OPR_ACT_GELU); });
  else
    each([](float z) { return activate(z, OPR_ACT_GELU_TANH); });
}

// W neighbouring outputs of row m (ProductArgs::vec), their bias and residual given.
template <int W>
__device__ __forceinline__ bool finish_row(const LinearEpilogue& e, bool f16, int64_t m, int64_t n, float (&v)[W],
                                           const float (&bias)[W], const float (&residual)[W]) {
  bool bad = false;
#pragma unroll
  for (int k = 0; k < W; ++k) v[k] += bias[k];
  if (e.z != nullptr) bad |= store_row<W>(e.z, f16 ? OPR_DTYPE_FP16 : OPR_DTYPE_BF16, m * e.ldz + n, v);
  activate_row<W>(v, e.activation);
#pragma unroll
  for (int k = 0; k < W; ++k) v[k] += residual[k];
  return store_row<W>(e.y, e.y_dtype, m * e.ldy + n, v) || bad;
}

template <int W>
__device__ __forceinline__ void load_bias(const LinearEpilogue& e, int64_t n, float (&v)[W]) {
#pragma unroll
  for (int k = 0; k < W; ++k) v[k] = 0.f;
  if (e.bias != nullptr) load_row<W>(e.bias, e.bias_dtype, n, v);
}
template <int W>
__device__ __forceinline__ void load_residual(const LinearEpilogue& e, int64_t m, int64_t n, float (&v)[W]) {
#pragma unroll
  for (int k = 0; k < W; ++k) v[k] = 0.f;
  if (e.residual != nullptr) load_row<W>(e.residual, e.residual_dtype, m * e.ld_residual + n, v);
}

// W entries, `step` from one to the next (along a row, or down a column: neighbouring
// lanes take neighbouring columns), those of `in` only: any alignment.  The loads go
// out together.
template <int W>
__device__ __forceinline__ void load_apart(const void* p, int32_t dtype, int64_t i, int64_t step, const bool (&in)[W],
                                           float (&v)[W]) {
  auto each = [&](auto type) {
    using T = decltype(type);
#pragma unroll
    for (int k = 0; k < W; ++k) v[k] = in[k] ? as_float(static_cast<const T*>(p)[i + k * step]) : 0.f;
  };
  if (dtype == OPR_DTYPE_BF16)
    each(__nv_bfloat16{});
  else if (dtype == OPR_DTYPE_FP16)
    each(__half{});
  else
    each(float{});
}
template <int W>
__device__ __forceinline__ bool store_apart(void* p, int32_t dtype, int64_t i, int64_t step, const bool (&in)[W],
                                            const float (&v)[W]) {
  bool bad = false;
  auto each = [&](auto type) {
    using T = decltype(type);
#pragma unroll
    for (int k = 0; k < W; ++k)
      if (in[k]) {
        bad |= beyond<T>(v[k]);
        static_cast<T*>(p)[i + k * step] = from_float<T>(v[k]);
      }
  };
  if (dtype == OPR_DTYPE_BF16)
    each(__nv_bfloat16{});
  else if (dtype == OPR_DTYPE_FP16)
    each(__half{});
  else
    each(float{});
  return bad;
}
// Outputs from (m, n) on, `cols` columns or, where that is 0, one row apart.
template <int W>
__device__ __forceinline__ bool finish_apart(const LinearEpilogue& e, bool f16, int64_t m, int64_t n, int cols,
                                             const bool (&in)[W], float (&v)[W], const float (&bias)[W]) {
  bool bad = false;
  float residual[W] = {};
  if (e.residual != nullptr)
    load_apart<W>(e.residual, e.residual_dtype, m * e.ld_residual + n, cols ? cols : e.ld_residual, in, residual);
#pragma unroll
  for (int k = 0; k < W; ++k) v[k] += bias[k];
  if (e.z != nullptr)
    bad |= store_apart<W>(e.z, f16 ? OPR_DTYPE_FP16 : OPR_DTYPE_BF16, m * e.ldz + n, cols ? cols : e.ldz, in, v);
  activate_row<W>(v, e.activation);
#pragma unroll
  for (int k = 0; k < W; ++k) v[k] += residual[k];
  return store_apart<W>(e.y, e.y_dtype, m * e.ldy + n, cols ? cols : e.ldy, in, v) || bad;
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ float load_peer(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 load_peer4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Limit of a wait for a whole tile: 2 us a slice (six times what one takes) on top of
// the limit of a single wait; 0 stays 0.
__device__ __forceinline__ uint64_t depth_limit(uint64_t wait_ns, int slices) {
  return wait_ns == 0 ? 0 : wait_ns + 2000ull * static_cast<uint64_t>(slices);
}

constexpr int kProductThreads = 320;  // warp 0 TMA, warp 1 MMA, warps 2..9 epilogue
constexpr int kProductSmem = 225 * 1024;
constexpr int kTileSmem = 110 * 1024;  // two CTAs an SM
constexpr int kMaxSplit = 8;

template <bool Q_MN, int BN>
struct TileSmem {
  static constexpr int kRowsQ = Q_MN && BN < 64 ? 64 : BN;  // an MN-major chunk has 64 rows
  static constexpr int kStageBytes = (kRowsP + kRowsQ) * 128;
  static constexpr int kStages = 108 * 1024 / kStageBytes;
  alignas(1024) uint8_t ring[kStages][kStageBytes];
  uint64_t full[kStages], empty[kStages], done;
  uint32_t tmem_base;
  int abort_flag;
};

// One 128 x BN tile per cluster, its depth split over the cluster's CTAs.  Each CTA
// leaves its partial tile (fp32) in its own shared memory, where the ring was; after
// the cluster's barrier each CTA adds up and finishes its share of the tile's lines,
// the partials in rank order (deterministic, no workspace, one launch).  Two CTAs
// share an SM, so that one's epilogue runs next to the other's products.
// SWAP: P holds the n side, Q the m side.
template <bool P_MN, bool Q_MN, int BN, bool SWAP>
__global__ void __launch_bounds__(kProductThreads, 2)
    product_tile_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ ProductArgs a) {
  using Smem = TileSmem<Q_MN, BN>;
  constexpr int kRowsQ = Smem::kRowsQ;
  constexpr int kStages = Smem::kStages;
  constexpr uint32_t kCols = BN < 32 ? 32 : BN;
  // floats from line to line of the partial tile: lines along the contiguous
  // direction of y, 16-byte accesses without bank conflicts
  constexpr int kLines = SWAP ? BN : kRowsP, kLine = SWAP ? kRowsP : BN, kLineLd = kLine + 4;
  static_assert(kLines * kLineLd * 4 <= static_cast<int>(sizeof(Smem::ring)), "the partial tile fits where the ring was");
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(align1024(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank(), ranks = cluster_size();
  const int tile = static_cast<int>(blockIdx.x / ranks);
  const int64_t p0 = static_cast<int64_t>(tile % a.tiles_p) * kRowsP;
  const int q0 = tile / a.tiles_p * BN;
  const int64_t slices = (a.depth + kDepth - 1) / kDepth;
  const int s0 = static_cast<int>(slices * rank / ranks), s1 = static_cast<int>(slices * (rank + 1) / ranks);
  const int n = s1 - s0;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&map_p);
    tma_prefetch_desc(&map_q);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.done, 1);
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc(&sm.tmem_base, kCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;
  wait_for_previous();

  if (warp == 0) {
    if (lane == 0) {
      constexpr uint32_t kBytes = Smem::kStageBytes;
      int issued = 0;
      for (int j = 0; j < n; ++j) {
        const int s = j % kStages;
        if (j >= kStages && !mbar_wait(&sm.empty[s], ((j / kStages) + 1) & 1, abort_flag, a.wait_ns)) break;
        mbar_arrive_expect_tx(&sm.full[s], kBytes);
        load_slice<P_MN, false>(&map_p, smem_u32(&sm.full[s]), sm.ring[s], static_cast<int>(p0), (s0 + j) * kDepth, kRowsP,
                                a.folded_p != 0);
        load_slice<Q_MN, false>(&map_q, smem_u32(&sm.full[s]), sm.ring[s] + kRowsP * 128, q0, (s0 + j) * kDepth, kRowsQ,
                                a.folded_q != 0);
        issued = j + 1;
      }
      // every copy issued has landed before the CTA goes on (also after an abort)
      for (int j = (issued > kStages ? issued - kStages : 0); j < issued; ++j)
        mbar_wait(&sm.full[j % kStages], (j / kStages) & 1, nullptr, kWaitLimitNs);
    }
  } else if (warp == 1) {
    const uint32_t idesc = idesc_f32acc(kRowsP, BN, a.f16 != 0, P_MN, Q_MN);
    for (int j = 0; j < n; ++j) {
      const int s = j % kStages;
      if (!warp_wait(&sm.full[s], (j / kStages) & 1, abort_flag, a.wait_ns)) break;
      tc_fence_after();
      const uint32_t sa = smem_u32(sm.ring[s]);
      const uint64_t dp = slice_desc<P_MN>(sa), dq = slice_desc<Q_MN>(sa + kRowsP * 128);
#pragma unroll
      for (int kk = 0; kk < kDepth / 16; ++kk)
        mma_ss(tmem, dp + slice_step<P_MN>(kk), dq + slice_step<Q_MN>(kk), idesc, (j | kk) != 0 ? 1u : 0u);
      mma_commit(&sm.empty[s]);
    }
    mma_commit(&sm.done);
    if (!warp_wait(&sm.done, 0, nullptr, kWaitLimitNs)) *abort_flag = 1;
  }
  __syncthreads();  // the producer's copies have landed, the products are complete
  const bool aborted = *abort_flag != 0;
  tc_fence_after();
  float* part = reinterpret_cast<float*>(sm.ring);
  if (warp >= 2) {
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const int row = quad * 32 + lane;
    for (int c = half * 16; c < BN; c += 32) {
      uint32_t r[16];
      tmem_ld16(tl + c, r);
      if constexpr (SWAP) {
#pragma unroll
        for (int i = 0; i < 16; ++i) part[(c + i) * kLineLd + row] = __uint_as_float(r[i]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(part + row * kLineLd + c + 4 * i) =
              make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
      }
    }
    tc_fence_before();
  }
  if (ranks > 1)
    cluster_sync();
  else
    __syncthreads();
  // line i of the tile is row m0 + i of y, entry j of a line its column n0 + j
  const int64_t m0 = SWAP ? q0 : p0, n0 = SWAP ? p0 : q0;
  const int64_t rows = SWAP ? a.rows_q : a.rows_p, cols = SWAP ? a.rows_p : a.rows_q;
  const int lines = rows - m0 < kLines ? static_cast<int>(rows - m0) : kLines;
  const int len = cols - n0 < kLine ? static_cast<int>(cols - n0) : kLine;
  const uint32_t base = smem_u32(part);
  uint32_t peer[kMaxSplit];
#pragma unroll
  for (int r = 0; r < kMaxSplit; ++r) peer[r] = peer_addr(base, r < static_cast<int>(ranks) ? r : 0);
  bool bad = false;
  if (a.vec) {
    constexpr int kQuads = kLine / 4;  // groups of four neighbours of a line
    for (int i = threadIdx.x + static_cast<int>(rank) * kProductThreads; i < lines * kQuads;
         i += static_cast<int>(ranks) * kProductThreads) {
      const int line = i / kQuads, j = i % kQuads * 4;
      if (j >= len) continue;
      float bias[4], residual[4];
      load_bias<4>(a.e, n0 + j, bias);
      load_residual<4>(a.e, m0 + line, n0 + j, residual);
      const uint32_t at = 4 * (line * kLineLd + j);
      float4 v;
      if (ranks == 1) {
        v = *reinterpret_cast<const float4*>(part + line * kLineLd + j);
      } else {
        v = load_peer4(peer[0] + at);
#pragma unroll
        for (int r = 1; r < kMaxSplit; ++r) {
          if (r >= static_cast<int>(ranks)) break;
          const float4 x = load_peer4(peer[r] + at);
          v.x += x.x;
          v.y += x.y;
          v.z += x.z;
          v.w += x.w;
        }
      }
      float f[4] = {v.x, v.y, v.z, v.w};
      bad |= finish_row<4>(a.e, a.f16 != 0, m0 + line, n0 + j, f, bias, residual);
    }
  } else {
    // a line of 128 entries to 32 lanes, one of 64 to 16
    constexpr int kLanes = kLine / 4, kTeams = kProductThreads / kLanes;
    const int team = threadIdx.x / kLanes, j = threadIdx.x % kLanes;
    bool in[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) in[k] = j + kLanes * k < len;
    float bias[4] = {};
    if (a.e.bias != nullptr) load_apart<4>(a.e.bias, a.e.bias_dtype, n0 + j, kLanes, in, bias);
    for (int line = team + static_cast<int>(rank) * kTeams; line < lines && in[0]; line += static_cast<int>(ranks) * kTeams) {
      float f[4] = {};
#pragma unroll
      for (int r = 0; r < kMaxSplit; ++r) {
        if (r >= static_cast<int>(ranks)) break;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (in[k]) f[k] += load_peer(peer[r] + 4 * (line * kLineLd + j + kLanes * k));
      }
      bad |= finish_apart<4>(a.e, a.f16 != 0, m0 + line, n0 + j, kLanes, in, f, bias);
    }
  }
  if (bad) atomicOr(a.dev_status, OPR_DEV_FP16_RANGE);
  if (aborted && threadIdx.x == 0) atomicOr(a.dev_status, OPR_DEV_WAIT_TIMEOUT);
  if (ranks > 1) cluster_sync();  // no CTA ends while another reads its shared memory
  if (warp == 1) tmem_dealloc(tmem, kCols);
}

// ---------------------------------------------------------------- large products
// Persistent CTA pairs: one 256 x 256 tile at a time per pair (cta_group::2), each
// CTA staging its own 128 rows of P and 128 of Q, so that a pair reads each staged
// byte once where two CTAs of their own would read Q twice (at the tensor cores' full rate
// an SM then takes in 64 bytes a clock; with tiles of 256 x 128 96, and those and 256 x 64
// were never the fastest).  Few tiles leave pairs idle: 2377 x 1024 over 4096 are 40 tiles,
// and its 28 us have the tensor pipes of those 80 SMs active 59 % of the time, the fetches
// from L2 at a third of their ports.  Two accumulators: the epilogue of a tile runs while the
// next one is multiplied.
constexpr int kPairTile = 256;
constexpr int kEpiWarps = 8;
constexpr int kWarpStage = 4096;  // bytes a warp stages its outputs in: two 32 x 32 blocks of 16 bits, or one of 32

struct PairSmem {
  static constexpr int kStageBytes = 2 * kRowsP * 128;
  static constexpr int kStages = 5;
  alignas(1024) uint8_t ring[kStages][kStageBytes];
  alignas(1024) uint8_t stage[kEpiWarps][kWarpStage];
  alignas(16) float bias[kEpiWarps][kRowsP];
  uint64_t full[kStages], empty[kStages];  // full: the leader's, counts both CTAs' bytes
  uint64_t acc_full[2], acc_empty[2];      // acc_empty: the leader's
  uint64_t done;
  uint32_t tmem_base;
  int abort_flag;
  int issued;
};
static_assert(sizeof(PairSmem) + 1024 <= kProductSmem, "the ring and the staging fit an SM");

__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred E, P;\n\t"
      "elect.sync _|E, 0xffffffff;\n\t"
      "setp.ne.b32 P, %4, 0;\n\t"
      "@E tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, P;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrives on `bar` of both CTAs when the MMAs issued so far are complete.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred E;\n\t"
      "elect.sync _|E, 0xffffffff;\n\t"
      "@E tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::
          "r"(smem_u32(bar)),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}

// Stores a 32 x 32 block staged by a warp (one lane calls), as one bulk group.
__device__ __forceinline__ void store_block(const CUtensorMap* map, const uint8_t* from, int n, int m) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(from)), "r"(n), "r"(m)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Until all but kLeft of this lane's groups have read their shared memory.
template <int kLeft>
__device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}

// A lane's row of 32 values into a staged block, in the swizzle of the block's map:
// 16 bits in 64-byte rows, 32 bits in 128-byte rows; without bank conflicts.
__device__ __forceinline__ void stage_row16(uint8_t* block, int row, const float (&v)[32], bool f16, bool& bad) {
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float lo = v[8 * g + 2 * k], hi = v[8 * g + 2 * k + 1];
      w[k] = f16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi);
    }
    *reinterpret_cast<uint4*>(block + row * 64 + ((g ^ (row >> 1)) & 3) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (f16) {
    float top = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      top = fmaxf(top, fabsf(v[i]));
      nan |= v[i] != v[i];
    }
    bad |= nan || beyond_f16(top);
  }
}
__device__ __forceinline__ void stage_row32(uint8_t* block, int row, const float (&v)[32]) {
#pragma unroll
  for (int g = 0; g < 8; ++g)
    *reinterpret_cast<float4*>(block + row * 128 + ((g ^ row) & 7) * 16) =
        make_float4(v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]);
}

// Finishes a lane's column of a block staged by stage_row32, eight rows at a time.  A
// call of its own: its code would slow the epilogue that it stands in.
__device__ __noinline__ bool finish_column(const LinearEpilogue& e, bool f16, int64_t m, int64_t n, int rows,
                                           const uint8_t* block, int lane, float bias) {
  bool bad = false;
  float b8[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) b8[k] = bias;
#pragma unroll 1
  for (int row = 0; row < rows; row += 8) {
    bool in[8];
    float f[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      in[k] = row + k < rows;
      f[k] = *reinterpret_cast<const float*>(block + (row + k) * 128 + (((lane >> 2) ^ (row + k)) & 7) * 16 + (lane & 3) * 4);
    }
    bad |= finish_apart<8>(e, f16, m + row, n, 0, in, f, b8);
  }
  return bad;
}

// A lane's row of a residual block, as loaded; columns past the end (a multiple of
// eight) are not read.
struct RawRow {
  uint4 v[8];
};
__device__ __forceinline__ void fetch_residual(const LinearEpilogue& e, int64_t m, int64_t n0, int32_t cols, RawRow& raw) {
  const bool wide = e.residual_dtype == OPR_DTYPE_FP32;
  const int per = wide ? 4 : 8;  // entries of 16 bytes
  const char* p = static_cast<const char*>(e.residual) + (m * e.ld_residual + n0) * (wide ? 4 : 2);
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    raw.v[g] = make_uint4(0, 0, 0, 0);
    if ((wide || g < 4) && n0 + per * g < cols) raw.v[g] = reinterpret_cast<const uint4*>(p)[g];
  }
}
__device__ __forceinline__ void add_residual(const RawRow& raw, int32_t dtype, float (&v)[32]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(raw.v);
  if (dtype == OPR_DTYPE_FP32) {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += __uint_as_float(w[i]);
  } else if (dtype == OPR_DTYPE_BF16) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[2 * i] += __uint_as_float(w[i] << 16);
      v[2 * i + 1] += __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] += f.x;
      v[2 * i + 1] += f.y;
    }
  }
}

// Tile t of the walk: groups of kGroup tile rows, columns outer inside a group, so
// that the pairs that run together share rows of P and Q in L2.
constexpr int kGroup = 8;
__device__ __forceinline__ void tile_at(int t, int tiles_p, int tiles_q, int& tp, int& tq) {
  const int per = kGroup * tiles_q;
  const int g = t / per, r = t % per;
  const int rows = tiles_p - g * kGroup < kGroup ? tiles_p - g * kGroup : kGroup;
  tp = g * kGroup + r % rows;
  tq = r / rows;
}

template <bool P_MN, bool Q_MN>
__global__ void __launch_bounds__(kProductThreads, 1) __cluster_dims__(2, 1, 1)
    product_pair_kernel(const __grid_constant__ CUtensorMap map_p, const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_y, const __grid_constant__ CUtensorMap map_z,
                        const __grid_constant__ ProductArgs a) {
  extern __shared__ uint8_t smem_raw[];
  using Smem = PairSmem;
  constexpr int kStages = Smem::kStages, BN = kPairTile;
  Smem& sm = *reinterpret_cast<Smem*>(align1024(smem_raw));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int slices = static_cast<int>((a.depth + kDepth - 1) / kDepth);
  const int tiles = a.tiles_p * a.tiles_q;
  const int pairs = gridDim.x / 2, first = blockIdx.x / 2;

  if (threadIdx.x == 0) {
    tma_prefetch_desc(&map_p);
    tma_prefetch_desc(&map_q);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], 2 * kEpiWarps);
    }
    mbar_init(&sm.done, 1);
    sm.abort_flag = 0;
    sm.issued = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // the peer's barriers are set up
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  volatile int* abort_flag = &sm.abort_flag;
  wait_for_previous();

  auto fill = [&](int j, int tp, int tq, int slice) {
    const int s = j % kStages;
    // the leader's barrier counts both CTAs' bytes of the stage
    if (rank == 0) mbar_arrive_expect_tx(&sm.full[s], 2 * Smem::kStageBytes);
    const uint32_t bar = peer_addr(smem_u32(&sm.full[s]), 0);
    load_slice<P_MN, true>(&map_p, bar, sm.ring[s], tp * kPairTile + static_cast<int>(rank) * kRowsP, slice * kDepth, kRowsP,
                           a.folded_p != 0);
    load_slice<Q_MN, true>(&map_q, bar, sm.ring[s] + kRowsP * 128, tq * kPairTile + static_cast<int>(rank) * kRowsP,
                           slice * kDepth, kRowsP, a.folded_q != 0);
  };

  if (warp == 0) {
    if (lane == 0) {
      int j = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += pairs) {
        int tp, tq;
        tile_at(t, a.tiles_p, a.tiles_q, tp, tq);
        for (int k = 0; k < slices; ++k, ++j) {
          if (j >= kStages &&
              !mbar_wait(&sm.empty[j % kStages], ((j / kStages) + 1) & 1, abort_flag, a.wait_ns)) {
            ok = false;
            break;
          }
          fill(j, tp, tq, k);
        }
      }
      sm.issued = j;
      // the releases of the last stages, which the leader's MMAs send here
      for (int u = j > kStages ? j - kStages : 0; ok && u < j; ++u)
        ok = mbar_wait(&sm.empty[u % kStages], (u / kStages) & 1, abort_flag, a.wait_ns);
    }
  } else if (warp == 1) {
    if (rank == 0) {
      const uint32_t idesc = idesc_f32acc(kPairTile, BN, a.f16 != 0, P_MN, Q_MN);
      int j = 0, i = 0;
      bool ok = true;
      for (int t = first; ok && t < tiles; t += pairs, ++i) {
        const int b = i & 1;
        if (i >= 2) ok = warp_wait(&sm.acc_empty[b], ((i >> 1) + 1) & 1, abort_flag, a.wait_ns);
        tc_fence_after();
        for (int k = 0; ok && k < slices; ++k, ++j) {
          const int s = j % kStages;
          ok = warp_wait(&sm.full[s], (j / kStages) & 1, abort_flag, a.wait_ns);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = smem_u32(sm.ring[s]);
          const uint64_t dp = slice_desc<P_MN>(sa), dq = slice_desc<Q_MN>(sa + kRowsP * 128);
#pragma unroll
          for (int kk = 0; kk < kDepth / 16; ++kk)
            mma_pair(tmem + b * BN, dp + slice_step<P_MN>(kk), dq + slice_step<Q_MN>(kk), idesc,
                     (k | kk) != 0 ? 1u : 0u);
          commit_pair(&sm.empty[s]);
        }
        if (ok) commit_pair(&sm.acc_full[b]);
      }
      // the releases of the last accumulators, which the peer sends here, and the last MMA
      for (int u = i > 2 ? i - 2 : 0; ok && u < i; ++u)
        ok = warp_wait(&sm.acc_empty[u & 1], (u >> 1) & 1, abort_flag, a.wait_ns);
      asm volatile(
          "{\n\t.reg .pred E;\n\t"
          "elect.sync _|E, 0xffffffff;\n\t"
          "@E tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(
              smem_u32(&sm.done))
          : "memory");
      if (!warp_wait(&sm.done, 0, nullptr, kWaitLimitNs)) *abort_flag = 1;
    }
  } else {
    // A warp finishes 32 rows (one a lane) x 128 columns of the CTA's tile in chunks of
    // 32 columns: in registers, then staged and stored by TMA, which leaves the ends off.
    const int quad = warp & 3, half = (warp - 2) >> 2;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    uint8_t* stage = sm.stage[warp - 2];
    float* bias = sm.bias[warp - 2];
    const LinearEpilogue& e = a.e;
    const bool f16 = a.f16 != 0, y32 = e.y_dtype == OPR_DTYPE_FP32, y16 = e.y_dtype == OPR_DTYPE_FP16;
    bool bad = false;
    int i = 0;
    uint32_t turn = 0;  // blocks of 16 bits staged so far
    // the block to stage next, free again (two take turns; a 32-bit one takes both)
    auto block16 = [&]() {
      if (lane == 0) {
        if (y32)
          stores_read<0>();
        else
          stores_read<1>();
      }
      __syncwarp();
      return stage + (y32 ? 0 : (turn++ & 1) * (kWarpStage / 2));
    };
    auto send = [&](const CUtensorMap* map, const uint8_t* block, int64_t n, int64_t m) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) store_block(map, block, static_cast<int>(n), static_cast<int>(m));
    };
    for (int t = first; t < tiles; t += pairs, ++i) {
      const int b = i & 1;
      int tp, tq;
      tile_at(t, a.tiles_p, a.tiles_q, tp, tq);
      const int64_t m0 = static_cast<int64_t>(tp) * kPairTile + rank * kRowsP + quad * 32;
      const int64_t nb = static_cast<int64_t>(tq) * kPairTile + half * kRowsP;
      const int64_t m = m0 + lane;
      const bool in_m = m0 < a.rows_p;
      if (e.bias != nullptr) {
        __syncwarp();
        for (int k = lane; k < kRowsP; k += 32) bias[k] = nb + k < a.rows_q ? load_typed(e.bias, e.bias_dtype, nb + k) : 0.f;
        __syncwarp();
      }
      // the residual comes one chunk ahead, the first while the products still run
      RawRow raw;
      const bool res = a.vec && e.residual != nullptr && m < a.rows_p;
      if (res && nb < a.rows_q) fetch_residual(e, m, nb, a.rows_q, raw);
      if (!warp_wait(&sm.acc_full[b], (i >> 1) & 1, abort_flag, depth_limit(a.wait_ns, slices))) break;
      tc_fence_after();
      const uint32_t acc = tl + b * BN + half * kRowsP;
#pragma unroll 1
      for (int c = 0; c < kRowsP / 32; ++c) {
        const int64_t n0 = nb + 32 * c;
        uint32_t r[32];
        tmem_ld32(acc + 32 * c, r);
        if (c + 1 == kRowsP / 32) {  // this warp has read its part of the accumulator
          tc_fence_before();
          if (lane == 0)
            asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                             peer_addr(smem_u32(&sm.acc_empty[b]), 0))
                         : "memory");
        }
        if (!in_m || n0 >= a.rows_q) continue;
        float v[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k]);
        if (!a.vec) {  // rows of y, z or the residual off the 16-byte grid: a lane a column
          __syncwarp();
          stage_row32(stage, lane, v);
          __syncwarp();
          const int rows = a.rows_p - m0 < 32 ? static_cast<int>(a.rows_p - m0) : 32;
          if (n0 + lane < a.rows_q)
            bad |= finish_column(e, f16, m0, n0 + lane, rows, stage, lane, e.bias != nullptr ? bias[32 * c + lane] : 0.f);
          continue;
        }
        if (e.bias != nullptr) {
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            const float4 x = reinterpret_cast<const float4*>(bias + 32 * c)[g];
            v[4 * g] += x.x;
            v[4 * g + 1] += x.y;
            v[4 * g + 2] += x.z;
            v[4 * g + 3] += x.w;
          }
        }
        if (e.z != nullptr) {
          uint8_t* block = block16();
          bool over = false;
          stage_row16(block, lane, v, f16, over);
          bad |= over && m < a.rows_p;
          send(&map_z, block, n0, m0);
        }
        activate_row<32>(v, e.activation);
        if (res) {
          add_residual(raw, e.residual_dtype, v);
          if (c + 1 < kRowsP / 32 && n0 + 32 < a.rows_q) fetch_residual(e, m, n0 + 32, a.rows_q, raw);
        }
        uint8_t* block = block16();
        if (y32) {
          stage_row32(block, lane, v);
        } else {
          bool over = false;
          stage_row16(block, lane, v, y16, over);
          bad |= over && m < a.rows_p;
        }
        send(&map_y, block, n0, m0);
      }
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (bad) atomicOr(a.dev_status, OPR_DEV_FP16_RANGE);
  }
  __syncthreads();
  cluster_sync();
  // After an abort the two producers may have stopped at different slices: the one
  // behind catches up (no MMA reads the ring any more), so that the leader's
  // barriers, which count both, say when every copy of both CTAs has landed.
  if (threadIdx.x == 0) {
    const int mine = sm.issued;
    int theirs;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(theirs) : "r"(peer_addr(smem_u32(&sm.issued), rank ^ 1u)));
    const int upto = mine > theirs ? mine : theirs;
    for (int j = mine; j < upto; ++j) fill(j, 0, 0, 0);
    if (rank == 0)
      for (int j = upto > kStages ? upto - kStages : 0; j < upto; ++j)
        mbar_wait(&sm.full[j % kStages], (j / kStages) & 1, nullptr, kWaitLimitNs);
    if (*abort_flag != 0) atomicOr(a.dev_status, OPR_DEV_WAIT_TIMEOUT);
  }
  __syncthreads();
  cluster_sync();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// Nothing to add up (the gradient of a weight over no rows): the epilogue of zeros.
__global__ void __launch_bounds__(256) no_depth_kernel(const __grid_constant__ ProductArgs a) {
  const int64_t n = a.rows_p * a.rows_q;
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < n;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x)
    finish(a.e, a.f16 != 0, i / a.rows_q, i % a.rows_q, 0.f);
}

// Matrices whose rows start off the 16-byte grid, copied to rows that start on it: a
// warp a row at a time, in 16-byte pieces of the copy, each shifted together from the
// two 16-byte pieces of the row that it lies across.  Far below the memory's rate at
// the sizes it is met with (1780 rows of 1111: 6 us for 8 MB, by itself, caches cold).
struct PackArgs {
  const uint16_t* x[2];
  uint16_t* y[2];
  int64_t ldx[2], ldy[2], rows[2];
  int32_t cols[2];
};
__global__ void __launch_bounds__(256) pack_kernel(const PackArgs a) {
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * 8;
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5); r < a.rows[0] + a.rows[1]; r += warps) {
    const bool one = r < a.rows[0];
    const int64_t row = one ? r : r - a.rows[0];
    const uint16_t* x = one ? a.x[0] + row * a.ldx[0] : a.x[1] + row * a.ldx[1];
    uint16_t* y = one ? a.y[0] + row * a.ldy[0] : a.y[1] + row * a.ldy[1];
    const int cols = one ? a.cols[0] : a.cols[1];
    // bytes that the row starts behind the grid, alike for all lanes
    const int off = static_cast<int>(reinterpret_cast<uintptr_t>(x) & 15u);
    const uint4* grid = reinterpret_cast<const uint4*>(reinterpret_cast<uintptr_t>(x) - off);
    // c: entry of the row that a piece of the copy begins with (a count of bytes would
    // pass 32 bits in the longest rows)
#pragma unroll 2
    for (int64_t c = 8 * lane; c < cols; c += 256) {
      const int64_t left = cols - c;
      // pieces that hold a byte of the row (a piece never leaves the row's allocation)
      const uint4 a0 = grid[c / 8];
      const uint4 a1 = off != 0 && 16 - off < 2 * left ? grid[c / 8 + 1] : make_uint4(0, 0, 0, 0);
      const uint32_t w[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
      uint32_t v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t lo = w[k], hi = w[k + 1];
        if (off >= 4) lo = w[k + 1], hi = w[k + 2];
        if (off >= 8) lo = w[k + 2], hi = w[k + 3];
        if (off >= 12) lo = w[k + 3], hi = k < 3 ? w[k + 4] : w[7];
        v[k] = (off & 2) != 0 ? __funnelshift_r(lo, hi, 16) : lo;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)  // zeros behind the row
        if (left < 2 * k + 2) v[k] = left > 2 * k ? v[k] & 0xFFFFu : 0u;
      *reinterpret_cast<uint4*>(y + c) = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
}

// dz = dy act'(z) (written when dz is not null) and the column sums of each block's
// rows, taken before dz is rounded.  A thread takes W neighbouring columns (eight
// where the rows allow 16-byte accesses, else one); the block's 256 threads are `wide`
// column groups times 256 / wide rows, whose sums are added in order at the end.
// dy and z are read once, dz written once (2377 x 4096 with SiLU and db: 13.1 us by itself,
// caches cold, for 58 MB, 4.5 TB/s, and 5 for the column sums' second kernel; holding z
// within the slopes' range is 5 % of it).
constexpr int kDzThreads = 256;
constexpr int kDzSpan = 32;      // column groups of a block
constexpr int kDzRows = kDzThreads / kDzSpan;  // rows at a time
constexpr int kDzMaxBlocks = 512;  // row blocks that fill the GPU, at most
constexpr int kDzMaxRun = 256;     // entries that a thread adds in fp32 at most; longer columns take more row blocks,
                                   // whose sums are added in fp64 (a chain of 4096 lost 2^-13 of its sum)

template <typename T, int W>
__global__ void __launch_bounds__(kDzThreads, 4) linear_dz_kernel(const T* dy, int64_t ld_dy, const T* z, int64_t ldz, int64_t m,
                                                               int32_t n, int32_t act, T* dz, int64_t ld_dz, float* partial,
                                                               int64_t rows_per_block, int32_t* dev_status) {
  constexpr int32_t kType = std::is_same_v<T, __half> ? OPR_DTYPE_FP16 : OPR_DTYPE_BF16;
  constexpr int kRows = kDzRows;
  __shared__ float sums[kRows][kDzSpan * W + 1];
  const int col = threadIdx.x % kDzSpan, row = threadIdx.x / kDzSpan;
  const int64_t j = (static_cast<int64_t>(blockIdx.x) * kDzSpan + col) * W;
  const int64_t row_block = blockIdx.y + static_cast<int64_t>(gridDim.y) * blockIdx.z;
  const int64_t r0 = row_block * rows_per_block;
  const int64_t r1 = r0 + rows_per_block < m ? r0 + rows_per_block : m;
  float sum[W] = {};
  bool bad = false;
  wait_for_previous();
  if (j < n) {
#pragma unroll 2
    for (int64_t i = r0 + row; i < r1; i += kRows) {
      float g[W];
      if constexpr (W == 1)
        g[0] = as_float(dy[i * ld_dy + j]);
      else
        load_row<W>(dy, kType, i * ld_dy + j, g);
      if (act != OPR_ACT_NONE) {
        float v[W];
        if constexpr (W == 1)
          v[0] = as_float(z[i * ldz + j]);
        else
          load_row<W>(z, kType, i * ldz + j, v);
        // __fmul_rn: one value for the sum and for dz, whether or not dz is wanted
        auto each = [&](auto slope) {
#pragma unroll
          for (int k = 0; k < W; ++k) g[k] = __fmul_rn(g[k], slope(v[k]));
        };
        if (act == OPR_ACT_SILU)
          each([](float x) { return activate_slope(x, OPR_ACT_SILU); });
        else if (act == OPR_ACT_GELU)
          each([](float x) { return activate_slope(x, OPR_ACT_GELU); });
        else
          each([](float x) { return activate_slope(x, OPR_ACT_GELU_TANH); });
      }
#pragma unroll
      for (int k = 0; k < W; ++k) sum[k] += g[k];
      if (dz != nullptr) {
        if constexpr (W == 1)
          bad |= store_typed(dz, kType, i * ld_dz + j, g[0]);
        else
          bad |= store_row<W>(dz, kType, i * ld_dz + j, g);
      }
    }
  }
  if (bad && dev_status != nullptr) atomicOr(dev_status, OPR_DEV_FP16_RANGE);
  if (partial == nullptr || r0 >= m) return;  // r0 >= m: blocks behind the last rows, of a grid with more than one z
#pragma unroll
  for (int k = 0; k < W; ++k) sums[row][col * W + k] = sum[k];
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kDzSpan * W;
  for (int c = threadIdx.x; c < kDzSpan * W && first + c < n; c += kDzThreads) {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < kRows; ++r) t += sums[r][c];
    partial[row_block * n + first + c] = t;
  }
}

// Sums of the row blocks' partials, 32 columns a block, eight threads to a column,
// added in a fixed order in fp64.  37 partials of 4096 columns: 5 us by
// itself, caches cold.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* partial, int32_t blocks, int32_t n, float* out) {
  __shared__ double sums[8][33];
  const int col = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int64_t j = static_cast<int64_t>(blockIdx.x) * 32 + col;
  double t = 0.0;
  wait_for_previous();
  if (j < n)
#pragma unroll 8
    for (int b = part; b < blocks; b += 8) t += partial[static_cast<int64_t>(b) * n + j];
  sums[part][col] = t;
  __syncthreads();
  if (part != 0 || j >= n) return;
  for (int p = 1; p < 8; ++p) t += sums[p][col];
  out[j] = static_cast<float>(t);
}

}  // namespace

namespace {

// A 16-bit operand as a map of slices of `box_rows` rows, 64 deep, 128-byte swizzle:
// of rows and depth, or folded (set to 1) of an MN-major operand's chunks of 64 rows.
bool operand_map(CUtensorMap* map, const Operand& o, int64_t rows, int64_t depth, bool f16, int box_rows,
                 int32_t* folded) {
  const bool mn = o.col != 1;
  const auto type = f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const cuuint64_t pitch = static_cast<cuuint64_t>(mn ? o.col : o.row) * 2;
  const cuuint32_t estr[3] = {1, 1, 1};
  *folded = mn && rows % 64 == 0;
  if (*folded) {
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(depth), static_cast<cuuint64_t>(rows / 64)};
    const cuuint64_t strides[2] = {pitch, 128};
    const cuuint32_t box[3] = {64, kDepth, static_cast<cuuint32_t>(box_rows / 64)};
    return encode_tiled(map, type, 3, const_cast<void*>(o.p), dims, strides, box, estr, CU_TENSOR_MAP_SWIZZLE_128B);
  }
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(mn ? rows : depth), static_cast<cuuint64_t>(mn ? depth : rows)};
  const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(mn ? kDepth : box_rows)};
  return encode_tiled(map, type, 2, const_cast<void*>(o.p), dims, &pitch, box, estr, CU_TENSOR_MAP_SWIZZLE_128B);
}

// An output matrix as a map of the 32 x 32 blocks that a warp stages.
bool block_map(CUtensorMap* map, void* p, int64_t ld, int32_t dtype, int64_t rows, int64_t cols) {
  const bool wide = dtype == OPR_DTYPE_FP32;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld) * (wide ? 4 : 2)};
  const cuuint32_t box[2] = {32, 32};
  const cuuint32_t estr[2] = {1, 1};
  return encode_tiled(map, wide                       ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                           : dtype == OPR_DTYPE_FP16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                     : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      2, p, dims, strides, box, estr, wide ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

// Lets a kernel use `bytes` of shared memory, once per device and kernel.
template <auto* kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> allowed{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = uint64_t{1} << (dev & 63);
  if (dev < 64 && (allowed.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) allowed.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Do all rows of y, z and the residual start on 16-byte boundaries?
bool rows_aligned(const LinearEpilogue& e) {
  auto fits = [](const void* p, int64_t ld) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0);
  };
  return fits(e.y, e.ldy) && fits(e.z, e.ldz) && fits(e.residual, e.ld_residual);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// CTAs of two to an SM that run at one time in clusters of 1 .. 8 (B200: 148 SMs,
// the clusters within its GPCs; as the occupancy query reports them).
constexpr int kSlots[kMaxSplit] = {296, 296, 279, 284, 280, 270, 259, 264};

// Time (us) of a product in 128 x BN tiles with the depth of each split over the
// least costly number of CTAs, which comes back in `split`; the 5 us or so that any
// product takes left out.  As measured over 128 to 16384 rows, 144 to 4096 columns and
// 64 to 65536 deep:
//   a 64-deep slice of a CTA that has its SM to itself   0.30 (BN 64)  0.44 (BN 128)
//   of two that share one, each                          0.44          0.54
//   joining c parts, each past the first                 0.1 .. 0.6    0.25 .. 1.1
//   (with the CTAs that read one another's at one time)
//   the epilogue of each tile of an SM past the first    1.6           2.9
// Other widths (BN 16) are taken as 64.
double tile_cost(int64_t tiles, int64_t slices, int bn, int* split) {
  const bool wide = bn == 128;
  double best = 0.0;
  for (int c = 1; c <= kMaxSplit; ++c) {
    const int64_t ctas = tiles * c;
    if (c > 1 && (ctas > kSlots[c - 1] || slices < 4 * c)) continue;
    const double each = static_cast<double>(slices) / c, own = wide ? 0.44 : 0.30, two = wide ? 0.54 : 0.44;
    double t = ctas <= 148 ? each * own : std::max(each * two, ctas * each / 148 * two / 2);
    t += (c - 1) * (wide ? 0.25 + ctas / 148.0 * 0.5 : 0.1 + ctas / 148.0 * 0.3);
    t += static_cast<double>(ceil_div(tiles, 148) - 1) * (wide ? 2.9 : 1.6);
    if (c == 1 || t < best) {
      best = t;
      *split = c;
    }
  }
  return best;
}

template <bool P_MN, bool Q_MN, int BN, bool SWAP>
cudaError_t launch_tiles(const Operand& p, const Operand& q, ProductArgs a, cudaStream_t stream) {
  CUtensorMap mp, mq;
  if (!operand_map(&mp, p, a.rows_p, a.depth, a.f16 != 0, kRowsP, &a.folded_p) ||
      !operand_map(&mq, q, a.rows_q, a.depth, a.f16 != 0, TileSmem<Q_MN, BN>::kRowsQ, &a.folded_q))
    return cudaErrorInvalidValue;
  constexpr auto* kernel = product_tile_kernel<P_MN, Q_MN, BN, SWAP>;
  static_assert(sizeof(TileSmem<Q_MN, BN>) + 1024 <= kTileSmem, "a tile's ring fits half an SM");
  const cudaError_t e = allow_smem<kernel>(kTileSmem);
  if (e != cudaSuccess) return e;
  const int64_t tiles_p = ceil_div(a.rows_p, kRowsP), tiles_q = ceil_div(a.rows_q, BN), tiles = tiles_p * tiles_q;
  const int64_t slices = ceil_div(a.depth, kDepth);
  int split = 1;
  tile_cost(tiles, slices, BN, &split);
  a.vec = rows_aligned(a.e) && (SWAP ? a.rows_p : a.rows_q) % 4 == 0 && reinterpret_cast<uintptr_t>(a.e.bias) % 16 == 0;
  a.tiles_p = static_cast<int32_t>(tiles_p);
  return launch_overlapped(kernel, dim3(static_cast<unsigned>(tiles * split)), kProductThreads, kTileSmem, split, stream,
                           mp, mq, a);
}

template <bool P_MN, bool Q_MN>
cudaError_t launch_pairs(const Operand& p, const Operand& q, ProductArgs a, cudaStream_t stream) {
  CUtensorMap mp, mq;
  if (!operand_map(&mp, p, a.rows_p, a.depth, a.f16 != 0, kRowsP, &a.folded_p) ||
      !operand_map(&mq, q, a.rows_q, a.depth, a.f16 != 0, kRowsP, &a.folded_q))
    return cudaErrorInvalidValue;
  constexpr auto* kernel = product_pair_kernel<P_MN, Q_MN>;
  const cudaError_t e = allow_smem<kernel>(kProductSmem);
  if (e != cudaSuccess) return e;
  a.tiles_p = static_cast<int32_t>(ceil_div(a.rows_p, kPairTile));
  a.tiles_q = static_cast<int32_t>(ceil_div(a.rows_q, kPairTile));
  // a row that ends inside 16 bytes would be stored up to their end
  a.vec = rows_aligned(a.e) && a.rows_q % 8 == 0;
  CUtensorMap my = mp, mz = mp;  // not used where the epilogue is entry by entry, or without z
  if (a.vec && (!block_map(&my, a.e.y, a.e.ldy, a.e.y_dtype, a.rows_p, a.rows_q) ||
                (a.e.z != nullptr && !block_map(&mz, a.e.z, a.e.ldz, a.f16 ? OPR_DTYPE_FP16 : OPR_DTYPE_BF16, a.rows_p, a.rows_q))))
    return cudaErrorInvalidValue;
  const int64_t pairs = std::min<int64_t>(static_cast<int64_t>(a.tiles_p) * a.tiles_q, 148 / 2);
  return launch_overlapped(kernel, dim3(static_cast<unsigned>(2 * pairs)), kProductThreads, kProductSmem, 0, stream, mp, mq,
                           my, mz, a);
}

// Which kernel: CTA pairs, 0.36 us a 256 x 256 slice in whole waves of 74 tiles and
// 3 us more than a single tile for their start and end, or tiles.  E.g. (device us)
// 777 x 4096 x 4096: pairs 29, tiles of 128 35, of 64 47; 512 rows: 31, 24, 27; 128
// rows: 30, 16, 15; a weight gradient of 1024 x 1024 over 16384 rows: 88, 38, 48.
template <bool P_MN, bool Q_MN>
cudaError_t launch_product(const Operand& p, const Operand& q, const ProductArgs& a, cudaStream_t stream) {
  const int64_t slices = ceil_div(a.depth, kDepth);
  const double pairs = 0.36 * slices * ceil_div(ceil_div(a.rows_p, kPairTile) * ceil_div(a.rows_q, kPairTile), 148 / 2) + 3.0;
  int split = 1;
  const double wide = tile_cost(ceil_div(a.rows_p, kRowsP) * ceil_div(a.rows_q, 128), slices, 128, &split);
  const double narrow = tile_cost(ceil_div(a.rows_p, kRowsP) * ceil_div(a.rows_q, 64), slices, 64, &split);
  if (pairs <= wide && pairs <= narrow) return launch_pairs<P_MN, Q_MN>(p, q, a, stream);
  if (wide <= narrow) return launch_tiles<P_MN, Q_MN, 128, false>(p, q, a, stream);
  return launch_tiles<P_MN, Q_MN, 64, false>(p, q, a, stream);
}

// Few rows of x: the weight fills the tiles' 128 rows, the rows of x their columns.
template <bool W_MN>
cudaError_t launch_few_rows(const Operand& x, const Operand& w, ProductArgs a, cudaStream_t stream) {
  const int64_t m = a.rows_p;
  a.rows_p = a.rows_q;
  a.rows_q = static_cast<int32_t>(m);
  if (m <= 16) return launch_tiles<W_MN, false, 16, true>(w, x, a, stream);
  return launch_tiles<W_MN, false, 64, true>(w, x, a, stream);
}
constexpr int64_t kFewRows = 64;

}  // namespace

cudaError_t launch_linear(const Operand& a, const Operand& b, int64_t m, int32_t n, int64_t k, int32_t dtype,
                          const LinearEpilogue& e, int32_t* dev_status, cudaStream_t stream) {
  if (m == 0 || n == 0) return cudaSuccess;
  ProductArgs args{};
  args.rows_p = m;
  args.rows_q = n;
  args.depth = k;
  args.f16 = dtype == OPR_DTYPE_FP16;
  args.e = e;
  args.dev_status = dev_status;
  args.wait_ns = wait_limit_ns();
  if (k == 0) {
    no_depth_kernel<<<static_cast<unsigned>(std::min<int64_t>((m * n + 255) / 256, 148 * 16)), 256, 0, stream>>>(args);
    return cudaGetLastError();
  }
  const bool a_mn = a.col != 1, b_mn = b.col != 1;
  if (a_mn) return launch_product<true, true>(a, b, args, stream);
  if (m <= kFewRows) return b_mn ? launch_few_rows<true>(a, b, args, stream) : launch_few_rows<false>(a, b, args, stream);
  return b_mn ? launch_product<false, true>(a, b, args, stream) : launch_product<false, false>(a, b, args, stream);
}

cudaError_t launch_pack(const PackJob (&jobs)[2], cudaStream_t stream) {
  PackArgs a{};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = static_cast<const uint16_t*>(jobs[i].from);
    a.y[i] = static_cast<uint16_t*>(jobs[i].to);
    a.ldx[i] = jobs[i].ld_from;
    a.ldy[i] = jobs[i].ld_to;
    a.rows[i] = jobs[i].from != nullptr ? jobs[i].rows : 0;
    a.cols[i] = jobs[i].cols;
  }
  const int64_t rows = a.rows[0] + a.rows[1];
  if (rows == 0) return cudaSuccess;
  return launch_overlapped(pack_kernel, dim3(static_cast<unsigned>(std::min<int64_t>(ceil_div(rows, 8), 148 * 8))), 256, 0,
                           0, stream, a);
}

namespace {
struct DzPlan {
  bool wide;  // eight columns a thread
  int32_t cols, rows;  // blocks
  int64_t rows_per_block;
};
DzPlan dz_plan(int64_t m, int32_t n, bool wide) {
  DzPlan p{};
  p.wide = wide;
  p.cols = static_cast<int32_t>(ceil_div(n, kDzSpan * (wide ? 8 : 1)));
  // row blocks: four blocks an SM in all, eight rows at least to each
  const int64_t want = std::max<int64_t>({1, std::min<int64_t>({ceil_div(148 * 4, p.cols), ceil_div(m, 8), kDzMaxBlocks}),
                                          ceil_div(m, kDzMaxRun * kDzRows)});
  p.rows_per_block = ceil_div(m, want);
  p.rows = m > 0 ? static_cast<int32_t>(ceil_div(m, p.rows_per_block)) : 0;
  return p;
}
}  // namespace

int32_t linear_dz_blocks(int64_t m, int32_t n) {
  return std::max(dz_plan(m, n, true).rows, dz_plan(m, n, false).rows);
}

cudaError_t launch_linear_dz(const void* dy, int64_t ld_dy, const void* z, int64_t ldz, int32_t dtype, int64_t m,
                             int32_t n, int32_t activation, void* dz, int64_t ld_dz, float* db, float* partial,
                             int32_t* dev_status, cudaStream_t stream) {
  auto fits = [](const void* p, int64_t ld) { return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld % 8 == 0); };
  const bool wide = n % 8 == 0 && fits(dy, ld_dy) && (activation == OPR_ACT_NONE || fits(z, ldz)) && fits(dz, ld_dz);
  const DzPlan plan = dz_plan(m, n, wide);
  if (plan.rows > 0) {
    const int32_t rows_y = std::min(plan.rows, 1 << 15);  // a grid's y has 65535 at most
    const dim3 grid(plan.cols, rows_y, static_cast<unsigned>(ceil_div(plan.rows, rows_y)));
    float* part = db != nullptr ? partial : nullptr;
    auto go = [&](auto type, auto width) {
      using T = decltype(type);
      return launch_overlapped(linear_dz_kernel<T, decltype(width)::value>, grid, kDzThreads, 0, 0, stream,
                               static_cast<const T*>(dy), ld_dy, static_cast<const T*>(z), ldz, m, n, activation,
                               static_cast<T*>(dz), ld_dz, part, plan.rows_per_block, dev_status);
    };
    auto typed = [&](auto width) {
      return dtype == OPR_DTYPE_BF16 ? go(__nv_bfloat16{}, width) : go(__half{}, width);
    };
    const cudaError_t e = wide ? typed(std::integral_constant<int, 8>{}) : typed(std::integral_constant<int, 1>{});
    if (e != cudaSuccess) return e;
  }
  if (db == nullptr) return cudaSuccess;
  return launch_overlapped(column_sum_kernel, dim3(static_cast<unsigned>(ceil_div(n, 32))), 256, 0, 0, stream, partial,
                           plan.rows, n, db);
}

}  // namespace opr
