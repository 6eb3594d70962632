// rotary.cu - rotary positions in their general form, and the norm of each head
// of q and k with the rotation in the same pass, forward and gradient.
//
// A head h of d values, r = 2 * pairs of them rotated.  Pair j is (j, j + r/2) in
// the half layout and (2j, 2j + 1) in the interleaved one; its angle is
// pos * freq[j], formed and reduced in fp64.
//   norm      n = h rs w,  rs = 1 / sqrt(mean(h^2) + eps)
//   rotation  y_a = s (a cos - b sin),  y_b = s (b cos + a sin)
//   gradient  g = R^T dy;  xh = h rs;  dw = sum g xh;  u = g w;
//             dh = rs (u - xh mean(u xh))
// All arithmetic in fp32, each output rounded once.
//
// Every element is read and written once, so HBM bounds them; next to it the issue of
// instructions (16 entries a lane: the packed arithmetic, the tables and the fast
// quotients are there for that).  Measured (device time; a plain copy of as many bytes
// in brackets):
//   16384 tokens x 32 heads of 128, half of each rotated, bf16 to fp16   49 us, 5.5 TB/s
//   32749 tokens x 8 heads of 128, fp32, interleaved                     45 us, 5.9 TB/s
//   16384 tokens, 32q/8kv heads of 128 and v, norm                       80 us, 5.0 TB/s [71 us]
//   65536 tokens, 64q/8kv heads of 128 and v, fp32 gradients            838 us, 6.2 TB/s [824 us]
// Tried and slower: persistent blocks that make the next tile's tables between rounds
// (norm 117 us), rows brought by bulk copies to a ring in shared memory (104 us), more
// blocks an SM with fewer registers (five 92 us, six 110 us).
#include <algorithm>

#include "layer.cuh"
#include "sm100.cuh"

namespace opr {
namespace {

constexpr int kWarps = 8;
constexpr int kMaxHeadDim = 256;

// cos and sin of pos * freq, times s.  The angle is reduced by whole turns in
// fp64 (Cody and Waite, the turn in two parts), and what fp32 drops of the
// remainder is put back to first order.
__device__ __forceinline__ void turn(int32_t pos, double freq, float s, float& c, float& sn) {
  constexpr double kTurnHi = 6.283185307179586, kTurnLo = 2.4492935982947064e-16, kInvTurn = 0.15915494309189535;
  const double angle = static_cast<double>(pos) * freq;
  const double n = rint(angle * kInvTurn);
  const double r = fma(-n, kTurnLo, fma(-n, kTurnHi, angle)) * (2.0 * kInvTurn);  // half turns in [-1, 1]
  const float hi = static_cast<float>(r);
  const float lo = static_cast<float>(r - static_cast<double>(hi)) * 3.14159265f;
  float s0, c0;
  sincospif(hi, &s0, &c0);
  c = s * fmaf(-s0, lo, c0);
  sn = s * fmaf(c0, lo, s0);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Entries of pair j.
__device__ __forceinline__ void pair_of(const HeadArgs& a, int j, int& ia, int& ib) {
  ia = a.interleaved ? 2 * j : j;
  ib = a.interleaved ? 2 * j + 1 : j + a.pairs;
}

// One warp per (token, head), entry by entry: any head_dim, stride and alignment.  What
// the vector form below does not take: widths that are no multiple of 16, rotated pairs
// that are no multiple of 8 (20 or 40 entries of a head of 80, 24 of 96), rows off the
// 16-byte grid.  At a quarter to a fifth of its speed (16384 tokens x 32 heads of 80, 20
// entries rotated: 193 us, with 16 37), each angle formed anew for every head.
template <typename TI, typename TO>
__global__ void __launch_bounds__(32 * kWarps) heads_kernel(const HeadArgs a, int32_t heads_total) {
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const int64_t items = a.total * heads_total;
  bool bad = false;
  // more than one item a warp only where the grid has all the blocks that a grid can have
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5); item < items;
       item += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t tok = item / heads_total;
    int h = static_cast<int>(item % heads_total), si = 0;
    while (h >= a.set[si].heads) h -= a.set[si++].heads;
    const HeadSet& s = a.set[si];
    const int64_t orow = a.row_map != nullptr ? a.row_map[tok] : tok;
    if (orow < 0 || orow >= a.total) {
      if (lane == 0 && a.dev_status != nullptr) atomicOr(a.dev_status, OPR_DEV_BAD_INPUT);
      continue;
    }
    const TI* x = static_cast<const TI*>(s.x) + tok * s.x_stride + static_cast<int64_t>(h) * a.d;
    TO* y = static_cast<TO*>(s.y) + orow * s.y_stride + static_cast<int64_t>(h) * a.d;
    float rs = 1.f;
    if (s.mode == kHeadNormRotate) {
      float sum = 0.f;
      for (int i = lane; i < a.d; i += 32) sum = fmaf(as_float(x[i]), as_float(x[i]), sum);
      rs = 1.f / sqrtf(warp_sum(sum) / a.d + a.eps);
    }
    auto value = [&](int i) {
      const float v = as_float(x[i]);
      return s.mode == kHeadNormRotate ? v * rs * load_typed(s.w, a.w_dtype, i) : v;
    };
    auto put = [&](int i, float v) {
      y[i] = from_float<TO>(v);
      bad |= beyond<TO>(as_float(y[i]));
    };
    const int pairs = s.mode == kHeadCopy ? 0 : a.pairs;
    for (int j = lane; j < pairs; j += 32) {
      float c, sn;
      turn(a.pos[tok], a.freq[j], a.scale, c, sn);
      if (a.inverse) sn = -sn;
      int ia, ib;
      pair_of(a, j, ia, ib);
      const float va = value(ia), vb = value(ib);
      put(ia, va * c - vb * sn);
      put(ib, vb * c + va * sn);
    }
    for (int i = 2 * pairs + lane; i < a.d; i += 32) put(i, value(i));
  }
  if (bad && a.dev_status != nullptr) atomicOr(a.dev_status, OPR_DEV_FP16_RANGE);
}

// Gradient, one warp per (token, head) of the set blockIdx.y; each warp keeps its
// sums for w in its own row of shared memory, entry by entry.
template <typename TI, typename TG, typename TO>
__global__ void __launch_bounds__(32 * kWarps) head_grads_kernel(const HeadArgs a) {
  __shared__ float sums[kWarps][kMaxHeadDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const HeadSet& s = a.set[blockIdx.y];
  for (int i = lane; i < a.d; i += 32) sums[warp][i] = 0.f;
  __syncwarp();  // an entry's sums are not added by the lane that cleared it
  bool bad = false;
  const int64_t items = a.total * s.heads;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + warp; item < items;
       item += static_cast<int64_t>(gridDim.x) * kWarps) {
    const int64_t tok = item / s.heads;
    const int h = static_cast<int>(item % s.heads);
    const int64_t grow = a.row_map != nullptr ? a.row_map[tok] : tok;
    if (grow < 0 || grow >= a.total) {
      if (lane == 0 && a.dev_status != nullptr) atomicOr(a.dev_status, OPR_DEV_BAD_INPUT);
      continue;
    }
    const TG* dy = static_cast<const TG*>(s.dy) + grow * s.dy_stride + static_cast<int64_t>(h) * a.d;
    TO* dx = static_cast<TO*>(s.y) + tok * s.y_stride + static_cast<int64_t>(h) * a.d;
    auto put = [&](int i, float v) {
      dx[i] = from_float<TO>(v);
      bad |= beyond<TO>(as_float(dx[i]));
    };
    if (s.mode == kHeadCopy) {
      for (int i = lane; i < a.d; i += 32) put(i, as_float(dy[i]));
      continue;
    }
    const TI* x = static_cast<const TI*>(s.x) + tok * s.x_stride + static_cast<int64_t>(h) * a.d;
    float sum = 0.f;
    for (int i = lane; i < a.d; i += 32) sum = fmaf(as_float(x[i]), as_float(x[i]), sum);
    const float rs = 1.f / sqrtf(warp_sum(sum) / a.d + a.eps);
    // entries of this lane: its pairs' (a, b), then its entries behind the rotated ones
    float u[2 * kMaxHeadDim / 32], xh[2 * kMaxHeadDim / 32];
    int n = 0;
    float dot = 0.f;
    auto take = [&](int i, float g) {
      xh[n] = as_float(x[i]) * rs;
      sums[warp][i] += g * xh[n];
      u[n] = g * load_typed(s.w, a.w_dtype, i);
      dot = fmaf(u[n], xh[n], dot);
      ++n;
    };
    for (int j = lane; j < a.pairs; j += 32) {
      float c, sn;
      turn(a.pos[tok], a.freq[j], a.scale, c, sn);
      int ia, ib;
      pair_of(a, j, ia, ib);
      const float ga = as_float(dy[ia]), gb = as_float(dy[ib]);
      take(ia, ga * c + gb * sn);
      take(ib, gb * c - ga * sn);
    }
    for (int i = 2 * a.pairs + lane; i < a.d; i += 32) take(i, as_float(dy[i]));
    dot = warp_sum(dot) / a.d;
    n = 0;
    for (int j = lane; j < a.pairs; j += 32) {
      int ia, ib;
      pair_of(a, j, ia, ib);
      put(ia, rs * (u[n] - xh[n] * dot));
      ++n;
      put(ib, rs * (u[n] - xh[n] * dot));
      ++n;
    }
    for (int i = 2 * a.pairs + lane; i < a.d; i += 32, ++n) put(i, rs * (u[n] - xh[n] * dot));
  }
  if (bad && a.dev_status != nullptr) atomicOr(a.dev_status, OPR_DEV_FP16_RANGE);
  if (s.mode == kHeadCopy) return;
  __syncthreads();
  for (int i = threadIdx.x; i < a.d; i += 32 * kWarps) {
    float t = 0.f;
    for (int w = 0; w < kWarps; ++w) t += sums[w][i];
    s.partial[static_cast<int64_t>(blockIdx.x) * a.d + i] = t;
  }
}

// dw of set blockIdx.y, 32 entries a block: the blocks' partial sums, 32 threads to
// an entry, added in a fixed order in fp64.  By itself, caches cold: 6 us
// after a first kernel of 295 blocks (2377 tokens), 13 us after one of 2368 (64K tokens).
__global__ void __launch_bounds__(1024) head_grad_sum_kernel(const HeadArgs a, int32_t blocks_q, int32_t blocks_k) {
  __shared__ double sums[32][33];
  const HeadSet& s = a.set[blockIdx.y];
  const int32_t blocks = blockIdx.y == 0 ? blocks_q : blocks_k;
  const int col = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int i = static_cast<int>(blockIdx.x) * 32 + col;
  double t = 0.0;
  if (i < a.d)
#pragma unroll 10
    for (int b = part; b < blocks; b += 32) t += s.partial[static_cast<int64_t>(b) * a.d + i];
  sums[part][col] = t;
  __syncthreads();
  if (part != 0 || i >= a.d) return;
  for (int p = 1; p < 32; ++p) t += sums[p][col];
  s.w_grad[i] = static_cast<float>(t);
}

// ---------------------------------------------------------------- vector form
// For heads whose rows start on 16-byte boundaries, d a multiple of 16 and the pairs
// a multiple of 8.  A head is d / 16 units of 16 entries, one unit a lane, a head a
// group of G lanes whose sums are a few shuffles.  A unit is 16 / VW vectors of VW
// entries: eight where all types have 16 bits, four where one is fp32, so that
// neighbouring lanes read neighbouring 16 bytes of the widest type (vectors side by
// side in a lane instead, 32 or 64 bytes from lane to lane, took 1.1 to 1.4 times as
// long).  Vector q of lane c lies at VW c + q (rotated entries) / (16 / VW) among the
// rotated entries, alike among those behind: either layout's unit then holds both
// entries of its eight pairs, and in the half layout the first eight entries are the
// pairs' first ones.  Entries 2i, 2i + 1 of a unit are one packed fp32 pair: the
// arithmetic runs two entries an instruction.
constexpr int kThreadsVec = 256;

template <int VW>
struct UnitAt {
  int first, step;  // of the vectors; entry of vector q: first + q * step
  __device__ __forceinline__ UnitAt(const HeadArgs& a, int c) {
    const int rot = 2 * a.pairs, rot_units = a.pairs / 8;
    const bool r = c < rot_units;
    first = r ? VW * c : rot + VW * (c - rot_units);
    step = (r ? rot : a.d - rot) / (16 / VW);
  }
  __device__ __forceinline__ int operator[](int q) const { return first + q * step; }
};

template <typename T>
struct Raw {  // a unit as loaded
  uint32_t w[4 * sizeof(T)];
};

template <int VW, typename T>
__device__ __forceinline__ Raw<T> load_unit(const T* p, const UnitAt<VW>& at) {
  constexpr int kWords = VW * sizeof(T) / 4;  // of a vector: 2 or 4
  Raw<T> r;
#pragma unroll
  for (int q = 0; q < 16 / VW; ++q) {
    if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p + at[q]);
      r.w[2 * q] = v.x;
      r.w[2 * q + 1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = reinterpret_cast<const uint4*>(p + at[q])[i];
        r.w[kWords * q + 4 * i] = v.x;
        r.w[kWords * q + 4 * i + 1] = v.y;
        r.w[kWords * q + 4 * i + 2] = v.z;
        r.w[kWords * q + 4 * i + 3] = v.w;
      }
    }
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack(const Raw<T>& r, uint64_t (&f)[8]) {
  const auto& w = r.w;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (std::is_same_v<T, float>) {
      f[i] = f2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      f[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    } else {
      const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[i] = f2(v.x, v.y);
    }
  }
}

// Stores a unit.  For fp16, `top` follows the largest size written (NaN stays).
template <int VW, typename T>
__device__ __forceinline__ void store_unit(T* p, const UnitAt<VW>& at, const uint64_t (&f)[8], __half2& top) {
  constexpr int kWords = VW * sizeof(T) / 4;
  Raw<T> r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float lo, hi;
    f2_split(f[i], lo, hi);
    if constexpr (std::is_same_v<T, float>) {
      r.w[2 * i] = __float_as_uint(lo);
      r.w[2 * i + 1] = __float_as_uint(hi);
    } else if constexpr (std::is_same_v<T, __nv_bfloat16>) {
      r.w[i] = pack_bf16x2(lo, hi);
    } else {
      r.w[i] = pack_f16x2(lo, hi);
      top = __hmax2_nan(top, __habs2(*reinterpret_cast<const __half2*>(&r.w[i])));
    }
  }
#pragma unroll
  for (int q = 0; q < 16 / VW; ++q) {
    if constexpr (kWords == 2)
      *reinterpret_cast<uint2*>(p + at[q]) = make_uint2(r.w[2 * q], r.w[2 * q + 1]);
    else
      *reinterpret_cast<uint4*>(p + at[q]) = make_uint4(r.w[4 * q], r.w[4 * q + 1], r.w[4 * q + 2], r.w[4 * q + 3]);
  }
}
__device__ __forceinline__ bool overflowed(__half2 top) {
  const float2 t = __half22float2(top);
  return beyond_f16(t.x) || beyond_f16(t.y);
}

// Rotates the unit's pairs.  t: for pairs 2i, 2i + 1, t[2i] = (cos, cos), t[2i + 1] = (sin, sin).
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate_unit(uint64_t (&x)[8], const uint64_t (&t)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint64_t c = t[2 * i], s = t[2 * i + 1];
    float s0, s1;
    f2_split(s, s0, s1);
    if constexpr (INTERLEAVED) {
      float c0, c1, a0, b0, a1, b1;
      f2_split(c, c0, c1);
      f2_split(x[2 * i], a0, b0);
      f2_split(x[2 * i + 1], a1, b1);
      x[2 * i] = ffma2(x[2 * i], f2(c0, c0), fmul2(f2(b0, a0), f2(-s0, s0)));
      x[2 * i + 1] = ffma2(x[2 * i + 1], f2(c1, c1), fmul2(f2(b1, a1), f2(-s1, s1)));
    } else {
      const uint64_t a = x[i], b = x[4 + i];
      x[i] = ffma2(a, c, fmul2(b, f2(-s0, -s1)));
      x[4 + i] = ffma2(b, c, fmul2(a, s));
    }
  }
}

// A unit's 16 words of a table float4 [4][units]: neighbouring lanes read
// neighbouring 16 bytes.
__device__ __forceinline__ void read16(const float4* t, int units, int c, uint64_t (&f)[8]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(t + q * units + c);
    f[2 * q] = x.x;
    f[2 * q + 1] = x.y;
  }
}

// i / by through a product: exact while i * by < 2^32; magic 0 where the host cannot
// promise that (or by is 1): the plain quotient.
struct Quotient {
  uint32_t by, magic;
};
__device__ __forceinline__ int quotient(int i, const Quotient& q) {
  return q.magic != 0 ? static_cast<int>(__umulhi(static_cast<uint32_t>(i), q.magic)) : i / static_cast<int>(q.by);
}
// cos and sin of `ntok` tokens from tok0 into cs [ntok][4][pairs / 8], in the order
// of rotate_unit; the transpose's have the sine negated.  `by_pairs`: quotient by pairs.
template <int VW>
__device__ __forceinline__ void fill_turns(const HeadArgs& a, const Quotient& by_pairs, int64_t tok0, int ntok,
                                           bool transpose, float4* cs) {
  const int units = a.pairs / 8;
  const int per = a.interleaved ? VW / 2 : VW;  // pairs that a vector (of the first halves) begins
  const int span = units * per;                 // pairs that one vector of each lane begins: all, 1/2 or 1/4
  for (int i = threadIdx.x; i < ntok * a.pairs; i += kThreadsVec) {
    const int t = quotient(i, by_pairs), j = i - t * a.pairs;
    float c, s;
    turn(a.pos[tok0 + t], a.freq[j], a.scale, c, s);
    const int seg = (j >= span) + (j >= 2 * span) + (j >= 3 * span), k = j - seg * span;
    const int shift = per == 8 ? 3 : per == 4 ? 2 : 1;
    const int unit = k >> shift, slot = seg * per + (k & (per - 1));
    float* to = reinterpret_cast<float*>(cs + (t * 4 + slot / 2) * units + unit) + (slot & 1);
    to[0] = c;
    to[2] = transpose ? -s : s;
  }
}

// The unit's entries of a weight (16-byte aligned).
template <int VW>
__device__ __forceinline__ void load_weight(const HeadArgs& a, const void* w, const UnitAt<VW>& at, uint64_t (&f)[8]) {
  if (a.w_dtype == OPR_DTYPE_BF16)
    unpack(load_unit(static_cast<const __nv_bfloat16*>(w), at), f);
  else if (a.w_dtype == OPR_DTYPE_FP16)
    unpack(load_unit(static_cast<const __half*>(w), at), f);
  else
    unpack(load_unit(static_cast<const float*>(w), at), f);
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = G / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

__device__ __forceinline__ float sum2(uint64_t v) {
  float lo, hi;
  f2_split(v, lo, hi);
  return lo + hi;
}

struct Quotients {
  Quotient set[3];  // by the set's heads
  Quotient pairs;
};

// A block takes `tokens` tokens, forms their cos and sin once, and its groups of G
// lanes walk each set's (token, head) items in rounds, the next round's loads in
// flight.
// NORM: the sets of opr_qk_norm_rope; else the one set of opr_rotary.  At four blocks an SM
// the forms with the norm keep 52 to 70 bytes a thread outside the registers, with fp32
// inputs 262 to 278; they run at the same share of a plain copy's rate either way (16384
// tokens, 32q/8kv and v: bf16 to fp16 76 us, a copy of as many bytes 63; fp32 to fp32 138
// and 123).
template <typename TI, typename TO, int VW, int G, bool NORM>
__global__ void __launch_bounds__(kThreadsVec, 4) heads_vec_kernel(const HeadArgs a, const Quotients quot, int32_t tokens) {
  constexpr int kGroups = kThreadsVec / G;
  extern __shared__ float4 tables[];
  const int units = a.d / 16, rot_units = a.pairs / 8;
  float4* cs = tables;                                                           // [tokens][4][rot_units]
  int32_t* orow = reinterpret_cast<int32_t*>(tables + tokens * 4 * rot_units);  // [tokens], -1: not written
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * tokens;
  const int ntok = static_cast<int>(a.total - tok0 < tokens ? a.total - tok0 : tokens);
  const int c = threadIdx.x % G, group = threadIdx.x / G;
  const bool live = c < units, turns = c < rot_units;
  const UnitAt<VW> at(a, live ? c : 0);
  const float inv_d = 1.f / a.d;

  int si = 0, base = 0;  // the round's set (0 without NORM) and its first item, uniform in the block
  Raw<TI> raw{};
  int t = 0, h = 0;
  bool valid = false;
  auto fetch = [&]() {
    const HeadSet& s = a.set[NORM ? si : 0];
    const int i = base + group;
    t = quotient(i, quot.set[NORM ? si : 0]);
    h = i - t * s.heads;
    valid = live && t < ntok;
    if (valid)
      raw = load_unit(static_cast<const TI*>(s.x) + (tok0 + t) * s.x_stride + static_cast<int64_t>(h) * a.d, at);
  };
  wait_for_previous();
  fetch();  // in flight while the tables are made
  fill_turns<VW>(a, quot.pairs, tok0, ntok, a.inverse != 0, cs);
  bool lost = false;
  for (int i = threadIdx.x; i < ntok; i += kThreadsVec) {
    const int64_t r = a.row_map != nullptr ? a.row_map[tok0 + i] : tok0 + i;
    const bool in = r >= 0 && r < a.total;
    lost |= !in;
    orow[i] = in ? static_cast<int32_t>(r) : -1;
  }
  __syncthreads();
  __half2 top = __float2half2_rn(0.f);
  uint64_t w[8];
  if (NORM) load_weight(a, a.set[0].w, at, w);
  while (true) {
    const HeadSet& s = a.set[NORM ? si : 0];
    uint64_t x[8];
    unpack(raw, x);
    const int now_t = t, now_h = h, now_si = si;
    const bool now_valid = valid;
    base += kGroups;
    if (base >= ntok * s.heads) {
      base = 0;
      ++si;
    }
    const bool more = si < (NORM ? a.n_sets : 1);
    if (more) fetch();
    if (NORM && s.mode == kHeadNormRotate) {
      uint64_t sq = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = ffma2(x[i], x[i], sq);
      const float rs = rsqrtf(fmaf(group_sum<G>(now_valid ? sum2(sq) : 0.f), inv_d, a.eps));
      const uint64_t rs2 = f2(rs, rs);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = fmul2(fmul2(x[i], rs2), w[i]);
    }
    const int to = now_valid ? orow[now_t] : -1;
    if (to >= 0) {
      if (turns && (!NORM || s.mode != kHeadCopy)) {
        uint64_t cw[8];
        read16(cs + now_t * 4 * rot_units, rot_units, c, cw);
        if (a.interleaved)
          rotate_unit<true>(x, cw);
        else
          rotate_unit<false>(x, cw);
      }
      store_unit(static_cast<TO*>(s.y) + to * s.y_stride + static_cast<int64_t>(now_h) * a.d, at, x, top);
    }
    if (!more) break;
    if (NORM && si != now_si && a.set[si].mode == kHeadNormRotate) load_weight(a, a.set[si].w, at, w);
  }
  if (a.dev_status != nullptr) {
    if (overflowed(top)) atomicOr(a.dev_status, OPR_DEV_FP16_RANGE);
    if (lost) atomicOr(a.dev_status, OPR_DEV_BAD_INPUT);
  }
}

// Gradient in the vector form.  Blocks are dealt to the sets in proportion to their
// heads; a block walks its set's tiles of `tokens` tokens with its groups, and keeps
// its sums for w in registers, entry by entry of the lanes' units.
struct GradBlocks {
  int32_t first[4];   // blocks of set i: first[i] .. first[i + 1] - 1
  int32_t tokens[3];  // of a tile of set i
  int32_t cs_bytes;   // of the largest tile's table
};

template <typename TI, typename TG, typename TO, int VW, int G>
__global__ void __launch_bounds__(kThreadsVec, 2) head_grads_vec_kernel(const HeadArgs a, const GradBlocks deal,
                                                                        const Quotients quot) {
  extern __shared__ float4 tables[];
  constexpr int kGroups = kThreadsVec / G;
  int si = 0;
  while (static_cast<int>(blockIdx.x) >= deal.first[si + 1]) ++si;
  const HeadSet& s = a.set[si];
  const bool copy = s.mode == kHeadCopy;
  const int units = a.d / 16, rot_units = a.pairs / 8;
  float4* cs = tables;                                                                             // [tokens][4][rot_units]
  float* red = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(tables) + deal.cs_bytes);  // [groups][d]
  const int block = static_cast<int>(blockIdx.x) - deal.first[si], blocks = deal.first[si + 1] - deal.first[si];
  const int tokens = deal.tokens[si];
  const int64_t tiles = (a.total + tokens - 1) / tokens;
  const int c = threadIdx.x % G, group = threadIdx.x / G;
  const bool live = c < units, turns = c < rot_units && !copy;
  const UnitAt<VW> at(a, live ? c : 0);
  const float inv_d = 1.f / a.d;
  uint64_t acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0;
  // the weight, for the lanes to read back by unit: next to the sums there are no registers
  // left for it
  float4* wt = reinterpret_cast<float4*>(red + kGroups * a.d);  // [4][units]
  if (!copy && threadIdx.x < G && live) {
    uint64_t w[8];
    load_weight(a, s.w, at, w);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      ulonglong2 pair;
      pair.x = w[2 * q];
      pair.y = w[2 * q + 1];
      *reinterpret_cast<ulonglong2*>(wt + q * units + c) = pair;
    }
  }
  __half2 top = __float2half2_rn(0.f);
  bool lost = false;

  for (int64_t tile = block; tile < tiles; tile += blocks) {
    const int64_t tok0 = tile * tokens;
    const int ntok = static_cast<int>(a.total - tok0 < tokens ? a.total - tok0 : tokens);
    const int items = ntok * s.heads;
    Raw<TI> rx{};
    Raw<TG> rg{};
    int t = 0, h = 0;
    bool valid = false;
    auto fetch = [&](int i) {
      t = quotient(i, quot.set[si]);
      h = i - t * s.heads;
      valid = live && t < ntok;
      if (!valid) return;
      const int64_t tok = tok0 + t;
      int64_t grow = tok;
      if (a.row_map != nullptr) {
        grow = a.row_map[tok];
        valid = grow >= 0 && grow < a.total;
        lost |= !valid;
        if (!valid) return;
      }
      rg = load_unit(static_cast<const TG*>(s.dy) + grow * s.dy_stride + static_cast<int64_t>(h) * a.d, at);
      if (!copy)
        rx = load_unit(static_cast<const TI*>(s.x) + tok * s.x_stride + static_cast<int64_t>(h) * a.d, at);
    };
    fetch(group);
    if (!copy) {
      __syncthreads();  // the tile before has been read
      fill_turns<VW>(a, quot.pairs, tok0, ntok, true, cs);
      __syncthreads();
    }
    for (int base = 0; base < items; base += kGroups) {
      uint64_t x[8], g[8];
      unpack(rx, x);
      unpack(rg, g);
      const bool now_valid = valid;
      const int now_t = t, now_h = h;
      if (base + kGroups < items) fetch(base + kGroups + group);
      if (turns && now_valid) {
        uint64_t cw[8];
        read16(cs + now_t * 4 * rot_units, rot_units, c, cw);
        if (a.interleaved)
          rotate_unit<true>(g, cw);
        else
          rotate_unit<false>(g, cw);
      }
      if (!copy) {
        // sums of x^2 and of u x in one round of shuffles (u = g w); xh = x rs after it
        uint64_t w[8], u[8], sq = 0, ux = 0;
        read16(wt, units, live ? c : 0, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[i] = fmul2(g[i], w[i]);
          sq = ffma2(x[i], x[i], sq);
          ux = ffma2(u[i], x[i], ux);
        }
        const float rs = rsqrtf(fmaf(group_sum<G>(now_valid ? sum2(sq) : 0.f), inv_d, a.eps));
        const float mean = group_sum<G>(now_valid ? sum2(ux) : 0.f) * rs * inv_d;  // of u xh
        if (now_valid) {
          const uint64_t rs2 = f2(rs, rs), nm2 = f2(-mean, -mean);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint64_t xh = fmul2(x[i], rs2);
            acc[i] = ffma2(g[i], xh, acc[i]);
            g[i] = fmul2(rs2, ffma2(xh, nm2, u[i]));
          }
        }
      }
      if (now_valid)
        store_unit(static_cast<TO*>(s.y) + (tok0 + now_t) * s.y_stride + static_cast<int64_t>(now_h) * a.d, at, g, top);
    }
  }
  if (a.dev_status != nullptr) {
    if (overflowed(top)) atomicOr(a.dev_status, OPR_DEV_FP16_RANGE);
    if (lost) atomicOr(a.dev_status, OPR_DEV_BAD_INPUT);
  }
  if (copy) return;
  float* mine = red + group * a.d;
  if (live) {
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint64_t*>(mine + at[2 * i / VW] + 2 * i % VW) = acc[i];
  }
  __syncthreads();
  // four threads to an entry, a quarter of the groups each
  for (int e = threadIdx.x / 4; e < a.d; e += kThreadsVec / 4) {
    float t = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups / 4; ++g) t += red[(threadIdx.x % 4 * (kGroups / 4) + g) * a.d + e];
    t += __shfl_xor_sync(0xffffffffu, t, 1);
    t += __shfl_xor_sync(0xffffffffu, t, 2);
    if (threadIdx.x % 4 == 0) s.partial[static_cast<int64_t>(block) * a.d + e] = t;
  }
}

template <typename F>
cudaError_t with_type(int32_t dtype, F f) {
  if (dtype == OPR_DTYPE_BF16) return f(__nv_bfloat16{});
  if (dtype == OPR_DTYPE_FP16) return f(__half{});
  return f(float{});
}

// Do all rows of heads allow the vector form?
bool vector_ready(const HeadArgs& a, int32_t x_dtype, int32_t dy_dtype, int32_t y_dtype) {
  if (a.d % 16 != 0 || a.pairs % 8 != 0) return false;
  auto fits = [](const void* p, int64_t stride, int32_t dtype) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * dtype_bytes(dtype) % 16 == 0);
  };
  for (int i = 0; i < a.n_sets; ++i) {
    const HeadSet& s = a.set[i];
    if (!fits(s.x, s.x_stride, x_dtype) || !fits(s.dy, s.dy_stride, dy_dtype) || !fits(s.y, s.y_stride, y_dtype) ||
        !fits(s.w, 0, a.w_dtype))
      return false;
  }
  return true;
}

// Entries of a unit's vectors: 16 bytes of the widest type.
template <typename... T>
constexpr int vector_width = (std::is_same_v<T, float> || ...) ? 4 : 8;

template <typename F>
cudaError_t with_group(int32_t d, F f) {
  const int units = d / 16;
  if (units <= 4) return f(std::integral_constant<int, 4>{});
  if (units <= 8) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

// Quotient for numbers below `most`.
Quotient quotient_by(int32_t by, int64_t most) {
  Quotient q{static_cast<uint32_t>(by), 0};
  if (by > 1 && most * by < (int64_t{1} << 32)) q.magic = static_cast<uint32_t>(((uint64_t{1} << 32) + q.by - 1) / q.by);
  return q;
}

// Those of tiles of tokens[i] tokens of set i; items of the last round may reach past
// the tile by a round of groups.
Quotients quotients(const HeadArgs& a, const int32_t (&tokens)[3]) {
  Quotients q{};
  int32_t most = 0;
  for (int i = 0; i < a.n_sets; ++i) {
    q.set[i] = quotient_by(a.set[i].heads, static_cast<int64_t>(tokens[i]) * a.set[i].heads + 2 * kThreadsVec);
    most = std::max(most, tokens[i]);
  }
  q.pairs = quotient_by(a.pairs, static_cast<int64_t>(most) * a.pairs + kThreadsVec);
  return q;
}

cudaError_t launch_heads_vec(const HeadArgs& a, int32_t x_dtype, int32_t y_dtype, cudaStream_t stream) {
  return with_group(a.d, [&](auto g) {
    constexpr int G = decltype(g)::value;
    int32_t fewest = a.set[0].heads, heads = 0;
    for (int i = 0; i < a.n_sets; ++i) {
      fewest = std::min(fewest, a.set[i].heads);
      heads += a.set[i].heads;
    }
    // full rounds for the smallest set and at least kRounds of them in all, where the
    // batch has the tokens; small batches spread over the SMs instead
    constexpr int kGroups = kThreadsVec / G, kRounds = 4;
    const int64_t want = std::max<int64_t>((kGroups + fewest - 1) / fewest, (kRounds * kGroups + heads - 1) / heads);
    const int32_t tokens =
        static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>({want, 32, a.total / (2 * 148)})));
    const size_t smem = sizeof(float4) * tokens * 4 * (a.pairs / 8) + sizeof(int32_t) * tokens;
    const unsigned blocks = static_cast<unsigned>((a.total + tokens - 1) / tokens);
    const int32_t each[3] = {tokens, tokens, tokens};
    const Quotients q = quotients(a, each);
    return with_type(x_dtype, [&](auto ti) {
      return with_type(y_dtype, [&](auto to) {
        using TI = decltype(ti);
        using TO = decltype(to);
        constexpr int VW = vector_width<TI, TO>;
        if (a.set[0].mode == kHeadNormRotate)
          return launch_overlapped(heads_vec_kernel<TI, TO, VW, G, true>, dim3(blocks), kThreadsVec, smem, 0, stream, a, q,
                                   tokens);
        return launch_overlapped(heads_vec_kernel<TI, TO, VW, G, false>, dim3(blocks), kThreadsVec, smem, 0, stream, a, q,
                                 tokens);
      });
    });
  });
}

}  // namespace

cudaError_t launch_heads(const HeadArgs& a, int32_t x_dtype, int32_t y_dtype, cudaStream_t stream) {
  int32_t heads = 0;
  for (int i = 0; i < a.n_sets; ++i) heads += a.set[i].heads;
  if (a.total == 0 || heads == 0) return cudaSuccess;
  if (vector_ready(a, x_dtype, y_dtype, y_dtype)) return launch_heads_vec(a, x_dtype, y_dtype, stream);
  const int64_t blocks = std::min<int64_t>((a.total * heads + kWarps - 1) / kWarps, 0x7FFFFFFF);  // of a grid at most
  return with_type(x_dtype, [&](auto ti) {
    return with_type(y_dtype, [&](auto to) {
      return launch_overlapped(heads_kernel<decltype(ti), decltype(to)>, dim3(static_cast<unsigned>(blocks)), 32 * kWarps, 0,
                               0, stream, a, heads);
    });
  });
}

namespace {
constexpr int32_t kGradBlocks = 16 * 148;  // at most

cudaError_t launch_head_grads_vec(const HeadArgs& a, int32_t x_dtype, int32_t dy_dtype, int32_t dx_dtype,
                                  int32_t (&blocks)[3], cudaStream_t stream) {
  // v counted whether it is there or not: the sums for w do not depend on it
  const int32_t heads = a.set[0].heads + 2 * a.set[1].heads;
  GradBlocks deal{};
  // Blocks over all sets: about 40 rounds of items to each, from the two to an SM that
  // run at one time up to eight times as many, which even the sets' speeds out (64K
  // tokens of 64q/8kv heads of 128: 1050 us with 296, 885 with 592, 842 with 2368;
  // 2377 tokens of 8q/2kv heads of 64: 13 with 296, 44 with 2368).
  const int64_t rounds = a.total * heads * (a.d / 16) / kThreadsVec;
  const int64_t total_blocks = std::max<int64_t>(2 * 148, std::min<int64_t>(kGradBlocks, rounds / 40));
  for (int i = 0; i < 3; ++i) {
    int64_t n = 0;
    if (i < a.n_sets) {
      n = std::max<int64_t>(1, (total_blocks * a.set[i].heads + heads / 2) / heads);
      n = std::min<int64_t>(n, a.total);
    }
    blocks[i] = static_cast<int32_t>(n);
    deal.first[i + 1] = deal.first[i] + blocks[i];
  }
  return with_group(a.d, [&](auto g) {
    constexpr int G = decltype(g)::value;
    int32_t most = 1;
    for (int i = 0; i < a.n_sets; ++i) {
      // about eight rounds a tile, at least a tile a block
      const int64_t want = (8 * (kThreadsVec / G) + a.set[i].heads - 1) / a.set[i].heads;
      deal.tokens[i] = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>({want, 32, a.total / blocks[i]})));
      most = std::max(most, deal.tokens[i]);
    }
    deal.cs_bytes = static_cast<int32_t>(sizeof(float4)) * most * 4 * (a.pairs / 8);
    const Quotients q = quotients(a, deal.tokens);
    const size_t smem = deal.cs_bytes + sizeof(float) * (kThreadsVec / G + 1) * a.d;
    return with_type(x_dtype, [&](auto ti) {
      return with_type(dy_dtype, [&](auto tg) {
        return with_type(dx_dtype, [&](auto to) {
          using TI = decltype(ti);
          using TG = decltype(tg);
          using TO = decltype(to);
          auto* kernel = head_grads_vec_kernel<TI, TG, TO, vector_width<TI, TG, TO>, G>;
          if (smem > 48 * 1024) {
            const cudaError_t e =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
            if (e != cudaSuccess) return e;
          }
          // not overlapped with its neighbours: 64K tokens took 837 us so, 850 otherwise
          kernel<<<deal.first[3], kThreadsVec, smem, stream>>>(a, deal, q);
          return cudaGetLastError();
        });
      });
    });
  });
}
}  // namespace

int32_t head_grad_blocks(int64_t total, int32_t heads) {
  return static_cast<int32_t>(std::min<int64_t>(std::max<int64_t>(total, (total * heads + kWarps - 1) / kWarps), kGradBlocks));
}

cudaError_t launch_head_grads(const HeadArgs& a, int32_t x_dtype, int32_t dy_dtype, int32_t dx_dtype,
                              cudaStream_t stream) {
  int32_t blocks[3] = {0, 0, 0};
  if (a.total > 0) {
    cudaError_t e;
    if (vector_ready(a, x_dtype, dy_dtype, dx_dtype)) {
      e = launch_head_grads_vec(a, x_dtype, dy_dtype, dx_dtype, blocks, stream);
    } else {
      int32_t heads = 0;
      for (int i = 0; i < a.n_sets; ++i) heads = std::max(heads, a.set[i].heads);
      blocks[0] = blocks[1] =
          static_cast<int32_t>(std::min<int64_t>(4 * 148, (a.total * heads + kWarps - 1) / kWarps));
      e = with_type(x_dtype, [&](auto ti) {
        return with_type(dy_dtype, [&](auto tg) {
          return with_type(dx_dtype, [&](auto to) {
            head_grads_kernel<decltype(ti), decltype(tg), decltype(to)>
                <<<dim3(blocks[0], a.n_sets), 32 * kWarps, 0, stream>>>(a);
            return cudaGetLastError();
          });
        });
      });
    }
    if (e != cudaSuccess) return e;
  }
  head_grad_sum_kernel<<<dim3((a.d + 31) / 32, 2), 1024, 0, stream>>>(a, blocks[0], blocks[1]);
  return cudaGetLastError();
}

}  // namespace opr
