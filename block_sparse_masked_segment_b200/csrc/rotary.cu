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
// All arithmetic in fp32, each output rounded once.  HBM-bound: every element is
// read and written once.
#include <algorithm>

#include "layer.cuh"

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

// One warp per (token, head), entry by entry: any head_dim, stride and alignment.
template <typename TI, typename TO>
__global__ void __launch_bounds__(32 * kWarps) heads_kernel(const HeadArgs a, int32_t heads_total) {
  const int lane = threadIdx.x & 31;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (item >= a.total * heads_total) return;
  const int64_t tok = item / heads_total;
  int h = static_cast<int>(item % heads_total), si = 0;
  while (h >= a.set[si].heads) h -= a.set[si++].heads;
  const HeadSet& s = a.set[si];
  const int64_t orow = a.row_map != nullptr ? a.row_map[tok] : tok;
  if (orow < 0 || orow >= a.total) {
    if (lane == 0 && a.dev_status != nullptr) atomicOr(a.dev_status, OPR_DEV_BAD_INPUT);
    return;
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
  bool bad = false;
  auto put = [&](int i, float v) {
    bad |= beyond<TO>(v);
    y[i] = from_float<TO>(v);
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
      bad |= beyond<TO>(v);
      dx[i] = from_float<TO>(v);
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
// an entry, added in a fixed order in fp64.
__global__ void __launch_bounds__(1024) head_grad_sum_kernel(const HeadArgs a, int32_t blocks_q, int32_t blocks_k) {
  __shared__ double sums[32][33];
  const HeadSet& s = a.set[blockIdx.y];
  const int32_t blocks = blockIdx.y == 0 ? blocks_q : blocks_k;
  const int col = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int i = static_cast<int>(blockIdx.x) * 32 + col;
  double t = 0.0;
  if (i < a.d)
    for (int b = part; b < blocks; b += 32) t += s.partial[static_cast<int64_t>(b) * a.d + i];
  sums[part][col] = t;
  __syncthreads();
  if (part != 0 || i >= a.d) return;
  for (int p = 1; p < 32; ++p) t += sums[p][col];
  s.w_grad[i] = static_cast<float>(t);
}

// ---------------------------------------------------------------- vector form
// For heads whose rows start on 16-byte boundaries, d a multiple of 16 and the pairs
// a multiple of 8.  A head is d / 16 units of two 8-entry vectors, one unit a lane:
//   half layout, rotated   entries 8c .. 8c+7 and pairs + 8c .. pairs + 8c + 7
//   otherwise              entries 16c .. 16c + 15
// so that a unit holds both entries of its eight pairs (pairs 8c .. 8c + 7) in either
// layout, and a head is a group of kGroup lanes whose sums are a few shuffles.
constexpr int kThreadsVec = 256;

template <typename T>
struct Raw {  // a unit as loaded
  uint4 v[sizeof(T) == 4 ? 4 : 2];
};

template <typename T>
__device__ __forceinline__ Raw<T> load_unit(const T* p, int o1, int o2) {
  Raw<T> r;
  if constexpr (sizeof(T) == 4) {
    r.v[0] = reinterpret_cast<const uint4*>(p + o1)[0];
    r.v[1] = reinterpret_cast<const uint4*>(p + o1)[1];
    r.v[2] = reinterpret_cast<const uint4*>(p + o2)[0];
    r.v[3] = reinterpret_cast<const uint4*>(p + o2)[1];
  } else {
    r.v[0] = *reinterpret_cast<const uint4*>(p + o1);
    r.v[1] = *reinterpret_cast<const uint4*>(p + o2);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void unpack(const Raw<T>& r, float (&f)[16]) {
  const T* e = reinterpret_cast<const T*>(r.v);
#pragma unroll
  for (int k = 0; k < 16; ++k) f[k] = as_float(e[k]);
}

// Stores a unit; true when an fp16 entry is beyond the range.
template <typename T>
__device__ __forceinline__ bool store_unit(T* p, int o1, int o2, const float (&f)[16]) {
  Raw<T> r;
  T* e = reinterpret_cast<T*>(r.v);
  bool bad = false;
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    bad |= beyond<T>(f[k]);
    e[k] = from_float<T>(f[k]);
  }
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<uint4*>(p + o1)[0] = r.v[0];
    reinterpret_cast<uint4*>(p + o1)[1] = r.v[1];
    reinterpret_cast<uint4*>(p + o2)[0] = r.v[2];
    reinterpret_cast<uint4*>(p + o2)[1] = r.v[3];
  } else {
    *reinterpret_cast<uint4*>(p + o1) = r.v[0];
    *reinterpret_cast<uint4*>(p + o2) = r.v[1];
  }
  return bad;
}

// Rotates the unit's pairs by t = (cos, sin) of each, sin with the sign `sign`.
template <bool INTERLEAVED>
__device__ __forceinline__ void rotate_unit(float (&x)[16], const float (&t)[16], float sign) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int ia = INTERLEAVED ? 2 * k : k, ib = INTERLEAVED ? 2 * k + 1 : k + 8;
    const float c = t[2 * k], s = sign * t[2 * k + 1];
    const float va = x[ia], vb = x[ib];
    x[ia] = va * c - vb * s;
    x[ib] = vb * c + va * s;
  }
}

// Tables in shared memory, as float4 [4][units] per token (cos, sin of two pairs) or
// per weight (four entries): neighbouring lanes read neighbouring 16 bytes.
__device__ __forceinline__ void read16(const float4* t, int units, int c, float (&f)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 x = t[q * units + c];
    f[4 * q] = x.x;
    f[4 * q + 1] = x.y;
    f[4 * q + 2] = x.z;
    f[4 * q + 3] = x.w;
  }
}

// cos and sin of `ntok` tokens from tok0 into cs [ntok][4][rot_units].
__device__ __forceinline__ void fill_turns(const HeadArgs& a, int64_t tok0, int ntok, float4* cs) {
  const int units = a.pairs / 8;
  for (int i = threadIdx.x; i < ntok * a.pairs; i += blockDim.x) {
    const int t = i / a.pairs, j = i % a.pairs;
    float c, s;
    turn(a.pos[tok0 + t], a.freq[j], a.scale, c, s);
    const int unit = j / 8, k = j % 8;
    reinterpret_cast<float2*>(cs + (t * 4 + k / 2) * units + unit)[k & 1] = make_float2(c, s);
  }
}

// Weight w [d] into t [4][units]: entries in unit order.
__device__ __forceinline__ void fill_weight(const HeadArgs& a, const void* w, float4* t) {
  const int units = a.d / 16;
  for (int i = threadIdx.x; i < a.d; i += blockDim.x) {
    const int c = i / 16, k = i % 16;
    const bool split = !a.interleaved && c < a.pairs / 8;
    const int e = split ? (k < 8 ? 8 * c + k : a.pairs + 8 * c + k - 8) : 16 * c + k;
    reinterpret_cast<float*>(t + (k / 4) * units + c)[k & 3] = load_typed(w, a.w_dtype, e);
  }
}

template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int m = G / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// A block takes `tokens` tokens, forms their cos and sin once, and its groups of G
// lanes walk the (token, head) items of all sets.
template <typename TI, typename TO, int G>
__global__ void __launch_bounds__(kThreadsVec) heads_vec_kernel(const HeadArgs a, int32_t heads_total, int32_t tokens) {
  extern __shared__ float4 tables[];
  const int units = a.d / 16, rot_units = a.pairs / 8;
  float4* wt = tables;                                 // [2][4][units], with a norm
  const bool norm = a.set[0].mode == kHeadNormRotate;  // of set 0 (and 1)
  float4* cs = tables + (norm ? 8 * units : 0);        // [tokens][4][rot_units]
  const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * tokens;
  const int ntok = static_cast<int>(a.total - tok0 < tokens ? a.total - tok0 : tokens);
  const int c = threadIdx.x % G;
  const int items = ntok * heads_total;
  const bool live = c < units;
  const bool turns = c < rot_units;
  const bool apart = !a.interleaved && turns;
  const int o1 = apart ? 8 * c : 16 * c, o2 = apart ? a.pairs + 8 * c : 16 * c + 8;
  const float sign = a.inverse ? -1.f : 1.f;

  struct Item {
    int t, h, si;
  };
  auto item_of = [&](int i) {
    Item it;
    it.t = i / heads_total;
    it.h = i % heads_total;
    it.si = 0;
    while (it.h >= a.set[it.si].heads) it.h -= a.set[it.si++].heads;
    return it;
  };
  auto fetch = [&](const Item& it) {
    const HeadSet& s = a.set[it.si];
    return load_unit(static_cast<const TI*>(s.x) + (tok0 + it.t) * s.x_stride + static_cast<int64_t>(it.h) * a.d, o1, o2);
  };
  int i = threadIdx.x / G;
  Item it{};
  Raw<TI> raw{};
  if (i < items) {
    it = item_of(i);
    if (live) raw = fetch(it);  // in flight while the tables are made
  }
  fill_turns(a, tok0, ntok, cs);
  if (norm)
    for (int s = 0; s < 2; ++s) fill_weight(a, a.set[s].w, wt + 4 * s * units);
  __syncthreads();
  bool bad = false, lost = false;
  // all lanes of a warp stay in the loop for the shuffles
  for (int first = threadIdx.x / 32 * (32 / G); first < items; first += kThreadsVec / G, i += kThreadsVec / G) {
    const Item now = it;
    float x[16];
    unpack(raw, x);
    const bool valid = i < items && live;
    if (i + kThreadsVec / G < items) {
      it = item_of(i + kThreadsVec / G);
      if (live) raw = fetch(it);
    }
    const HeadSet& s = a.set[now.si];
    if (norm) {
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) sum = fmaf(x[k], x[k], sum);
      sum = group_sum<G>(valid ? sum : 0.f);
      if (valid && s.mode == kHeadNormRotate) {
        const float rs = 1.f / sqrtf(sum / a.d + a.eps);
        float w[16];
        read16(wt + 4 * now.si * units, units, c, w);
#pragma unroll
        for (int k = 0; k < 16; ++k) x[k] *= rs * w[k];
      }
    }
    if (!valid) continue;
    const int64_t tok = tok0 + now.t;
    const int64_t orow = a.row_map != nullptr ? a.row_map[tok] : tok;
    if (orow < 0 || orow >= a.total) {
      lost = true;
      continue;
    }
    if (turns && s.mode != kHeadCopy) {
      float t[16];
      read16(cs + now.t * 4 * rot_units, rot_units, c, t);
      if (a.interleaved)
        rotate_unit<true>(x, t, sign);
      else
        rotate_unit<false>(x, t, sign);
    }
    bad |= store_unit(static_cast<TO*>(s.y) + orow * s.y_stride + static_cast<int64_t>(now.h) * a.d, o1, o2, x);
  }
  if (a.dev_status != nullptr) {
    if (bad) atomicOr(a.dev_status, OPR_DEV_FP16_RANGE);
    if (lost) atomicOr(a.dev_status, OPR_DEV_BAD_INPUT);
  }
}

// Gradient in the vector form.  Blocks are dealt to the sets in proportion to their
// heads; a block walks its set's tiles of `tokens` tokens with its groups, and keeps
// its sums for w in registers, entry by entry of the lanes' units.
struct GradBlocks {
  int32_t first[4];  // blocks of set i: first[i] .. first[i + 1] - 1
};

template <typename TI, typename TG, typename TO, int G>
__global__ void __launch_bounds__(kThreadsVec, 2) head_grads_vec_kernel(const HeadArgs a, const GradBlocks deal,
                                                                        int32_t max_tokens) {
  extern __shared__ float4 tables[];
  constexpr int kGroups = kThreadsVec / G;
  int si = 0;
  while (static_cast<int>(blockIdx.x) >= deal.first[si + 1]) ++si;
  const HeadSet& s = a.set[si];
  const int units = a.d / 16, rot_units = a.pairs / 8;
  float4* wt = tables;                                                  // [4][units]
  float* red = reinterpret_cast<float*>(tables + 4 * units);            // [groups][d]
  float4* cs = tables + 4 * units + kGroups * 4 * units;                // [tokens][4][rot_units]
  const int block = static_cast<int>(blockIdx.x) - deal.first[si], blocks = deal.first[si + 1] - deal.first[si];
  // items a tile: about eight to a group
  const int tokens = min(max_tokens, max(1, 8 * kGroups / s.heads));
  const int64_t tiles = (a.total + tokens - 1) / tokens;
  const int c = threadIdx.x % G;
  const bool live = c < units, turns = c < rot_units && s.mode != kHeadCopy;
  const bool apart = !a.interleaved && c < rot_units;
  const int o1 = apart ? 8 * c : 16 * c, o2 = apart ? a.pairs + 8 * c : 16 * c + 8;
  const float inv_d = 1.f / a.d;
  float acc[16] = {};
  bool bad = false, lost = false;
  if (s.mode != kHeadCopy) fill_weight(a, s.w, wt);

  for (int64_t tile = block; tile < tiles; tile += blocks) {
    const int64_t tok0 = tile * tokens;
    const int ntok = static_cast<int>(a.total - tok0 < tokens ? a.total - tok0 : tokens);
    const int items = ntok * s.heads;
    Raw<TI> rx{};
    Raw<TG> rg{};
    bool known = false;  // of the item held: its gradient row is in range
    auto fetch = [&](int i) {
      const int t = i / s.heads, h = i % s.heads;
      const int64_t tok = tok0 + t;
      const int64_t grow = a.row_map != nullptr ? a.row_map[tok] : tok;
      known = grow >= 0 && grow < a.total;
      if (!known) {
        lost = true;
        return;
      }
      if (!live) return;
      rg = load_unit(static_cast<const TG*>(s.dy) + grow * s.dy_stride + static_cast<int64_t>(h) * a.d, o1, o2);
      if (s.mode != kHeadCopy)
        rx = load_unit(static_cast<const TI*>(s.x) + tok * s.x_stride + static_cast<int64_t>(h) * a.d, o1, o2);
    };
    int i = threadIdx.x / G;
    if (i < items) fetch(i);
    __syncthreads();  // the tile before has been read
    if (s.mode != kHeadCopy) fill_turns(a, tok0, ntok, cs);
    __syncthreads();
    for (int first = threadIdx.x / 32 * (32 / G); first < items; first += kGroups, i += kGroups) {
      float x[16], g[16];
      unpack(rx, x);
      unpack(rg, g);
      const bool valid = i < items && live && known;
      const int t = i / s.heads, h = i % s.heads;
      if (i + kGroups < items) fetch(i + kGroups);
      if (turns && valid) {
        float w[16];
        read16(cs + t * 4 * rot_units, rot_units, c, w);
        if (a.interleaved)
          rotate_unit<true>(g, w, -1.f);
        else
          rotate_unit<false>(g, w, -1.f);
      }
      if (s.mode != kHeadCopy) {
        // sum of x^2 and of u x in one round of shuffles; xh = x rs comes after
        float w[16], sq = 0.f, ux = 0.f;
        read16(wt, units, live ? c : 0, w);
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          sq = fmaf(x[k], x[k], sq);
          w[k] *= g[k];  // u
          ux = fmaf(w[k], x[k], ux);
        }
        sq = group_sum<G>(valid ? sq : 0.f);
        ux = group_sum<G>(valid ? ux : 0.f);
        if (!valid) continue;
        const float rs = 1.f / sqrtf(sq * inv_d + a.eps);
        const float mean = ux * rs * inv_d;  // of u xh
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float xh = x[k] * rs;
          acc[k] = fmaf(g[k], xh, acc[k]);
          g[k] = rs * (w[k] - xh * mean);
        }
      }
      if (!valid) continue;
      bad |= store_unit(static_cast<TO*>(s.y) + (tok0 + t) * s.y_stride + static_cast<int64_t>(h) * a.d, o1, o2, g);
    }
  }
  if (a.dev_status != nullptr) {
    if (bad) atomicOr(a.dev_status, OPR_DEV_FP16_RANGE);
    if (lost) atomicOr(a.dev_status, OPR_DEV_BAD_INPUT);
  }
  if (s.mode == kHeadCopy) return;
  float* mine = red + (threadIdx.x / G) * a.d;
  if (live) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      mine[o1 + k] = acc[k];
      mine[o2 + k] = acc[8 + k];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.d; e += kThreadsVec) {
    float t = 0.f;
    for (int g = 0; g < kGroups; ++g) t += red[g * a.d + e];
    s.partial[static_cast<int64_t>(block) * a.d + e] = t;
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
    if (!fits(s.x, s.x_stride, x_dtype) || !fits(s.dy, s.dy_stride, dy_dtype) || !fits(s.y, s.y_stride, y_dtype))
      return false;
  }
  return true;
}

template <typename F>
cudaError_t with_group(int32_t d, F f) {
  const int units = d / 16;
  if (units <= 4) return f(std::integral_constant<int, 4>{});
  if (units <= 8) return f(std::integral_constant<int, 8>{});
  return f(std::integral_constant<int, 16>{});
}

cudaError_t launch_heads_vec(const HeadArgs& a, int32_t heads, int32_t x_dtype, int32_t y_dtype, cudaStream_t stream) {
  return with_group(a.d, [&](auto g) {
    constexpr int G = decltype(g)::value;
    // four items a group where the batch has them and the tables stay small, one
    // token a block for small batches
    const int64_t want = 4 * (kThreadsVec / G) / heads;
    const int32_t tokens = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>({want, 32, a.total / 148})));
    const bool norm = a.set[0].mode == kHeadNormRotate;
    const size_t smem = sizeof(float4) * (static_cast<size_t>(tokens) * 4 * (a.pairs / 8) + (norm ? 8 * (a.d / 16) : 0));
    const unsigned blocks = static_cast<unsigned>((a.total + tokens - 1) / tokens);
    return with_type(x_dtype, [&](auto ti) {
      return with_type(y_dtype, [&](auto to) {
        heads_vec_kernel<decltype(ti), decltype(to), G><<<blocks, kThreadsVec, smem, stream>>>(a, heads, tokens);
        return cudaGetLastError();
      });
    });
  });
}

}  // namespace

cudaError_t launch_heads(const HeadArgs& a, int32_t x_dtype, int32_t y_dtype, cudaStream_t stream) {
  int32_t heads = 0;
  for (int i = 0; i < a.n_sets; ++i) heads += a.set[i].heads;
  if (a.total == 0 || heads == 0) return cudaSuccess;
  if (vector_ready(a, x_dtype, y_dtype, y_dtype)) return launch_heads_vec(a, heads, x_dtype, y_dtype, stream);
  const int64_t blocks = (a.total * heads + kWarps - 1) / kWarps;
  return with_type(x_dtype, [&](auto ti) {
    return with_type(y_dtype, [&](auto to) {
      heads_kernel<decltype(ti), decltype(to)><<<static_cast<unsigned>(blocks), 32 * kWarps, 0, stream>>>(a, heads);
      return cudaGetLastError();
    });
  });
}

namespace {
constexpr int32_t kGradBlocks = 4 * 148;   // at most, per set
constexpr int32_t kVecGradBlocks = 2 * 148;  // over all sets: what runs at one time

cudaError_t launch_head_grads_vec(const HeadArgs& a, int32_t x_dtype, int32_t dy_dtype, int32_t dx_dtype,
                                  int32_t (&blocks)[3], cudaStream_t stream) {
  // v counted whether it is there or not: the sums for w do not depend on it
  const int32_t heads = a.set[0].heads + 2 * a.set[1].heads;
  GradBlocks deal{};
  const int32_t tokens = static_cast<int32_t>(std::max<int64_t>(1, std::min<int64_t>(32, a.total / 148)));
  for (int i = 0; i < 3; ++i) {
    int64_t n = 0;
    if (i < a.n_sets) {
      n = std::max<int64_t>(1, (static_cast<int64_t>(kVecGradBlocks) * a.set[i].heads + heads / 2) / heads);
      n = std::min<int64_t>(n, a.total);
    }
    blocks[i] = static_cast<int32_t>(n);
    deal.first[i + 1] = deal.first[i] + blocks[i];
  }
  return with_group(a.d, [&](auto g) {
    constexpr int G = decltype(g)::value;
    const int units = a.d / 16;
    const size_t smem = sizeof(float4) * (4 * units + kThreadsVec / G * 4 * units + static_cast<size_t>(tokens) * 4 * (a.pairs / 8));
    return with_type(x_dtype, [&](auto ti) {
      return with_type(dy_dtype, [&](auto tg) {
        return with_type(dx_dtype, [&](auto to) {
          using TI = decltype(ti);
          using TG = decltype(tg);
          using TO = decltype(to);
          auto* kernel = head_grads_vec_kernel<TI, TG, TO, G>;
          if (smem > 48 * 1024) {
            const cudaError_t e =
                cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
            if (e != cudaSuccess) return e;
          }
          kernel<<<deal.first[3], kThreadsVec, smem, stream>>>(a, deal, tokens);
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
          static_cast<int32_t>(std::min<int64_t>(kGradBlocks, (a.total * heads + kWarps - 1) / kWarps));
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
