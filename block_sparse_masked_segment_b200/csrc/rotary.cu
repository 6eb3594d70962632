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

// dw of set blockIdx.y: the blocks' partial sums, added in block order.
__global__ void __launch_bounds__(256) head_grad_sum_kernel(const HeadArgs a, int32_t blocks) {
  const HeadSet& s = a.set[blockIdx.y];
  if (s.mode == kHeadCopy) return;
  for (int i = threadIdx.x; i < a.d; i += blockDim.x) {
    double t = 0.0;
    for (int b = 0; b < blocks; ++b) t += s.partial[static_cast<int64_t>(b) * a.d + i];
    s.w_grad[i] = static_cast<float>(t);
  }
}

template <typename F>
cudaError_t with_type(int32_t dtype, F f) {
  if (dtype == OPR_DTYPE_BF16) return f(__nv_bfloat16{});
  if (dtype == OPR_DTYPE_FP16) return f(__half{});
  return f(float{});
}

}  // namespace

cudaError_t launch_heads(const HeadArgs& a, int32_t x_dtype, int32_t y_dtype, cudaStream_t stream) {
  int32_t heads = 0;
  for (int i = 0; i < a.n_sets; ++i) heads += a.set[i].heads;
  if (a.total == 0 || heads == 0) return cudaSuccess;
  const int64_t blocks = (a.total * heads + kWarps - 1) / kWarps;
  return with_type(x_dtype, [&](auto ti) {
    return with_type(y_dtype, [&](auto to) {
      heads_kernel<decltype(ti), decltype(to)><<<static_cast<unsigned>(blocks), 32 * kWarps, 0, stream>>>(a, heads);
      return cudaGetLastError();
    });
  });
}

int32_t head_grad_blocks(int64_t total, int32_t heads) {
  return static_cast<int32_t>(std::min<int64_t>((total * heads + kWarps - 1) / kWarps, 4 * 148));
}

cudaError_t launch_head_grads(const HeadArgs& a, int32_t x_dtype, int32_t dy_dtype, int32_t dx_dtype,
                              cudaStream_t stream) {
  int32_t heads = 0;
  for (int i = 0; i < a.n_sets; ++i) heads = std::max(heads, a.set[i].heads);
  const int32_t blocks = head_grad_blocks(a.total, heads);
  if (blocks > 0) {
    const cudaError_t e = with_type(x_dtype, [&](auto ti) {
      return with_type(dy_dtype, [&](auto tg) {
        return with_type(dx_dtype, [&](auto to) {
          head_grads_kernel<decltype(ti), decltype(tg), decltype(to)>
              <<<dim3(blocks, a.n_sets), 32 * kWarps, 0, stream>>>(a);
          return cudaGetLastError();
        });
      });
    });
    if (e != cudaSuccess) return e;
  }
  head_grad_sum_kernel<<<dim3(1, a.n_sets), 256, 0, stream>>>(a, blocks);
  return cudaGetLastError();
}

}  // namespace opr
