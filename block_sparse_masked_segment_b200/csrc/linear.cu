// linear.cu - matrix product with bias, activation and residual in its epilogue,
// and its gradients.
//   z = x w^T + bias;  y = act(z) + residual
//   dz = dy act'(z);  db = sum over rows of dz;  dx = dz w;  dw = dz^T x
// 16-bit operands, fp32 sums, each output rounded once.
#include <algorithm>

#include "layer.cuh"

namespace opr {
namespace {

__device__ __forceinline__ float sigmoid(float x) { return 1.f / (1.f + expf(-x)); }

// gelu with tanh: z/2 (1 + tanh u) = z sigmoid(2u), u = sqrt(2/pi) (z + 0.044715 z^3)
constexpr float kGeluC = 0.79788456080286536f, kGeluA = 0.044715f, kSqrtHalf = 0.70710678118654752f,
                kInvSqrt2Pi = 0.39894228040143268f;

__device__ __forceinline__ float activate(float z, int32_t act) {
  if (act == OPR_ACT_SILU) return z * sigmoid(z);
  if (act == OPR_ACT_GELU) return 0.5f * z * (1.f + erff(z * kSqrtHalf));
  if (act == OPR_ACT_GELU_TANH) return z * sigmoid(2.f * kGeluC * (z + kGeluA * z * z * z));
  return z;
}

__device__ __forceinline__ float activate_slope(float z, int32_t act) {
  if (act == OPR_ACT_SILU) {
    const float s = sigmoid(z);
    return s * (1.f + z * (1.f - s));
  }
  if (act == OPR_ACT_GELU) return 0.5f * (1.f + erff(z * kSqrtHalf)) + z * kInvSqrt2Pi * expf(-0.5f * z * z);
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
    return !(fabsf(v) <= 65504.f);
  } else {
    static_cast<float*>(p)[i] = v;
  }
  return false;
}

constexpr int kEdge = 64, kDepth = 16;

// One 64 x 64 tile per block of 256 threads, 4 x 4 outputs a thread, fp32 sums.
template <typename T>
__global__ void __launch_bounds__(256) linear_kernel(const Operand a, const Operand b, int64_t m, int32_t n, int64_t k,
                                                     int32_t dtype, const LinearEpilogue e, int32_t* dev_status) {
  __shared__ float as[kDepth][kEdge + 1], bs[kDepth][kEdge + 1];
  const int64_t i0 = static_cast<int64_t>(blockIdx.x) * kEdge;
  const int64_t j0 = static_cast<int64_t>(blockIdx.y) * kEdge;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const T *pa = static_cast<const T*>(a.p), *pb = static_cast<const T*>(b.p);
  float acc[4][4] = {};
  for (int64_t k0 = 0; k0 < k; k0 += kDepth) {
    for (int t = threadIdx.x; t < kEdge * kDepth; t += 256) {
      // neighbouring threads along the operand's contiguous direction
      const int ra = a.col == 1 ? t / kDepth : t % kEdge, ka = a.col == 1 ? t % kDepth : t / kEdge;
      as[ka][ra] = i0 + ra < m && k0 + ka < k ? as_float(pa[(i0 + ra) * a.row + (k0 + ka) * a.col]) : 0.f;
      const int rb = b.col == 1 ? t / kDepth : t % kEdge, kb = b.col == 1 ? t % kDepth : t / kEdge;
      bs[kb][rb] = j0 + rb < n && k0 + kb < k ? as_float(pb[(j0 + rb) * b.row + (k0 + kb) * b.col]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < kDepth; ++kk) {
      float av[4], bv[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) av[q] = as[kk][ty + 16 * q], bv[q] = bs[kk][tx + 16 * q];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[q][r] = fmaf(av[q], bv[r], acc[q][r]);
    }
    __syncthreads();
  }
  bool bad = false;
  for (int q = 0; q < 4; ++q)
    for (int r = 0; r < 4; ++r) {
      const int64_t i = i0 + ty + 16 * q, j = j0 + tx + 16 * r;
      if (i >= m || j >= n) continue;
      float z = acc[q][r];
      if (e.bias != nullptr) z += load_typed(e.bias, e.bias_dtype, j);
      if (e.z != nullptr) bad |= store_typed(e.z, dtype, i * e.ldz + j, z);
      z = activate(z, e.activation);
      if (e.residual != nullptr) z += load_typed(e.residual, e.residual_dtype, i * e.ld_residual + j);
      bad |= store_typed(e.y, e.y_dtype, i * e.ldy + j, z);
    }
  if (bad && dev_status != nullptr) atomicOr(dev_status, OPR_DEV_FP16_RANGE);
}

constexpr int kDzRows = 64;

// dz = dy act'(z) (written when dz is not null) and the column sums of each
// block's rows, taken before dz is rounded.  One column per thread.
template <typename T>
__global__ void __launch_bounds__(256) linear_dz_kernel(const T* dy, int64_t ld_dy, const T* z, int64_t ldz, int64_t m,
                                                        int32_t n, int32_t act, T* dz, int64_t ld_dz, float* partial,
                                                        int64_t rows_per_block, int32_t* dev_status) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (j >= n) return;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * rows_per_block;
  const int64_t r1 = r0 + rows_per_block < m ? r0 + rows_per_block : m;
  float sum = 0.f;
  bool bad = false;
  for (int64_t i = r0; i < r1; ++i) {
    float g = as_float(dy[i * ld_dy + j]);
    // __fmul_rn: one value for the sum and for dz, whether or not dz is wanted
    if (act != OPR_ACT_NONE) g = __fmul_rn(g, activate_slope(as_float(z[i * ldz + j]), act));
    sum += g;
    if (dz != nullptr) {
      bad |= beyond<T>(g);
      dz[i * ld_dz + j] = from_float<T>(g);
    }
  }
  if (partial != nullptr) partial[static_cast<int64_t>(blockIdx.y) * n + j] = sum;
  if (bad && dev_status != nullptr) atomicOr(dev_status, OPR_DEV_FP16_RANGE);
}

__global__ void __launch_bounds__(256) column_sum_kernel(const float* partial, int32_t blocks, int32_t n, float* out) {
  const int64_t j = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (j >= n) return;
  double t = 0.0;
  for (int b = 0; b < blocks; ++b) t += partial[static_cast<int64_t>(b) * n + j];
  out[j] = static_cast<float>(t);
}

}  // namespace

cudaError_t launch_linear(const Operand& a, const Operand& b, int64_t m, int32_t n, int64_t k, int32_t dtype,
                          const LinearEpilogue& e, int32_t* dev_status, cudaStream_t stream) {
  if (m == 0 || n == 0) return cudaSuccess;
  const dim3 grid(static_cast<unsigned>((m + kEdge - 1) / kEdge), static_cast<unsigned>((n + kEdge - 1) / kEdge));
  if (dtype == OPR_DTYPE_BF16)
    linear_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(a, b, m, n, k, dtype, e, dev_status);
  else
    linear_kernel<__half><<<grid, 256, 0, stream>>>(a, b, m, n, k, dtype, e, dev_status);
  return cudaGetLastError();
}

int32_t linear_dz_blocks(int64_t m) {
  return static_cast<int32_t>(std::min<int64_t>((m + kDzRows - 1) / kDzRows, 1024));
}

cudaError_t launch_linear_dz(const void* dy, int64_t ld_dy, const void* z, int64_t ldz, int32_t dtype, int64_t m,
                             int32_t n, int32_t activation, void* dz, int64_t ld_dz, float* db, float* partial,
                             int32_t* dev_status, cudaStream_t stream) {
  const int32_t blocks = linear_dz_blocks(m);
  const unsigned cols = static_cast<unsigned>((n + 255) / 256);
  if (blocks > 0) {
    const int64_t rows = (m + blocks - 1) / blocks;
    const dim3 grid(cols, blocks);
    float* part = db != nullptr ? partial : nullptr;
    if (dtype == OPR_DTYPE_BF16)
      linear_dz_kernel<__nv_bfloat16><<<grid, 256, 0, stream>>>(
          static_cast<const __nv_bfloat16*>(dy), ld_dy, static_cast<const __nv_bfloat16*>(z), ldz, m, n, activation,
          static_cast<__nv_bfloat16*>(dz), ld_dz, part, rows, dev_status);
    else
      linear_dz_kernel<__half><<<grid, 256, 0, stream>>>(static_cast<const __half*>(dy), ld_dy,
                                                         static_cast<const __half*>(z), ldz, m, n, activation,
                                                         static_cast<__half*>(dz), ld_dz, part, rows, dev_status);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  if (db == nullptr) return cudaSuccess;
  column_sum_kernel<<<cols, 256, 0, stream>>>(partial, blocks, n, db);
  return cudaGetLastError();
}

}  // namespace opr
