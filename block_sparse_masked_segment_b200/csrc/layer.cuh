// layer.cuh - what the layer operators around the attention share: element
// conversions, the description of the rotated heads, and their launchers.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

#include "../../include/opr.h"

namespace opr {

template <typename T>
__device__ __forceinline__ float as_float(T v) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>)
    return __bfloat162float(v);
  else if constexpr (std::is_same_v<T, __half>)
    return __half2float(v);
  else
    return v;
}
template <typename T>
__device__ __forceinline__ T from_float(float v) {
  if constexpr (std::is_same_v<T, __nv_bfloat16>)
    return __float2bfloat16_rn(v);
  else if constexpr (std::is_same_v<T, __half>)
    return __float2half_rn(v);
  else
    return v;
}

// Element i of an array whose type is known at run time only.
__device__ __forceinline__ float load_typed(const void* p, int32_t dtype, int64_t i) {
  if (dtype == OPR_DTYPE_BF16) return __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
  if (dtype == OPR_DTYPE_FP16) return __half2float(static_cast<const __half*>(p)[i]);
  return static_cast<const float*>(p)[i];
}

// Is v, or what it was rounded from, stored as an infinity or NaN where the output is
// fp16?  Below 65520 it rounds to 65504 at most.
__device__ __forceinline__ bool beyond_f16(float v) { return !(fabsf(v) < 65520.f); }
template <typename TO>
__device__ __forceinline__ bool beyond(float v) {
  if constexpr (std::is_same_v<TO, __half>) return beyond_f16(v);
  return false;
}

inline int64_t dtype_bytes(int32_t t) { return t == OPR_DTYPE_FP32 ? 4 : 2; }
inline bool known_dtype(int32_t t) { return t == OPR_DTYPE_BF16 || t == OPR_DTYPE_FP16 || t == OPR_DTYPE_FP32; }

// Most of the layer's kernels may start while the one before them in the stream still runs
// (launch_overlapped): one sets up, waits here until that kernel is complete and its
// writes are visible, and only then lets the kernel behind it start and touches memory.  In
// this order, whatever starts early behind it finds all kernels but this one complete: a
// foreign kernel may read, before it waits itself, what they wrote (weights, say).
// It takes 1.1 to 1.4 us off each kernel of a sequence (one row of 6144 x 4096:
// 13.6 to 12.3 us; 128 x 64 x 64: 4.7 to 3.6).  Letting the next one start first, before
// the wait, would take off 0.1 more.
__device__ __forceinline__ void wait_for_previous() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Launches a kernel that may overlap the end of the one before it (wait_for_previous).
template <typename... P, typename... A>
inline cudaError_t launch_overlapped(void (*kernel)(P...), dim3 grid, int threads, size_t smem, int cluster,
                              cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---------------------------------------------------------------- rotated heads
// What happens to the heads of one tensor.
enum : int32_t { kHeadCopy = 0, kHeadRotate = 1, kHeadNormRotate = 2 };

// Heads of one tensor: x [total][heads][d] with x_stride elements from token to
// token (the heads of a token are contiguous), y alike.
struct HeadSet {
  const void* x;
  int64_t x_stride;
  void* y;
  int64_t y_stride;
  const void* w;  // kHeadNormRotate: [d], HeadArgs::w_dtype
  // gradients: x is the forward's input, dy [total][heads][d] the gradient of its
  // output, y the gradient of x, partial [blocks][d] the blocks' sums for w
  const void* dy;
  int64_t dy_stride;
  float* partial;
  float* w_grad;  // [d]
  int32_t heads;
  int32_t mode;
};

struct HeadArgs {
  HeadSet set[3];
  int32_t n_sets;
  const int32_t* pos;
  const double* freq;        // [pairs] radians per position
  const int32_t* row_map;    // output row of each token, or null
  int64_t total;
  int32_t d;
  int32_t pairs;             // rotated pairs: the first 2 * pairs entries of a head
  int32_t interleaved;
  int32_t inverse;
  float scale;               // on the rotated entries
  float eps;
  int32_t w_dtype;
  int32_t* dev_status;
};

cudaError_t launch_heads(const HeadArgs& a, int32_t x_dtype, int32_t y_dtype, cudaStream_t stream);
// Blocks per set of the gradient pass, which sizes the workspace of partial sums.
int32_t head_grad_blocks(int64_t total, int32_t heads);
cudaError_t launch_head_grads(const HeadArgs& a, int32_t x_dtype, int32_t dy_dtype, int32_t dx_dtype,
                              cudaStream_t stream);

// ---------------------------------------------------------------- matrix products
struct LinearEpilogue {
  const void* bias;  // [n] or null
  int32_t bias_dtype;
  int32_t activation;
  const void* residual;  // [m][n] or null
  int64_t ld_residual;
  int32_t residual_dtype;
  void* y;
  int64_t ldy;
  int32_t y_dtype;
  void* z;  // pre-activation [m][n], the operands' type, or null
  int64_t ldz;
};

// C[i][j] = sum_k A(i, k) B(j, k): element (r, k) of an operand is p[r * row + k * col].
struct Operand {
  const void* p;
  int64_t row, col;
};

cudaError_t launch_linear(const Operand& a, const Operand& b, int64_t m, int32_t n, int64_t k, int32_t dtype,
                          const LinearEpilogue& e, int32_t* dev_status, cudaStream_t stream);
// A 16-bit matrix to be copied to rows of ld_to entries (a multiple of eight; the
// entries past `cols` of a row's last eight are written as zeros); from null: none.
struct PackJob {
  const void* from;
  int64_t ld_from;
  void* to;
  int64_t ld_to, rows;
  int32_t cols;
};
cudaError_t launch_pack(const PackJob (&jobs)[2], cudaStream_t stream);
cudaError_t launch_linear_dz(const void* dy, int64_t ld_dy, const void* z, int64_t ldz, int32_t dtype, int64_t m,
                             int32_t n, int32_t activation, void* dz, int64_t ld_dz, float* db, float* partial,
                             int32_t* dev_status, cudaStream_t stream);
// Row blocks of the dz pass at most, which sizes its partial column sums.
int32_t linear_dz_blocks(int64_t m, int32_t n);

}  // namespace opr
