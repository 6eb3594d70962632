// host_status.h - host-side pieces shared by the entry points: error reporting,
// the device check and the profiler range of a call.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <nvtx3/nvToolsExt.h>

#include "../../include/opr.h"

namespace opr {

// Records the text of a CUDA error for opr_last_error() on this host thread and
// returns OPR_CUDA_ERROR (defined in api.cu).
opr_status record_cuda_error(cudaError_t e);

// OPR_OK, or the recorded CUDA error.
inline opr_status status_of(cudaError_t e) { return e == cudaSuccess ? OPR_OK : record_cuda_error(e); }

// OPR_UNSUPPORTED unless the current device has compute capability 10.x (defined in api.cu).
opr_status device_check();

// Limit of the kernels' pipeline waits, as AttnParams::wait_ns (defined in api.cu).
uint32_t wait_limit_ns();

// Encodes a tiled TMA map with interleave off, 256-byte L2 promotion and zeros out
// of bounds; false when the driver refuses it (defined in api.cu).
bool encode_tiled(CUtensorMap* map, CUtensorMapDataType type, int rank, void* p, const cuuint64_t* dims,
                  const cuuint64_t* strides, const cuuint32_t* box, const cuuint32_t* elem_strides,
                  CUtensorMapSwizzle swizzle);

// Host check of the sizes shared by the layout and attention calls: non-negative,
// int32 token offsets, and total tokens within n_seqs * ceil(max_seqlen / 128) * 128,
// the bound the workspaces are sized by (defined in api.cu).
bool sizes_ok(int32_t n_seqs, int32_t n_convs, int32_t n_turns, int64_t total, int32_t max_seqlen);

// One NVTX range per entry-point call (named after the call), so that a
// profiler timeline shows where each library call's launches begin and end.
// Without an attached tool the push and pop cost a branch each.
struct CallRange {
  explicit CallRange(const char* name) { nvtxRangePushA(name); }
  ~CallRange() { nvtxRangePop(); }
  CallRange(const CallRange&) = delete;
  CallRange& operator=(const CallRange&) = delete;
};

}  // namespace opr
