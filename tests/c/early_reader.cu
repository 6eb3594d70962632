// Two kernels around a library call, for tests/test_gpu_overlap.py: one that writes a word after
// a while, and one that starts as early as the kernel before it in the stream allows and
// reads the word before it waits for that kernel.
#include <cuda_runtime.h>

#include <cstdint>

namespace {

__global__ void late_writer(int32_t* word, int32_t value, uint32_t ns) {
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  for (int i = 0; i < (1 << 20); ++i) {  // bounded, also where the clock stood still
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (t - t0 > ns) break;
  }
  *word = value;
}

__global__ void early_reader(const int32_t* word, int32_t* out) {
  const int32_t seen = *static_cast<const volatile int32_t*>(word);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  *out = seen;
}

}  // namespace

extern "C" __attribute__((visibility("default"))) int write_late(int32_t* word, int32_t value, uint32_t ns, void* stream) {
  late_writer<<<1, 1, 0, static_cast<cudaStream_t>(stream)>>>(word, value, ns);
  return cudaGetLastError();
}

extern "C" __attribute__((visibility("default"))) int read_early(const int32_t* word, int32_t* out, void* stream) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(1);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, early_reader, word, out);
}
