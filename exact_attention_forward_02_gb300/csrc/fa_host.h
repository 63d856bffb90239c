// fa_host.h -- host-side state that the library's translation units share (defined in
// fa_fwd.cu): device checks, the launch counter, the pipeline wait limit, the tensor-map
// encoder and the device-side status word. Internal; not part of the C ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

namespace fa_host {

// SM count and index of the current device; FA_ERR_DEVICE when it is not an sm_103 GPU.
__attribute__((visibility("hidden"))) int current_device(int* index, int* sms);
// Device address of the status word on the current device (looked up once per device).
__attribute__((visibility("hidden"))) int status_word(int** out);
// Counts a launch and turns its outcome into a status code.
__attribute__((visibility("hidden"))) int launched(cudaError_t e);
__attribute__((visibility("hidden"))) unsigned long long wait_limit_ns();
// The cut of fa_debug_cap_workspace in floats, or -1 (always, in release builds).
__attribute__((visibility("hidden"))) long long debug_part_cap();
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);
__attribute__((visibility("hidden"))) EncodeTiledFn encode_tiled();

constexpr int MAX_DEVICES = 64;

}  // namespace fa_host
