// host_common.h -- what the translation units of the library share on the
// host: error reporting, the per-device workspace pool and device facts.
// Defined in vattn_api.cu.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/vattn.h"

namespace vattn {
namespace host {

constexpr int kMaxDevices = 64;

// Clears / sets the calling thread's last-error text; fail returns `st`.
void clear_error();
vattn_status fail(vattn_status st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
vattn_status cuda_fail(cudaError_t e, const char* what);

// Streaming multiprocessors of `device`, read once per device.
vattn_status sm_count(int device, int* out);

// Device address of the status word that vattn_device_status reads.
vattn_status status_word(int device, uint32_t** out);

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// The driver's tensor-map encoder.
vattn_status tensor_map_encoder(EncodeTiledFn* out);

// Stream-ordered workspace of one call from the device's pool; goes back to
// the pool, in stream order, when the object dies.
class Workspace {
 public:
  Workspace() = default;
  Workspace(const Workspace&) = delete;
  Workspace& operator=(const Workspace&) = delete;
  ~Workspace() { (void)release(); }
  vattn_status take(size_t bytes, int device, cudaStream_t stream);
  vattn_status release();
  uint8_t* data() const { return static_cast<uint8_t*>(ptr_); }

 private:
  void* ptr_ = nullptr;
  cudaStream_t stream_ = nullptr;
};

}  // namespace host
}  // namespace vattn
