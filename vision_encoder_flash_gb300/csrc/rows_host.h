// rows_host.h -- host side of the calls on strided tensors [batch, heads, rows,
// head_dim]: checks of their memory, tensor maps, launches.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>

#include "../../include/vattn_decoder.h"
#include "host_common.h"
#include "window_pipe.cuh"

namespace vattn {
namespace host {

inline int elem_size(int32_t dtype) { return dtype == VATTN_F32 ? 4 : 2; }

// ------------------------------------------------------------ tensor checks
// A tensor of a call: its rows and the sizes of its dimensions.
struct Tensor {
  const char* name;
  const vattn_rows* t;
  int64_t size[3];  // batch, heads, rows
  int64_t dim;
  int esize;
  bool out;

  uintptr_t base() const { return reinterpret_cast<uintptr_t>(t->data); }
  bool empty() const { return size[0] == 0 || size[1] == 0 || size[2] == 0; }
  // bytes from the first element to the end of the last row (stride checks passed)
  uint64_t extent() const {
    uint64_t e = static_cast<uint64_t>(dim);
    for (int i = 0; i < 3; ++i) e += static_cast<uint64_t>(size[i] - 1) * static_cast<uint64_t>(t->stride[i]);
    return e * static_cast<uint64_t>(esize);
  }
};

// Every element of a tensor of these sizes and strides has its own address:
// from the innermost dimension outwards each stride passes all that is inside.
inline bool distinct(const int64_t (&size)[3], const int64_t (&stride)[3], int64_t dim) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return stride[a] < stride[b]; });
  int64_t inside = dim;
  for (int i : order) {
    if (size[i] <= 1) continue;
    if (stride[i] < inside) return false;
    inside += (size[i] - 1) * stride[i];
  }
  return true;
}

inline vattn_status check_tensor(const Tensor& x, int row_align_bytes) {
  if (x.empty()) return VATTN_OK;
  if (!x.t || !x.t->data) return fail(VATTN_ERR_INVALID_ARG, "null %s", x.name);
  const char* dims[3] = {"batch", "head", "row"};
  for (int i = 0; i < 3; ++i) {
    const int64_t s = x.t->stride[i];
    if (x.size[i] <= 1) continue;
    if (s < 0) return fail(VATTN_ERR_INVALID_ARG, "%s: negative %s stride", x.name, dims[i]);
    if (s > (int64_t{1} << 38) || (x.size[i] - 1) > (int64_t{1} << 58) / (s > 0 ? s : 1))
      return fail(VATTN_ERR_UNSUPPORTED, "%s: %s stride %lld too large", x.name, dims[i], (long long)s);
    if (s * x.esize % row_align_bytes != 0)
      return fail(VATTN_ERR_MISALIGNED, "%s: %s stride %lld is not a multiple of %d bytes", x.name,
                  dims[i], (long long)s, row_align_bytes);
  }
  const int align = row_align_bytes > x.esize ? row_align_bytes : x.esize;
  if (x.base() % static_cast<uintptr_t>(align) != 0)
    return fail(VATTN_ERR_MISALIGNED, "%s must be %d-byte aligned", x.name, align);
  if (x.out && !distinct(x.size, x.t->stride, x.dim))
    return fail(VATTN_ERR_INVALID_ARG, "%s: elements share addresses (a broadcast or overlapping view)", x.name);
  return VATTN_OK;
}

inline bool same_rows(const Tensor& a, const Tensor& b) {
  if (a.base() != b.base() || a.dim != b.dim || a.esize != b.esize) return false;
  for (int i = 0; i < 3; ++i)
    if (a.size[i] != b.size[i] || (a.size[i] > 1 && a.t->stride[i] != b.t->stride[i])) return false;
  return true;
}

// No element of a is an element of b: their byte ranges are apart, or they
// are parts of one packed buffer: equal strides, the one's first element some
// whole number of strides behind the other's, a box around both whose elements
// are distinct, and a dimension in which one's indexes end before the other's
// begin.
inline bool apart(const Tensor& a, const Tensor& b) {
  if (a.empty() || b.empty()) return true;
  if (a.base() + a.extent() <= b.base() || b.base() + b.extent() <= a.base()) return true;
  const Tensor& lo = a.base() <= b.base() ? a : b;
  const Tensor& hi = a.base() <= b.base() ? b : a;
  if (lo.esize != hi.esize || lo.dim != hi.dim) return false;
  const uint64_t bytes = hi.base() - lo.base();
  if (bytes % static_cast<uint64_t>(lo.esize) != 0) return false;
  int64_t delta = static_cast<int64_t>(bytes / static_cast<uint64_t>(lo.esize));
  int64_t size[3], stride[3] = {0, 0, 0}, off[3] = {0, 0, 0};
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i) {
    if (lo.size[i] > 1 && hi.size[i] > 1 && lo.t->stride[i] != hi.t->stride[i]) return false;
    if (lo.size[i] > 1 || hi.size[i] > 1) {
      stride[i] = lo.size[i] > 1 ? lo.t->stride[i] : hi.t->stride[i];
      if (stride[i] <= 0) return false;
    }
  }
  std::sort(order, order + 3, [&](int x, int y) { return stride[x] > stride[y]; });
  for (int i : order)
    if (stride[i] > 0) {
      off[i] = delta / stride[i];
      delta -= off[i] * stride[i];
    }
  if (delta > 0) {  // one head each: their distance is the buffer's head stride
    if (stride[1] > 0) return false;
    stride[1] = delta;
    off[1] = 1;
  }
  bool clear = false;
  for (int i = 0; i < 3; ++i) {
    size[i] = std::max(lo.size[i], off[i] + hi.size[i]);
    clear |= off[i] >= lo.size[i];
  }
  return clear && distinct(size, stride, lo.dim);
}

inline vattn_status check_apart(const Tensor& a, const Tensor& b) {
  if (apart(a, b)) return VATTN_OK;
  return fail(VATTN_ERR_INVALID_ARG, "%s overlaps %s", a.name, b.name);
}

// Plain memory [p, p + bytes) against a tensor's range.
inline vattn_status check_apart_bytes(const void* p, uint64_t bytes, const char* name, const Tensor& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p);
  if (p == nullptr || bytes == 0 || b.empty()) return VATTN_OK;
  if (x + bytes <= b.base() || b.base() + b.extent() <= x) return VATTN_OK;
  return fail(VATTN_ERR_INVALID_ARG, "%s overlaps %s", name, b.name);
}

inline vattn_status current_device(int* device) {
  const cudaError_t e = cudaGetDevice(device);
  return e == cudaSuccess ? VATTN_OK : cuda_fail(e, "cudaGetDevice");
}

inline vattn_status launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VATTN_OK : cuda_fail(e, what);
}

// Launches a kernel whose blocks may start while the kernel before it on the
// stream ends (they wait with griddepcontrol.wait before they read its work).
template <typename K, typename... A>
vattn_status launch_behind(const char* what, K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                           const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess ? VATTN_OK : cuda_fail(e, what);
}

// Opts a kernel in to its dynamic shared memory, once per device.
template <typename K>
vattn_status allow_smem(K kernel, int bytes, std::atomic<uint8_t>* done, int device) {
  if (done[device].load(std::memory_order_acquire)) return VATTN_OK;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  done[device].store(1, std::memory_order_release);
  return VATTN_OK;
}

inline RowsTensor rows_tensor(const vattn_rows* t) {
  RowsTensor r{};
  if (t) {
    r.p = t->data;
    for (int i = 0; i < 3; ++i) r.s[i] = t->stride[i];
  }
  return r;
}

// Tensors that are read through a tensor map have their rows apart: a map's
// row stride is not below the row's own length.
inline vattn_status check_map_rows(const Tensor& x) {
  if (x.empty() || x.size[2] <= 1 || x.t->stride[2] >= x.dim) return VATTN_OK;
  return fail(VATTN_ERR_UNSUPPORTED, "%s: row stride %lld below head_dim (rows broadcast or overlapping)", x.name,
              (long long)x.t->stride[2]);
}

// Tensor map {dim, rows, heads, batch} of 16-bit rows with boxes of
// `box_cols` columns (64: 128-byte swizzle, 32: 64-byte) x `box_rows` rows;
// what is outside reads 0 and is not written.  A
// head or batch dimension of stride 0 (or size 1) becomes a single one, and
// *mul zeroes its coordinate.
inline vattn_status make_rows_map(CUtensorMap* tm, MapMul* mul, const Tensor& x, int32_t dtype, int box_rows,
                           int box_cols = 64) {
  EncodeTiledFn enc = nullptr;
  const vattn_status st = tensor_map_encoder(&enc);
  if (st != VATTN_OK) return st;
  const bool one_h = x.size[1] <= 1 || x.t->stride[1] == 0, one_b = x.size[0] <= 1 || x.t->stride[0] == 0;
  mul->h = one_h ? 0 : 1;
  mul->b = one_b ? 0 : 1;
  const cuuint64_t row = static_cast<cuuint64_t>(x.dim) * 2u;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(x.dim), static_cast<cuuint64_t>(x.size[2]),
                              static_cast<cuuint64_t>(one_h ? 1 : x.size[1]),
                              static_cast<cuuint64_t>(one_b ? 1 : x.size[0])};
  const cuuint64_t strides[3] = {x.size[2] <= 1 ? row : static_cast<cuuint64_t>(x.t->stride[2]) * 2u,
                                 one_h ? row : static_cast<cuuint64_t>(x.t->stride[1]) * 2u,
                                 one_b ? row : static_cast<cuuint64_t>(x.t->stride[0]) * 2u};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1u, 1u};
  const cuuint32_t steps[4] = {1u, 1u, 1u, 1u};
  const CUresult r = enc(tm, dtype == VATTN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         4, x.t->data, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(VATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult %d", static_cast<int>(r));
  return VATTN_OK;
}

}  // namespace host
}  // namespace vattn
