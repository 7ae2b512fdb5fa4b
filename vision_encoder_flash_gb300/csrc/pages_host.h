// pages_host.h -- the paged cache on the host: its pools as tensors, their tensor
// maps, and the launch of attention over it, which has translation units of its own.
#pragma once

#include <algorithm>
#include <cstdint>

#include "../../include/vattn_serving.h"
#include "paged_kernel.cuh"
#include "window_host.h"

namespace vattn {
namespace host {

inline FastDiv fast_div(int64_t d) { return FastDiv::make(static_cast<uint32_t>(std::max<int64_t>(1, d))); }

// The two pools of a cache as tensors [n_pages, heads, page_size, head_dim] of bytes.
struct Pools {
  vattn_rows k_rows, v_rows;
  Tensor k, v;
  Pools(const vattn_pages* c, int64_t heads, int64_t dim)
      : k_rows{c->k, {c->k_stride[0], c->k_stride[1], c->k_stride[2]}},
        v_rows{c->v, {c->v_stride[0], c->v_stride[1], c->v_stride[2]}},
        k{"k pages", &k_rows, {c->n_pages, heads, c->page_size}, dim, 1, true},
        v{"v pages", &v_rows, {c->n_pages, heads, c->page_size}, dim, 1, true} {}
  Pools(const Pools&) = delete;
};

// Tensor map {dim, rows of a page, heads, pages} of bytes with boxes of `cols`
// columns (32, 64 or 128: swizzled as wide) x `box` rows; what is outside reads 0.
inline vattn_status make_pages_map(CUtensorMap* tm, const Tensor& x, int cols, int box) {
  EncodeTiledFn enc = nullptr;
  const vattn_status st = tensor_map_encoder(&enc);
  if (st != VATTN_OK) return st;
  cuuint64_t dims[4] = {static_cast<cuuint64_t>(x.dim), static_cast<cuuint64_t>(x.size[2]),
                        static_cast<cuuint64_t>(x.size[1]), static_cast<cuuint64_t>(x.size[0])};
  cuuint64_t strides[3];
  const int order[3] = {2, 1, 0};
  for (int i = 0; i < 3; ++i)
    strides[i] = x.size[order[i]] <= 1 ? static_cast<cuuint64_t>(x.dim)
                                       : static_cast<cuuint64_t>(x.t->stride[order[i]]);
  const cuuint32_t boxes[4] = {static_cast<cuuint32_t>(cols), static_cast<cuuint32_t>(box), 1u, 1u};
  const cuuint32_t steps[4] = {1u, 1u, 1u, 1u};
  const CUresult r = enc(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, x.t->data, dims, strides, boxes, steps,
                         CU_TENSOR_MAP_INTERLEAVE_NONE,
                         cols == 128  ? CU_TENSOR_MAP_SWIZZLE_128B
                         : cols == 64 ? CU_TENSOR_MAP_SWIZZLE_64B
                                      : CU_TENSOR_MAP_SWIZZLE_32B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(VATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult %d", static_cast<int>(r));
  return VATTN_OK;
}

// paged_launch.cuh, in paged_f16.cu and paged_bf16.cu
template <typename T>
vattn_status paged_dispatch(const PagedParams& p, const Pools& pools, int sms, int device, cudaStream_t stream);

}  // namespace host
}  // namespace vattn
