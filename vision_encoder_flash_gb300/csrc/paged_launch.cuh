// paged_launch.cuh -- variant choice and launches of attention over the paged cache
// (vattn_forward_paged, checked by serving_api.cu).
#pragma once

#include <atomic>

#include "pages_host.h"

namespace vattn {
namespace host {

// Blocks of a kernel that a multiprocessor holds, asked once per device.
template <typename K>
vattn_status resident_blocks(K kernel, int threads, int smem, std::atomic<int>* known, int device, int* out) {
  *out = known[device].load(std::memory_order_acquire);
  if (*out > 0) return VATTN_OK;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(out, kernel, threads, static_cast<size_t>(smem));
  if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor");
  *out = std::max(1, *out);
  known[device].store(*out, std::memory_order_release);
  return VATTN_OK;
}

template <typename T, int DP, int NB, int RW, int kDim>
vattn_status paged_launch(PagedParams p, const Pools& pools, int sms, int device, cudaStream_t stream) {
  using P = PagedPlan<DP, NB, RW>;
  auto kernel = vattn_paged_kernel<T, DP, NB, RW, kDim>;
  static std::atomic<uint8_t> done[kMaxDevices];
  static std::atomic<int> known[kMaxDevices];
  vattn_status st = allow_smem(kernel, P::kSmemBytes, done, device);
  if (st != VATTN_OK) return st;
  int resident = 0;
  if ((st = resident_blocks(kernel, P::kThreads, P::kSmemBytes, known, device, &resident)) != VATTN_OK) return st;
  p.log_box = P::kLogStep;  // boxes as large as a step, if pages are
  while (p.page % (1 << p.log_box) != 0) --p.log_box;
  p.box = 1 << p.log_box;
  const long long seqs = static_cast<long long>(p.w.batch) * p.w.kv_heads;
  p.row_blocks = (p.rows + P::kRows - 1) / P::kRows;
  if (seqs * p.row_blocks > kMaxRows || seqs * p.rows > INT32_MAX)
    return fail(VATTN_ERR_UNSUPPORTED, "too many query rows");
  // Shares of the keys, as many for each sequence, from what the table has room for (lengths
  // are on the device; shares behind a sequence's end are empty): as many blocks as are
  // resident at a time, of 256 keys at least, or of 128 where that makes no more than 32
  // shares.  Four, which a cluster joins, where that leaves a warp five steps at most and
  // enough blocks: 4 us less host time for a call than more shares and their join on the
  // device, and from 24 blocks on about the same device time (24 blocks of 600 to 2500 keys
  // x 64 5.9 to 7.6 us, with more shares 6.4 to 7.5, x 128 6.8 to 8.9 and 6.1 to 8.3; 32
  // blocks x 128 6.8 to 9.1 and 6.7 to 9.1).  With fewer blocks the device pays for it: 16
  // of 2500 keys x 128 8.8 and 8.4, 10 8.8 and 7.2; with 4, where the rule does not hold,
  // 8.7 and 6.2.
  const long long most_keys = std::min<long long>(p.w.n_keys, static_cast<long long>(p.w.sinks) + p.w.window + p.w.n_queries);
  const long long blocks = seqs * p.row_blocks, room = static_cast<long long>(resident) * sms;
  const long long fill = room / blocks >= 4 ? room / blocks : (room + blocks - 1) / blocks;
  const long long fine = std::max(std::min(32LL, (most_keys + 127) / 128), (most_keys + 255) / 256);
  p.splits = static_cast<int>(std::max(1LL, std::min({fill, fine, static_cast<long long>(kCachedMaxSplits)})));
  if (p.splits > kPagedCluster && most_keys <= kPagedCluster * 5LL * P::kStepKeys && blocks * kPagedCluster >= sms / 4)
    p.splits = kPagedCluster;
  if (blocks * p.splits > kMaxRows) p.splits = 1;
  p.d_splits = fast_div(p.splits);
  p.d_row_blocks = fast_div(p.row_blocks);
  Workspace ws;
  const bool clustered = p.splits > 1 && p.splits <= kPagedCluster;
  if (p.splits > 1 && !clustered) {
    const size_t rows = static_cast<size_t>(blocks) * p.splits * P::kRows;
    if ((st = ws.take(rows * (p.w.dim + 2) * 4, device, stream)) != VATTN_OK) return st;
    p.part_o = reinterpret_cast<float*>(ws.data());
    p.part_ml = p.part_o + rows * p.w.dim;
  }
  CUtensorMap tk{}, tv{};
  if (paged_tight(kDim)) {
    for (int i = 0; i < 2; ++i) {
      const vattn_rows* t = i == 0 ? pools.k.t : pools.v.t;
      p.pool[i] = static_cast<const uint8_t*>(t->data);
      p.ps[i][0] = t->stride[0];
      p.ps[i][1] = t->stride[1];
    }
  } else if (pools.k.empty()) {  // no box is ever loaded: any valid map does
    vattn_rows any{const_cast<void*>(p.q.p), {0, 0, 0}};
    const Tensor t{"q", &any, {1, 1, 1}, p.w.dim, 1, false};
    if ((st = make_pages_map(&tk, t, DP, p.box)) != VATTN_OK) return st;
    tv = tk;
  } else if ((st = make_pages_map(&tk, pools.k, DP, p.box)) != VATTN_OK ||
             (st = make_pages_map(&tv, pools.v, DP, p.box)) != VATTN_OK) {
    return st;
  }
  const dim3 grid(static_cast<unsigned>(blocks * p.splits));
  if (clustered) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(P::kThreads);
    cfg.dynamicSmemBytes = P::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.splits);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tk, tv, p);
    return e == cudaSuccess ? VATTN_OK : cuda_fail(e, "paged attention kernel launch");
  }
  kernel<<<grid, P::kThreads, P::kSmemBytes, stream>>>(tk, tv, p);
  if ((st = launched("paged attention kernel launch")) != VATTN_OK) return st;
  if (p.splits == 1) return VATTN_OK;
  const long long out_rows = seqs * p.rows;
  const long long join_blocks = out_rows * ((p.w.dim + 31) / 32);
  if (p.splits <= 32 && join_blocks > 2 * sms)  // a warp a row, else blocks that share a row
    st = launch_behind("paged attention join kernel launch", vattn_paged_join_few_kernel<T, P::kRows, P::kKw>,
                       dim3(static_cast<unsigned>((out_rows + 7) / 8)), dim3(256), 0, stream, p);
  else
    st = launch_behind("paged attention join kernel launch", vattn_paged_join_kernel<T, P::kRows, P::kKw>,
                       dim3(static_cast<unsigned>(out_rows), static_cast<unsigned>((p.w.dim + 31) / 32)), dim3(256), 0,
                       stream, p);
  if (st != VATTN_OK) return st;
  return ws.release();
}

// The rows of a block: 8 NB a warp, which each word of keys and values that it makes f16
// serves, RW such groups; the warps left share the keys.  At head_dim 128 a warp's
// registers hold 24 rows of O: 17 to 24 rows in two groups of 16 took 21.4 us where one of
// 24 takes 19.6 (24 rows, 32 x 8000 keys; head_dim 64 16.4 and 14.1), 33 to 48 in four of
// 16 took 204 us, in two of 24 150 (44 rows, 52 x 38131 keys).  Beyond, blocks of 48 rows
// where they need little more time than those of 64: a block of 48 takes 0.62 to 0.72
// of one of four groups of 16 (head_dim 128: 128 rows 73.4 and 78.7 us, 64 rows 93.6 and
// 67.2), and 0.75 of one of two groups of 32, for which smaller rows have room (head_dim
// 64, 64 x 8000 keys, 64 rows: 41.1 us, in four of 16 46.4, in two blocks of 48 61.4).
template <typename T, int DP, int kDim>
vattn_status paged_rows(const PagedParams& p, const Pools& pools, int sms, int device, cudaStream_t stream) {
  if (p.rows <= 8) return paged_launch<T, DP, 1, 1, kDim>(p, pools, sms, device, stream);
  if (p.rows <= 16) return paged_launch<T, DP, 2, 1, kDim>(p, pools, sms, device, stream);
  if (p.rows <= 24) return paged_launch<T, DP, 3, 1, kDim>(p, pools, sms, device, stream);
  if (p.rows <= 32) return paged_launch<T, DP, 2, 2, kDim>(p, pools, sms, device, stream);
  const int by48 = (p.rows + 47) / 48, by64 = (p.rows + 63) / 64;
  if constexpr (DP <= 64) {
    if (3 * by48 < 4 * by64) return paged_launch<T, DP, 3, 2, kDim>(p, pools, sms, device, stream);
    return paged_launch<T, DP, 4, 2, kDim>(p, pools, sms, device, stream);
  } else {
    if (2 * by48 <= 3 * by64) return paged_launch<T, DP, 3, 2, kDim>(p, pools, sms, device, stream);
    return paged_launch<T, DP, 2, 4, kDim>(p, pools, sms, device, stream);
  }
}

template <typename T>
vattn_status paged_dispatch(const PagedParams& p, const Pools& pools, int sms, int device, cudaStream_t stream) {
  // rows of an odd number of 16 bytes that follow each other in their page: by untiled
  // copies (both sides' times are at vattn_paged_kernel)
  const bool tight = pools.k.t->stride[2] == p.w.dim && pools.v.t->stride[2] == p.w.dim;
  if (p.w.dim <= 32) return paged_rows<T, 32, 0>(p, pools, sms, device, stream);
  if (p.w.dim == 48 && tight) return paged_rows<T, 64, 48>(p, pools, sms, device, stream);
  if (p.w.dim <= 64) return paged_rows<T, 64, 0>(p, pools, sms, device, stream);
  if (p.w.dim == 80 && tight) return paged_rows<T, 128, 80>(p, pools, sms, device, stream);
  if (p.w.dim == 96) return paged_rows<T, 128, 96>(p, pools, sms, device, stream);
  if (p.w.dim == 112 && tight) return paged_rows<T, 128, 112>(p, pools, sms, device, stream);
  return paged_rows<T, 128, 0>(p, pools, sms, device, stream);
}

}  // namespace host
}  // namespace vattn
