// packed_list_kernel.cuh -- the work list of attention over packed prompts
// (vattn_forward_packed).
//
// The windowed forward kernel takes pairs of units (128 query rows of one head) of
// one sequence, longest first.  With lengths on the device, one block writes
// them down: a pair counts for the last row block that it holds, which its key
// tiles follow, a counting sort puts the pairs of late row blocks first, and
// pairs of one row block come in any order (no result depends on it).  Prompts that
// together have more rows than there are (starts that do not ascend) make an empty
// list: the room for it is that of prompts that do not overlap.  A warp stops where its
// own prompts are too many already, so whatever the starts hold, its pairs are no more
// than those of prompts that fit.
#pragma once

#include "window_pipe.cuh"

namespace vattn {

constexpr int kListThreads = 1024;
constexpr int kListBuckets = 8192;  // counts in shared memory up to here (2^20 rows), else in the workspace

struct PackedListParams {
  const int32_t* cu;
  int n_seqs, total;
  int group, kv_heads, sms;
  int buckets;  // row blocks of the longest sequence there can be
  int* counts;  // [buckets] or null: shared memory
  int4* list;   // {items, whole, 0, 0}, then {first row, rows, pair, 0} each
};

__global__ void __launch_bounds__(kListThreads) vattn_packed_list_kernel(const __grid_constant__ PackedListParams p) {
  __shared__ int counts_s[kListBuckets];
  __shared__ int warps_s[kListThreads / 32];
  __shared__ long long rows_s[kListThreads / 32];
  ptx::grid_dep_launch();  // the attention kernel sets itself up meanwhile, and waits for this one's end
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  constexpr int threads = kListThreads, warps = threads / 32;
  int* const counts = p.counts != nullptr ? p.counts : counts_s;
  for (int i = tid; i < p.buckets; i += threads) counts[i] = 0;
  __syncthreads();
  // (first row, rows, pair, its last row block): a warp has up to 32 prompts at a time, whose
  // lanes take the pairs of short ones by themselves and of long ones together
  const int at_a_time = min(32, (p.n_seqs + warps - 1) / warps);
  auto pairs_of = [&](int rows) { return (static_cast<long long>((rows + kTile - 1) / kTile) * p.group + 1) / 2; };
  auto block_of = [&](int rows, long long i) {
    return min((rows + kTile - 1) / kTile - 1, static_cast<int>((2 * i + 1) / p.group));
  };
  auto each = [&](auto&& take) {  // -> rows of the warp's prompts
    long long sum = 0;
    for (int b0 = warp * at_a_time; b0 < p.n_seqs; b0 += warps * at_a_time) {
      const int b = b0 + lane;
      int first = 0, rows = 0;
      if (lane < at_a_time && b < p.n_seqs) {
        first = min(max(p.cu[b], 0), p.total);
        rows = max(0, min(max(p.cu[b + 1], 0), p.total) - first);
      }
      sum += __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(rows) & 0xffffu) +
             (static_cast<long long>(__reduce_add_sync(0xffffffffu, static_cast<uint32_t>(rows) >> 16)) << 16);
      if (sum > p.total) break;
      const long long pairs = rows > 0 ? pairs_of(rows) : 0;
      const bool alone = pairs <= 8;
      if (alone)
        for (int i = 0; i < static_cast<int>(pairs); ++i) take(first, rows, i, block_of(rows, i));
      for (uint32_t left = __ballot_sync(0xffffffffu, !alone); left != 0; left &= left - 1) {
        const int l = __ffs(static_cast<int>(left)) - 1;
        const int f = __shfl_sync(0xffffffffu, first, l), n = __shfl_sync(0xffffffffu, rows, l);
        const long long all = pairs_of(n);
        for (long long i = lane; i < all; i += 32) take(f, n, static_cast<int>(i), block_of(n, i));
      }
    }
    return sum;
  };
  const long long mine = each([&](int, int, int, int block) { atomicAdd(&counts[block], 1); });
  if (lane == 0) rows_s[warp] = mine;
  __syncthreads();
  // counts to places: behind the pairs of all later row blocks
  const int per = (p.buckets + threads - 1) / threads;
  int sum = 0;
  for (int i = tid * per; i < min(p.buckets, (tid + 1) * per); ++i) sum += counts[p.buckets - 1 - i];
  int upto = sum;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  if (lane == 31) warps_s[warp] = upto;
  __syncthreads();
  int before = upto - sum, all = 0;
  long long rows = 0;
  for (int i = 0; i < warps; ++i) {
    if (i < warp) before += warps_s[i];
    all += warps_s[i];
    rows += rows_s[i];
  }
  if (rows > p.total) {
    if (tid == 0) p.list[0] = make_int4(0, 0, 0, 0);
    return;
  }
  for (int i = tid * per; i < min(p.buckets, (tid + 1) * per); ++i) {
    const int n = counts[p.buckets - 1 - i];
    counts[p.buckets - 1 - i] = before;
    before += n;
  }
  __syncthreads();
  each([&](int first, int rows, int pair, int block) {
    const int at = atomicAdd(&counts[block], 1);
    p.list[1 + at] = make_int4(first, rows, pair, 0);
  });
  if (tid == 0) {
    const int items = all * p.kv_heads;
    const bool single = 2 * items <= p.sms;  // every unit an item of its own, as forward_window does
    p.list[0] = make_int4(single ? 2 * items : items, single ? 0 : items, 0, 0);
  }
}

}  // namespace vattn
