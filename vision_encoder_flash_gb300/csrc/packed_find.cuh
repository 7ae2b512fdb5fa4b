// packed_find.cuh -- a block's own pairs of attention over packed prompts
// (vattn_forward_packed), without a list in memory.
//
// The order of pairs is that of packed_list_kernel.cuh: by the last row block that
// a pair holds, late ones first, then by prompt.  A prompt of nb row blocks has
// floor((v + 1) group / 2) pairs that end in row blocks 0 .. v < nb - 1, so how
// many pairs end behind v is a sum over the prompts, of which a warp's lanes hold up
// to kFindPrompts.  The row block of the pair of a given rank is found by
// bisection, its prompt by a prefix sum: some 500 cycles a pair, the warps of the
// block taking its rounds in turn.  (A kernel for the list costs 3 us and, with its
// workspace, 5 us of host time.)
#pragma once

#include "window_common.cuh"

namespace vattn {

constexpr int kFindPrompts = 128;  // most prompts, 4 a lane
constexpr int kFindRounds = 64;    // most items of a block
constexpr int kFindTile = 128;     // rows of a row block

// The block's: {items, whole, 0, 0}, then of each round {first row, rows, pair, key head}.
__device__ __forceinline__ int4* found_pairs() {
  __shared__ int4 found[1 + kFindRounds];
  return found;
}

struct FindParams {
  const int32_t* cu;
  int n_seqs, total;
  int group, n_kv_heads, sms;
  FastDiv kv_heads;
};

// entry_of(r): the block's entry of round r (an item, or half of one where items are single units).
template <typename F>
__device__ __forceinline__ void find_pairs(const FindParams p, int warps, F&& entry_of) {
  constexpr int N = kFindPrompts / 32;
  const int warp = static_cast<int>(threadIdx.x) >> 5, lane = static_cast<int>(threadIdx.x) & 31;
  int first[N], rows[N], blocks[N];
  uint32_t low = 0, high = 0, all = 0, most = 0;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int b = lane + 32 * j;
    first[j] = rows[j] = blocks[j] = 0;
    if (b < p.n_seqs) {
      first[j] = min(max(p.cu[b], 0), p.total);
      rows[j] = max(0, min(max(p.cu[b + 1], 0), p.total) - first[j]);
      blocks[j] = (rows[j] + kFindTile - 1) / kFindTile;
    }
    low += static_cast<uint32_t>(rows[j]) & 0xffffu;
    high += static_cast<uint32_t>(rows[j]) >> 16;
  }
  low = __reduce_add_sync(0xffffffffu, low);
  high = __reduce_add_sync(0xffffffffu, high);
  // prompts with more rows than there are (starts that do not ascend): none is computed
  const bool bad = (static_cast<uint64_t>(high) << 16) + low > static_cast<uint64_t>(p.total);
  auto upto = [&](int j, int v) {  // pairs of the prompt that end in row blocks 0 .. v
    return v >= blocks[j] - 1 ? (blocks[j] * p.group + 1) / 2 : (v + 1) * p.group / 2;
  };
  if (!bad) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      all += static_cast<uint32_t>(upto(j, blocks[j]));
      most = max(most, static_cast<uint32_t>(blocks[j]));
    }
    all = __reduce_add_sync(0xffffffffu, all);
    most = __reduce_max_sync(0xffffffffu, most);
  }
  const int items = static_cast<int>(all) * p.n_kv_heads;
  const bool single = 2 * items <= p.sms;
  const int entries = single ? 2 * items : items;
  if (threadIdx.x == 0) found_pairs()[0] = make_int4(entries, single ? 0 : items, 0, 0);
  auto behind = [&](int v) {  // pairs of all prompts that end behind row block v
    uint32_t n = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) n += static_cast<uint32_t>(upto(j, blocks[j]) - upto(j, v));
    return static_cast<int>(__reduce_add_sync(0xffffffffu, n));
  };
  for (int r = warp; r < kFindRounds; r += warps) {
    const int entry = entry_of(r);
    if (entry >= entries) break;
    uint32_t kh;
    const int rank = static_cast<int>(p.kv_heads.div(static_cast<uint32_t>(single ? entry / 2 : entry), &kh));
    int lo = 0, hi = static_cast<int>(most) - 1;  // the first row block with no more than rank pairs behind it
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (behind(mid) <= rank) hi = mid;
      else lo = mid + 1;
    }
    const int v = lo;
    int left = rank - behind(v);  // its place among the pairs that end there
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int before = v * p.group / 2, n = blocks[j] > v ? upto(j, v) - before : 0;
      int to = n;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, to, o);
        if (lane >= o) to += y;
      }
      if (left >= to - n && left < to)
        found_pairs()[1 + r] = make_int4(first[j], rows[j], before + left - (to - n), static_cast<int>(kh));
      left -= __shfl_sync(0xffffffffu, to, 31);
    }
  }
}

}  // namespace vattn
