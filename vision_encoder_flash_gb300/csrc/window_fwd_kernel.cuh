// window_fwd_kernel.cuh -- causal attention under a sliding window with
// visible first keys (vattn_forward_window), on the tensor cores.
//
// A unit is 128 query rows of one head.  Its row at position p sees keys j
// <= p with j > p - window or j < sinks, so it reads the key tiles of the
// first keys and those from its first row's window to its last row; no other
// tile is loaded.  A work item is two units of one key head, consecutive in
// (row block, head of the group): with an even group both have the same
// rows, hence the same tiles, and each K and V tile that comes from L2
// serves 256 query rows.  The grid is one block per multiprocessor, each
// walking over items from the longest to the shortest (late rows first).  A
// call with few items takes each unit by itself.
//
// Two products of 2 D flops and one exponential a pair: the tensor core needs
// 65 cycles for each 128 x 128 x 16, the four warps of a unit about 1300 for the
// exponentials of a tile pair, and the two are coupled tile by tile.  1 x 32(8)
// x 2048 x 128 without a window 32.6 us, 1056 TFLOP/s on the visible pairs (55 %
// of the measured rate); 1 x 8 x 8192 x 64 90.8 us, 755 TFLOP/s.  Under a window
// the first and the last tile of a row block are half masked and the tile of the
// first keys nearly all: 1 x 16(4) x 8192 x 128, window 1024, 4 first keys, 71.3
// us, 908 TFLOP/s.
//
//   warp 0   K and V tiles by TMA into a ring (K0 V0 K1 V1 ...)
//   warp 2   the item's two Q tiles by TMA
//   warp 1   issues S_t = Q_t K^T and O_t += P_t V (tcgen05.mma, TMEM
//            accumulators) from one thread, so they run in order; its loops
//            are unrolled with the descriptors as 32-bit halves: 65 cycles a
//            128 x 128 x 16 product, the tensor core's rate, where a rolled
//            loop took 100 to 130
//   warp 3   cleans V tiles in a second pass (below)
//   warps 4-7, 8-11   online softmax of unit 0, 1: thread = query row
//
// TMEM (512 columns).  head_dim <= 64: S_t at 128 t, P_t at 256 + 64 t, O_t at
// 384 + 64 t; the next S_t is issued as soon as this one is in registers.
// Above: S_t at 128 t, O_t at 256 + 128 t, and P_t (16-bit) overwrites S_t; the
// next S_t is issued behind the P_t V that reads P_t, and one unit's softmax
// runs while the tensor core works for the other.
//
// Statistics and accumulators are f32.  The weights are rounded to the
// tensors' type for the second product (relative 2^-9 / 2^-12 at most, and in f16
// 2^-32 of the row's largest; the sum l takes them unrounded), as the product
// needs; O is rescaled in TMEM only when a row's maximum grew by more than 2^8
// (exact after the final 1 / l).  A masked score is -infinity by selection, so
// nothing that K holds there gets through, and V rows behind the sequence are
// zeroed in shared memory before the product.
//
// Other masked V elements that are not finite would stay in O as 0 x infinity.  A
// warp whose results are not finite although its weights are looks whether such
// an element, in a partly masked tile, is hidden from one of its rows
// (window_leak); if so the block takes its items from the first such one to the
// last once more, with every partly masked V tile cleaned by warp 3 before its
// product, and what was taken out added to the O of the rows that see it.  Both
// looks are at two to five tiles of an item, whatever its length: 16(4) heads x 8192
// x 128, window 1024, as calls 77 us; with a NaN at a first key 122; with nothing
// but NaN in V 513.  (Cleaning in the only pass: clean calls 4 to 19 % slower, by
// the look itself and by the registers that it takes from the softmax.)
#pragma once

#include "window_pipe.cuh"

namespace vattn {

struct WindowFwdParams {
  WindowParams w;
  RowsTensor q, k, v, out;
  float* lse;
  uint32_t* status;
  MapMul mq, mk, mv, mo;
  int pairs;           // items of one (batch, key head): its units by twos
  int units;           // ceil(n_queries / 128) * group
  int items;           // < 2^30
  int whole;           // items from here on are single units (none of them, or all)
  FastDiv seqs, kv_heads, group;  // batch * kv_heads, kv_heads, group
  float scale_log2;    // scale * log2(e)
};

// Key tiles [0, ns) and [a, b] of one unit (b < a: none).
struct UnitRange {
  int ns, a, b;
  __device__ __forceinline__ bool empty() const { return b < a; }
  __device__ __forceinline__ bool uses(int j) const { return j < ns || (j >= a && j <= b); }
};

__device__ __forceinline__ UnitRange unit_range(const WindowParams& w, const Seq& s, int row0) {
  UnitRange u{0, 0, -1};
  const int lo = max(0, s.start + row0);
  const int hi = min(s.start + min(row0 + kTile, w.n_queries), s.len) - 1;
  if (hi < lo) return u;
  u.a = max(0, lo - w.window + 1) / kTile;
  u.b = hi / kTile;
  u.ns = min((min(w.sinks, s.len) + kTile - 1) / kTile, u.a);
  return u;
}

// One item: its two units and the tiles that either uses, in order.
struct WindowItem {
  int b, kh;
  int head[2], row0[2];
  bool on[2];
  UnitRange u[2];
  Seq s;
  int first_n, second, n;  // tiles 0 .. first_n - 1, then second, second + 1, ...
  __device__ __forceinline__ int tile(int x) const { return x < first_n ? x : second + (x - first_n); }
};

// The block's item of round r: back and forth over the blocks, so that none
// has the longer item of every round (1 x 32(8) x 2048 x 128 without a window:
// 33.2 us, in the same order every round 46.6; 2 x 16(4) x 4096 x 64, window
// 1024: 52.6 and 59.0).
__device__ __forceinline__ int window_entry(int r) {
  const int grid = static_cast<int>(gridDim.x), k = static_cast<int>(blockIdx.x);
  return r * grid + ((r & 1) ? grid - 1 - k : k);
}

__device__ __forceinline__ WindowItem window_item(const WindowFwdParams& p, int entry) {
  WindowItem it;
  uint32_t bk, kh;
  const bool pair_on = entry < p.whole;
  const int item = pair_on ? entry : p.whole + (entry - p.whole) / 2, only = (entry - p.whole) & 1;
  const int pair = p.pairs - 1 - static_cast<int>(p.seqs.div(static_cast<uint32_t>(item), &bk));
  it.b = static_cast<int>(p.kv_heads.div(bk, &kh));
  it.kh = static_cast<int>(kh);
  it.s = window_seq(p.w, it.b);
  int last = -1, first = 0x7fffffff;
  it.first_n = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int unit = 2 * pair + t;
    uint32_t g;
    it.on[t] = unit < p.units && (pair_on || only == t);
    it.row0[t] = static_cast<int>(p.group.div(static_cast<uint32_t>(unit), &g)) * kTile;
    it.head[t] = it.kh * p.w.group + static_cast<int>(g);
    it.u[t] = it.on[t] ? unit_range(p.w, it.s, it.row0[t]) : UnitRange{0, 0, -1};
    if (!it.u[t].empty()) {
      it.first_n = max(it.first_n, it.u[t].ns);
      first = min(first, it.u[t].a);
      last = max(last, it.u[t].b);
    }
  }
  it.second = max(first, it.first_n);
  it.n = last < 0 ? 0 : it.first_n + max(0, last - it.second + 1);
  return it;
}

template <int NKB>
struct WindowFwdPlan {
  static constexpr int kTileBytes = NKB * kBlockBytes;
  static constexpr int kStages = NKB == 1 ? 8 : 4;  // K and V tiles
  static constexpr int kOffQ = 0;
  static constexpr int kOffKv = 2 * kTileBytes;
  // results: two buffers a softmax warp of 32 rows x 32 elements (64-byte swizzle)
  static constexpr int kOffOut = kOffKv + kStages * kTileBytes;
  static constexpr int kOffBar = kOffOut + 8 * 4096;
  static constexpr int kSmemBytes = kOffBar + 640 + 1024;  // + alignment slack
  static constexpr uint32_t kVStages = kStages / 2;
  static constexpr int kThreads = 384;
  static constexpr bool kOwnP = NKB == 1;  // P has TMEM columns of its own
  static constexpr uint32_t kColP = kOwnP ? 256 : 0, kStrideP = kOwnP ? 64 : 128;
  static constexpr uint32_t kColO = kOwnP ? 384 : 256, kStrideO = kOwnP ? 64 : 128;
  // registers: 72 + 2 x 216 a thread = 3 x 168, what the launch has
  static constexpr uint32_t kRegsOther = 72, kRegsSoftmax = 216;
  static_assert(kSmemBytes <= 232448, "shared memory");
};

enum WindowBar : int {
  kWbQFull = 0, kWbQEmpty = 1, kWbKvFull = 2, kWbKvEmpty = 10, kWbSFull = 18, kWbPFull = 20,
  kWbPvDone = 22, kWbSFree = 24, kWbMmaDone = 26, kWbCount = 27,
  // second pass: a set of its own, and these
  kWbVLanded = 27, kWbNotes = 31, kWbNotesFree = 33, kWbSecondCount = 35,
};

// What the roles of a block share, and behind the pipe's words: the rounds of the
// second pass, from and to, and [2] tiles of an item that were cleaned in it (see
// window_add_back).
struct WindowCtx {
  const WindowFwdParams& p;
  Pipe pipe;
  uint32_t base_s, tmem;
  int warp, lane;
  __device__ __forceinline__ int again(int i) const {
    return static_cast<int>(ptx::ld_shared_volatile(pipe.at + kPipeBytes + 4 * i));
  }
  __device__ __forceinline__ uint32_t note_at(uint32_t i) const { return pipe.at + kPipeBytes + 8 + 4 * i; }
  // All threads of the block, after the first pass: is there a second?
  __device__ __forceinline__ bool second() const {
    ptx::tc_fence_before();
    __syncwarp();  // the loaders' lanes come one by one
    ptx::named_barrier_sync(1, 384);
    ptx::tc_fence_after();
    return again(0) <= again(1) && !pipe.aborted();
  }
};

// Two 16-bit elements at once: a + x * 0, NaN from the first x that is not finite.
template <typename T>
__device__ __forceinline__ uint32_t poison2(uint32_t x, uint32_t a) {
  uint32_t d;
  if constexpr (Elem<T>::kBf16)
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(a));
  else
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(x), "r"(0u), "r"(a));
  return d;
}
template <typename T>
__device__ __forceinline__ bool not_finite(uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  return (poison2<T>(x, poison2<T>(y, poison2<T>(z, poison2<T>(w, 0u)))) & 0x7fff7fffu) != 0;
}

// Tiles of an item with a key that is hidden from one of its rows that see any
// (rows from the first of its first unit to the last of its last).
struct WindowMasked {
  int full_first, full_last, sinks;
  __device__ __forceinline__ WindowMasked(const WindowParams& w, const WindowItem& it) : sinks(w.sinks) {
    const int lo = max(0, it.s.start + (it.on[0] ? it.row0[0] : it.row0[1]));
    const int hi = min(it.s.start + min((it.on[1] ? it.row0[1] : it.row0[0]) + kTile, w.n_queries), it.s.len) - 1;
    full_last = (lo + 1) / kTile - 1;
    full_first = (max(0, hi - w.window + 1) + kTile - 1) / kTile;
  }
  __device__ __forceinline__ bool operator()(int j) const {
    return j > full_last || (j < full_first && (j + 1) * kTile > sinks);
  }
};

// Keys of tile j that the thread's row of unit t sees, 32 a word.
struct WindowSee {
  int pos;  // of the row; -1 where it sees nothing
  __device__ __forceinline__ WindowSee(const WindowParams& w, const WindowItem& it, int t) {
    const int row = (t == 0 ? it.row0[0] : it.row0[1]) + static_cast<int>(threadIdx.x & 127);
    const int at = it.s.start + row;
    pos = row < w.n_queries && at >= 0 && at < it.s.len ? at : -1;
  }
  __device__ __forceinline__ uint32_t word(const WindowParams& w, int j, int c) const {
    const int k0 = j * kTile;
    return pos < 0 ? 0u
                   : bits_upto(pos - k0, c) & (~bits_upto(pos - w.window - k0, c) | bits_upto(w.sinks - 1 - k0, c));
  }
};

// Does V hold something that is not finite at a key which is hidden from one of
// the warp's rows (unit t of an item), in a tile that the unit uses?
template <typename T>
__device__ __noinline__ bool window_leak(const WindowFwdParams& p, int entry, int t) {
  const WindowItem it = window_item(p, entry);
  const WindowMasked masked(p.w, it);
  const WindowSee see(p.w, it, t);
  const UnitRange u = t == 0 ? it.u[0] : it.u[1];
  const int lane = static_cast<int>(threadIdx.x) & 31, chunks = p.w.dim / 8;
  bool leak = false;
  for (int x = 0; x < it.n; ++x) {
    const int j = it.tile(x);
    if (!u.uses(j) || !masked(j)) continue;
    uint32_t hidden[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) hidden[c] = __reduce_or_sync(0xffffffffu, see.pos < 0 ? 0u : ~see.word(p.w, j, c));
    const T* v = rows_at<T>(p.v, it.b, it.kh, j * kTile);
    const int end = min(kTile, it.s.len - j * kTile) * chunks;
#pragma unroll 8
    for (int i = lane; i < end; i += 32) {
      const int r = i / chunks;
      const uint4 y = *reinterpret_cast<const uint4*>(v + r * p.v.s[2] + (i - r * chunks) * 8);
      const uint32_t h = r < 64 ? (r < 32 ? hidden[0] : hidden[1]) : (r < 96 ? hidden[2] : hidden[3]);
      leak |= ((h >> (r & 31)) & 1u) != 0 && not_finite<T>(y.x, y.y, y.z, y.w);
    }
  }
  return __any_sync(0xffffffffu, leak);
}

// Elements that are not finite in the `left` rows of a V tile that belong to the
// sequence become zeros (one warp).  Were there any?
template <typename T, int NKB>
__device__ __forceinline__ bool window_clean_v(uint32_t v, int left) {
  constexpr uint32_t kExp = Elem<T>::kBf16 ? 0x7f80u : 0x7c00u;
  const int lane = static_cast<int>(threadIdx.x) & 31, end = min(left, kTile) * 8;  // 16-byte chunks of 64 columns
  bool any = false;
  for (int kb = 0; kb < NKB; ++kb)
    for (int i = lane; i < end; i += 32) {
      const uint32_t at = v + kb * kBlockBytes + i * 16;
      const float4 x = ptx::ld_shared_v4(at);
      uint32_t y[4] = {__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z), __float_as_uint(x.w)};
      if (!not_finite<T>(y[0], y[1], y[2], y[3])) continue;
      any = true;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        y[e] &= ((y[e] & kExp) == kExp ? 0u : 0xffffu) | (((y[e] >> 16) & kExp) == kExp ? 0u : 0xffff0000u);
      ptx::st_shared_v4(at, __uint_as_float(y[0]), __uint_as_float(y[1]), __uint_as_float(y[2]), __uint_as_float(y[3]));
    }
  ptx::fence_proxy_async_smem();
  return __any_sync(0xffffffffu, any);
}

// What window_clean_v took out of the item's tiles, added to the O of unit t's
// rows in TMEM (one warp, its 32 rows); bit i of `note`: the i-th partly masked
// tile.  Every weight is positive, so an infinity stays what it is.
template <typename T>
__device__ __noinline__ void window_add_back(const WindowFwdParams& p, int entry, int t, uint32_t note, uint32_t o_addr) {
  constexpr uint32_t kExp = Elem<T>::kBf16 ? 0x7f80u : 0x7c00u, kMan = Elem<T>::kBf16 ? 0x7fu : 0x3ffu;
  constexpr int kAhead = 8;
  const WindowItem it = window_item(p, entry);
  const WindowMasked masked(p.w, it);
  const WindowSee see(p.w, it, t);
  const UnitRange u = t == 0 ? it.u[0] : it.u[1];
  const int lane = static_cast<int>(threadIdx.x) & 31, D = p.w.dim;
  // bit l of [e]: column 4 l + e gets +infinity, -infinity, NaN
  uint32_t pos[4] = {}, neg[4] = {}, nan[4] = {}, nth = 0;
  for (int x = 0; x < it.n; ++x) {
    const int j = it.tile(x);
    if (!masked(j)) continue;
    if (((note >> nth++) & 1u) == 0 || !u.uses(j)) continue;
    const T* v = rows_at<T>(p.v, it.b, it.kh, j * kTile);
    const int rows = min(kTile, it.s.len - j * kTile);
    for (int r0 = 0; r0 < rows; r0 += kAhead) {
      uint2 y[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        y[i] = make_uint2(0u, 0u);
        if (r0 + i < rows && lane * 4 < D) y[i] = *reinterpret_cast<const uint2*>(v + (r0 + i) * p.v.s[2] + lane * 4);
      }
      const uint32_t sees = see.word(p.w, j, r0 >> 5);
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (!__any_sync(0xffffffffu, not_finite<T>(y[i].x, y[i].y, 0u, 0u))) continue;
        const uint32_t on = (sees >> ((r0 + i) & 31)) & 1u ? 0xffffffffu : 0u;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t h = ((e & 2) ? y[i].y : y[i].x) >> ((e & 1) * 16) & 0xffffu;
          const bool odd = (h & kExp) == kExp;
          pos[e] |= __ballot_sync(0xffffffffu, odd && (h & kMan) == 0 && h < 0x8000u) & on;
          neg[e] |= __ballot_sync(0xffffffffu, odd && (h & kMan) == 0 && h >= 0x8000u) & on;
          nan[e] |= __ballot_sync(0xffffffffu, odd && (h & kMan) != 0) & on;
        }
      }
    }
  }
  for (int c = 0; c < D; c += 16) {
    uint32_t y[16];
    ptx::tmem_ld_32x32b_x16(o_addr + c, y);
    ptx::tmem_wait_ld_dep16(y);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int l = (c + i) >> 2, e = i & 3;
      float f = __uint_as_float(y[i]);
      if ((pos[e] >> l) & 1u) f += INFINITY;
      if ((neg[e] >> l) & 1u) f -= INFINITY;
      if ((nan[e] >> l) & 1u) f = __uint_as_float(0x7fffffffu);
      y[i] = __float_as_uint(f);
    }
    ptx::tmem_st_32x32b_x16(o_addr + c, y);
  }
  ptx::tmem_wait_st();
}

// Warps 0 to 3: loads, matrix products, and in the second pass clean V tiles.
// One code for both passes: a second instance, though never run, made calls
// between other kernels 6 to 8 us slower.
template <typename T, int NKB>
__device__ __forceinline__ void window_feed(const WindowCtx& x, bool second, uint32_t bar0, const CUtensorMap& tm_q,
                                            const CUtensorMap& tm_k, const CUtensorMap& tm_v) {
  using P = WindowFwdPlan<NKB>;
  constexpr int S = P::kStages;
  const WindowFwdParams& p = x.p;
  const Pipe& pipe = x.pipe;
  const uint32_t base_s = x.base_s, tmem = x.tmem;
  const int warp = x.warp, lane = x.lane;
  auto bar = [bar0](uint32_t i) -> uint32_t { return bar0 + 8u * i; };
  const int from = second ? x.again(0) : 0, to = second ? x.again(1) : 0x7fffffff;
  if (warp == 0 && lane == 0) {
    // ---------------------------------------------------- K and V tiles
    const uint64_t keep = ptx::policy_evict_last();  // read again by other heads and rows
    long long c = 0;  // ring entries so far
    bool ok = true;
    // where entry st arrives: V in the second pass at warp 3's, which passes it on
    auto lands = [&](int st) { return bar(second && (st & 1) != 0 ? kWbVLanded + (st >> 1) : kWbKvFull + st); };
    for (int r = from, item; ok && r <= to && (item = window_entry(r)) < p.items; ++r) {
      const WindowItem it = window_item(p, item);
      for (int i = 0; ok && i < it.n; ++i) {
        const int row = it.tile(i) * kTile;
        for (int kv = 0; kv < 2; ++kv, ++c) {
          const int st = static_cast<int>(c % S);
          if (!(ok = pipe.wait(bar(kWbKvEmpty + st), static_cast<uint32_t>((c / S) & 1) ^ 1u, kSiteWinKv))) break;
          ptx::mbar_arrive_expect_tx(lands(st), P::kTileBytes);
          const MapMul m = kv ? p.mv : p.mk;
          for (int kb = 0; kb < NKB; ++kb)
            ptx::tma_load_4d_hint(base_s + P::kOffKv + st * P::kTileBytes + kb * kBlockBytes,
                                  kv ? &tm_v : &tm_k, lands(st), kb * 64, row,
                                  it.kh * m.h, it.b * m.b, keep);
        }
      }
    }
    for (long long d = c > S ? c - S : 0; d < c; ++d)
      pipe.drain(lands(static_cast<int>(d % S)), static_cast<uint32_t>((d / S) & 1), kSiteWinDrain);
  } else if (warp == 2 && lane == 0) {
    // ------------------------------------------------------- Q tiles
    const uint64_t once = ptx::policy_evict_first();
    uint32_t n_q = 0;
    for (int r = from, item; r <= to && (item = window_entry(r)) < p.items; ++r) {
      const WindowItem it = window_item(p, item);
      if (it.n == 0) continue;
      if (n_q > 0 && !pipe.wait(bar(kWbQEmpty), (n_q - 1) & 1u, kSiteWinQ)) break;
      ptx::mbar_arrive_expect_tx(bar(kWbQFull), (it.on[0] && it.on[1] ? 2 : 1) * P::kTileBytes);
#pragma unroll
      for (int t = 0; t < 2; ++t)
        for (int kb = 0; it.on[t] && kb < NKB; ++kb)
          ptx::tma_load_4d_hint(base_s + P::kOffQ + t * P::kTileBytes + kb * kBlockBytes, &tm_q,
                                bar(kWbQFull), kb * 64, it.row0[t], it.head[t] * p.mq.h,
                                it.b * p.mq.b, once);
      ++n_q;
    }
    if (n_q > 0) pipe.drain(bar(kWbQFull), (n_q - 1) & 1u, kSiteWinDrain);
  } else if (warp == 1) {
    // ------------------------------------------------------ MMA issue
    // The whole warp walks and waits; one elected lane issues.
    const int ksteps = (p.w.dim + 15) >> 4;
    const uint32_t idesc_s = ptx::idesc_16bit_f32(kTile, kTile, false, Elem<T>::kBf16);
    const uint32_t idesc_o = ptx::idesc_16bit_f32(kTile, static_cast<uint32_t>(ksteps) * 16u, true, Elem<T>::kBf16);
    constexpr uint32_t hi = ptx::smem_desc_hi(1024, ptx::kSwizzle128B);
    const uint32_t q_lo = ptx::smem_desc_lo(base_s + P::kOffQ, 16);
    const uint32_t k_lo = ptx::smem_desc_lo(base_s + P::kOffKv, 16);
    const uint32_t v_lo = ptx::smem_desc_lo(base_s + P::kOffKv, kBlockBytes);
    auto wait_kv = [&](uint32_t c) -> bool {
      return pipe.wait_warp(bar(kWbKvFull + c % S), (c / S) & 1u, kSiteWinMma);
    };
    auto commit = [&](uint32_t b) {
      if (ptx::elect_one()) ptx::mma_commit(bar(b));
    };
    uint32_t n_q = 0, n_s[2] = {0, 0}, n_p[2] = {0, 0};
    // S_t of ring entry c; with P of its own, once the softmax has read the last S_t
    auto issue_s = [&](int t, uint32_t c) -> bool {
      if (P::kOwnP && n_s[t] > 0) {
        if (!pipe.wait_warp(bar(kWbSFree + t), (n_s[t] - 1) & 1u, kSiteWinMma)) return false;
        ptx::tc_fence_after();
      }
      ++n_s[t];
      const uint32_t q = q_lo + t * (P::kTileBytes >> 4);
      const uint32_t k = k_lo + c % S * (P::kTileBytes >> 4);
      if (ptx::elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4 * NKB; ++ks) {
          constexpr int kStep = 32 >> 4, kBlock = kBlockBytes >> 4;
          const uint32_t off = (ks >> 2) * kBlock + (ks & 3) * kStep;
          if (ks < ksteps)
            ptx::mma_ss(tmem + t * 128u, ptx::smem_desc_join(q + off, hi), ptx::smem_desc_join(k + off, hi),
                        idesc_s, ks > 0);
        }
        ptx::mma_commit(bar(kWbSFull + t));
      }
      return true;
    };
    // O_t += P_t V of ring entry c, once P_t is written
    auto issue_o = [&](int t, uint32_t c, bool first) -> bool {
      if (!pipe.wait_warp(bar(kWbPFull + t), n_p[t] & 1u, kSiteWinMma)) return false;
      ++n_p[t];
      ptx::tc_fence_after();
      const uint32_t v = v_lo + c % S * (P::kTileBytes >> 4);
      if (ptx::elect_one()) {
#pragma unroll
        for (int ks = 0; ks < kTile / 16; ++ks)
          ptx::mma_ts(tmem + P::kColO + t * P::kStrideO, tmem + P::kColP + t * P::kStrideP + ks * 8u,
                      ptx::smem_desc_join(v + ks * (2048u >> 4), hi), idesc_o, !first || ks > 0);
        ptx::mma_commit(bar(kWbPvDone + t));
      }
      return true;
    };
    uint32_t g = 0;  // key tiles of this block so far (modulo 2^32); K of tile g is ring entry 2 g, V 2 g + 1
    bool ok = true;
    for (int r = from, item; ok && r <= to && (item = window_entry(r)) < p.items; ++r) {
      const WindowItem it = window_item(p, item);
      if (it.n == 0) continue;
      if (!(ok = pipe.wait_warp(bar(kWbQFull), n_q & 1u, kSiteWinMma))) break;
      ++n_q;
      if (!(ok = wait_kv(2 * g))) break;
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (ok && it.u[t].uses(it.tile(0))) ok = issue_s(t, 2 * g);
      commit(kWbKvEmpty + (2 * g) % S);
      if (it.n == 1) commit(kWbQEmpty);
      bool begun[2] = {false, false};
      for (int i = 0; ok && i < it.n; ++i, ++g) {
        const int j = it.tile(i), jn = i + 1 < it.n ? it.tile(i + 1) : -1;
        if (P::kOwnP && jn >= 0) {
          if (!(ok = wait_kv(2 * g + 2))) break;
#pragma unroll
          for (int t = 0; t < 2; ++t)
            if (ok && it.u[t].uses(jn)) ok = issue_s(t, 2 * g + 2);
          if (!ok) break;
          commit(kWbKvEmpty + (2 * g + 2) % S);
          if (i + 2 == it.n) commit(kWbQEmpty);
        }
        if (!(ok = wait_kv(2 * g + 1))) break;
        const int left = it.s.len - j * kTile;  // V rows of the sequence in this tile
        if (left < kTile && it.s.len < p.w.n_keys) {
          const uint32_t v = base_s + P::kOffKv + (2 * g + 1) % S * P::kTileBytes;
          for (int kb = 0; kb < NKB; ++kb)
            for (int y = left * 8 + lane; y < kTile * 8; y += 32)
              ptx::st_shared_v4(v + kb * kBlockBytes + y * 16, 0.0f, 0.0f, 0.0f, 0.0f);
          ptx::fence_proxy_async_smem();
          __syncwarp();
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (ok && it.u[t].uses(j)) {
            ok = issue_o(t, 2 * g + 1, !begun[t]);
            begun[t] = true;
          }
          if (!P::kOwnP && ok && jn >= 0) {
            if (t == 0) ok = wait_kv(2 * g + 2);
            if (ok && it.u[t].uses(jn)) ok = issue_s(t, 2 * g + 2);
          }
        }
        if (!ok) break;
        commit(kWbKvEmpty + (2 * g + 1) % S);
        if (!P::kOwnP && jn >= 0) commit(kWbKvEmpty + (2 * g + 2) % S);
        if (!P::kOwnP && i + 2 == it.n) commit(kWbQEmpty);
      }
    }
    commit(kWbMmaDone);
  } else if (second && warp == 3) {
    // ------------------------ V tiles passed on, partly masked ones cleaned
    uint32_t g = 0, n_items = 0;  // tiles, items with tiles so far
    bool ok = true;
    for (int r = from, item; ok && r <= to && (item = window_entry(r)) < p.items; ++r) {
      const WindowItem it = window_item(p, item);
      if (it.n == 0) continue;
      const WindowMasked masked(p.w, it);
      const uint32_t slot = n_items & 1u;
      if (!(ok = pipe.wait_warp(bar(kWbNotesFree + slot), ((n_items >> 1) & 1u) ^ 1u, kSiteWinClean))) break;
      ++n_items;
      uint32_t note = 0, nth = 0;
      for (int i = 0; i < it.n; ++i, ++g) {
        const uint32_t vs = g % P::kVStages, st = 2 * vs + 1;
        if (!(ok = pipe.wait_warp(bar(kWbVLanded + vs), (g / P::kVStages) & 1u, kSiteWinClean))) break;
        const int j = it.tile(i);
        if (masked(j)) {
          if (window_clean_v<T, NKB>(base_s + P::kOffKv + st * P::kTileBytes, it.s.len - j * kTile)) note |= 1u << nth;
          ++nth;
        }
        pipe_warp_arrive(bar(kWbKvFull + st));
      }
      if (lane == 0) ptx::st_shared_volatile(x.note_at(slot), note);
      pipe_warp_arrive(bar(kWbNotes + slot));
    }
  }
}

// Warps 4 to 11: softmax and results.
template <typename T, int NKB, bool kSecond>
__device__ __forceinline__ void window_soft(const WindowCtx& x, uint32_t bar0, const CUtensorMap& tm_o) {
  using P = WindowFwdPlan<NKB>;
  const WindowFwdParams& p = x.p;
  const Pipe& pipe = x.pipe;
  const uint32_t base_s = x.base_s, tmem = x.tmem;
  const int warp = x.warp, lane = x.lane;
  auto bar = [bar0](uint32_t i) -> uint32_t { return bar0 + 8u * i; };
  const int t = (warp - 4) >> 2;
  const int r = (warp & 3) * 32 + lane;  // row of the unit
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t s_addr = tmem + lanes + t * 128u;
  const uint32_t p_addr = tmem + lanes + P::kColP + t * P::kStrideP;
  const uint32_t o_addr = tmem + lanes + P::kColO + t * P::kStrideO;
  const uint32_t stage_out = base_s + P::kOffOut + static_cast<uint32_t>(warp - 4) * 4096u;
  const uint64_t once = ptx::policy_evict_first();
  const int D = p.w.dim, W = p.w.window;
  uint32_t n_s = 0;  // tiles of this unit so far
  int n_out = 0;     // result boxes of this warp so far
  bool ok = true;
  uint32_t n_items = 0;  // second pass: items with tiles so far
  for (int round = kSecond ? x.again(0) : 0, item; ok && (!kSecond || round <= x.again(1)) && (item = window_entry(round)) < p.items; ++round) {
    const WindowItem it = window_item(p, item);
    if (!(t == 0 ? it.on[0] : it.on[1])) {
      if (kSecond && it.n > 0) pipe_warp_arrive(bar(kWbNotesFree + (n_items++ & 1u)));
      continue;
    }
    const UnitRange u = t == 0 ? it.u[0] : it.u[1];
    const int row0 = t == 0 ? it.row0[0] : it.row0[1], head = t == 0 ? it.head[0] : it.head[1];
    const int p0 = it.s.start + row0, pos = p0 + r;
    const bool row_on = pos >= 0 && pos < it.s.len;
    float m = -INFINITY, l = 0.0f;  // m: running maximum in log2 units, may lag by < 8
    bool begun = false;
    for (int i = 0; i < it.n; ++i) {
      const int j = it.tile(i);
      if (!u.uses(j)) continue;
      if (!(ok = pipe.wait_warp(bar(kWbSFull + t), n_s & 1u, kSiteWinSoft))) break;
      ptx::tc_fence_after();
      uint32_t s[4][32];
#pragma unroll
      for (int c = 0; c < 4; ++c) ptx::tmem_ld_32x32b_x32(s_addr + c * 32, s[c]);
#pragma unroll
      for (int c = 0; c < 4; ++c) ptx::tmem_wait_ld_dep(s[c]);
      if (P::kOwnP) {
        ptx::tc_fence_before();
        pipe_warp_arrive(bar(kWbSFree + t));
      }
      const int k0 = j * kTile;
      // every row of the unit sees every key of the tile?
      const bool full = p0 >= k0 + kTile - 1 && p0 + kTile <= it.s.len &&
                        (p0 + kTile - 1 - W < k0 || k0 + kTile <= p.w.sinks);
      if (!full) {
        const int c_hi = row_on ? pos - k0 : -1, c_lo = pos - W - k0, c_sink = p.w.sinks - 1 - k0;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t see = bits_upto(c_hi, c) & (~bits_upto(c_lo, c) | bits_upto(c_sink, c));
          if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((see >> e) & 1u)) s[c][e] = 0xff800000u;
        }
      }
      float mc[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        float a = -INFINITY;
#pragma unroll
        for (int e = 0; e < 32; e += 2)
          a = ptx::max3(a, __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
        mc[c] = a;
      }
      const float mt = ptx::max3(mc[0], mc[1], fmaxf(mc[2], mc[3])) * p.scale_log2;
      const bool grew = mt > m + kLazyLog2;
      const float alpha = grew ? ptx::ex2_approx(m - mt) : 1.0f;  // 0 for the row's first keys
      if (grew) m = mt;
      const float ref = m == -INFINITY ? 0.0f : kWeightLog2<T> - m;  // a row that saw nothing yet: all weights 0
      const float2 scale = make_float2(p.scale_log2, p.scale_log2), shift = make_float2(ref, ref);
      float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const float2 y = __ffma2_rn(
              make_float2(__uint_as_float(s[c][2 * e]), __uint_as_float(s[c][2 * e + 1])), scale, shift);
          const float2 w = make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y));
          acc[e & 3] = __fadd2_rn(acc[e & 3], w);
          s[c][e] = pack2<T>(w.x, w.y);
        }
      const float2 s01 = __fadd2_rn(acc[0], acc[1]), s23 = __fadd2_rn(acc[2], acc[3]);
      l = fmaf(l, alpha, (s01.x + s01.y) + (s23.x + s23.y));
      // P free and O stable: with P over S, S of this tile follows the unit's
      // previous P V in issue order; else that product has to be awaited
      if (P::kOwnP && begun) {
        if (!(ok = pipe.wait_warp(bar(kWbPvDone + t), (n_s - 1) & 1u, kSiteWinSoft))) break;
        ptx::tc_fence_after();
      }
      if (begun && __any_sync(0xffffffffu, grew)) {
        for (int c = 0; c < D; c += 16) {
          uint32_t y[16];
          ptx::tmem_ld_32x32b_x16(o_addr + c, y);
          ptx::tmem_wait_ld_dep16(y);
#pragma unroll
          for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * alpha);
          ptx::tmem_st_32x32b_x16(o_addr + c, y);
        }
      }
      begun = true;
      ++n_s;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        ptx::tmem_st_32x32b_x16(p_addr + c * 16, *reinterpret_cast<uint32_t(*)[16]>(s[c]));
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      pipe_warp_arrive(bar(kWbPFull + t));
    }
    if (!ok) break;
    // ------------------------------------------------- out = O / l, lse
    // 32 columns at a time: TMEM, registers, a swizzled buffer, one TMA
    // store of the warp's rows (rows >= n_queries and columns >= head_dim
    // are not written), which completes behind the next item's work
    if (!u.empty()) {
      if (!(ok = pipe.wait_warp(bar(kWbPvDone + t), (n_s - 1) & 1u, kSiteWinOut))) break;
      ptx::tc_fence_after();
    }
    if (kSecond && it.n > 0) {
      const uint32_t slot = n_items & 1u;
      if (!(ok = pipe.wait_warp(bar(kWbNotes + slot), (n_items >> 1) & 1u, kSiteWinOut))) break;
      ++n_items;
      const uint32_t note = ptx::ld_shared_volatile(x.note_at(slot));
      pipe_warp_arrive(bar(kWbNotesFree + slot));
      if (note != 0 && !u.empty()) window_add_back<T>(p, item, t, note, o_addr);
    }
    const float inv = 1.0f / l;
    float check = 0.0f;  // NaN once an element is not finite
    for (int c = 0; c < D; c += 32) {
      uint32_t y[32];
      if (!u.empty()) {
        ptx::tmem_ld_32x32b_x32(o_addr + c, y);
        ptx::tmem_wait_ld_dep(y);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float a = l == 0.0f ? 0.0f : __uint_as_float(y[2 * e]) * inv;
        const float b = l == 0.0f ? 0.0f : __uint_as_float(y[2 * e + 1]) * inv;
        if (c + 2 * e < D) check = fmaf(a, 0.0f, fmaf(b, 0.0f, check));
        y[e] = pack2<T>(a, b);
      }
      const uint32_t buf = stage_out + static_cast<uint32_t>(n_out & 1) * 2048u;
      if (lane == 0) ptx::bulk_wait_group_read<1>();  // the box before the last has left this buffer
      __syncwarp();
#pragma unroll
      for (int k = 0; k < 4; ++k)
        ptx::st_shared_v4(buf + static_cast<uint32_t>(lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)),
                          __uint_as_float(y[4 * k]), __uint_as_float(y[4 * k + 1]),
                          __uint_as_float(y[4 * k + 2]), __uint_as_float(y[4 * k + 3]));
      ptx::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        ptx::tma_store_4d_hint(&tm_o, buf, c, row0 + (warp & 3) * 32, head * p.mo.h, it.b * p.mo.b, once);
        ptx::bulk_commit_group();
      }
      ++n_out;
    }
    ptx::tc_fence_before();
    const int row = row0 + r;
    // finite weights, but not the result: was it a hidden element of V?
    if (!kSecond && __any_sync(0xffffffffu, row < p.w.n_queries && row_on && check != 0.0f && l - l == 0.0f) &&
        window_leak<T>(p, item, t) && lane == 0) {
      asm volatile("red.shared.min.s32 [%0], %1;" ::"r"(pipe.at + kPipeBytes), "r"(round) : "memory");
      asm volatile("red.shared.max.s32 [%0], %1;" ::"r"(pipe.at + kPipeBytes + 4), "r"(round) : "memory");
    }
    if (row < p.w.n_queries && p.lse != nullptr)
      p.lse[(static_cast<long long>(it.b) * p.w.heads + head) * p.w.n_queries + row] =
          l == 0.0f ? -INFINITY : (m + (log2f(l) - kWeightLog2<T>)) * kLn2;
  }
  // before the rows are written again, or the block's shared memory goes
  if (lane == 0) ptx::bulk_wait_group_all();
}

template <typename T, int NKB>
__global__ void __launch_bounds__(WindowFwdPlan<NKB>::kThreads, 1)
    vattn_window_fwd_kernel(const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ CUtensorMap tm_o,
                            const __grid_constant__ WindowFwdParams p) {
  using P = WindowFwdPlan<NKB>;
  constexpr int S = P::kStages;
  static_assert(8 * (kWbCount + kWbSecondCount) + 8 + kPipeBytes + 16 <= 640 && P::kVStages <= 4, "barriers");
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = ptx::smem_addr(smem_raw);
  const uint32_t base_s = (raw_s + 1023u) & ~1023u;
  uint8_t* const base = smem_raw + (base_s - raw_s);
  const uint32_t bar0 = base_s + P::kOffBar;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(base + P::kOffBar + 8 * (kWbCount + kWbSecondCount));
  const Pipe pipe{base_s + P::kOffBar + 8 * (kWbCount + kWbSecondCount) + 8};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (uint32_t pass = 0; pass < 2; ++pass) {
      auto init = [&](uint32_t i, uint32_t count) { ptx::mbar_init(bar0 + 8u * (pass * kWbCount + i), count); };
      init(kWbQFull, 1);
      init(kWbQEmpty, 1);
      for (int i = 0; i < S; ++i) {
        init(kWbKvFull + i, 1);
        init(kWbKvEmpty + i, 1);
      }
      for (int t = 0; t < 2; ++t) {
        init(kWbSFull + t, 1);
        init(kWbPFull + t, 4);
        init(kWbPvDone + t, 1);
        init(kWbSFree + t, 4);
      }
      init(kWbMmaDone, 1);
    }
    for (uint32_t i = kWbVLanded; i < kWbSecondCount; ++i)
      ptx::mbar_init(bar0 + 8u * (kWbCount + i), i >= kWbNotesFree ? 8 : 1);
    pipe.init(p.w, p.status);
    ptx::st_shared_volatile(pipe.at + kPipeBytes, 0x7fffffffu);  // rounds of the second pass: none
    ptx::st_shared_volatile(pipe.at + kPipeBytes + 4, 0xffffffffu);
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_q);
    ptx::prefetch_tensormap(&tm_k);
    ptx::prefetch_tensormap(&tm_v);
    ptx::prefetch_tensormap(&tm_o);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(const_cast<uint32_t*>(tmem_slot)), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const WindowCtx x{p, pipe, base_s, *tmem_slot, warp, lane};
  ptx::grid_dep_wait();  // what earlier kernels of the stream wrote is visible

  bool two = false;
  if (warp < 4) {
    ptx::regs_decrease<P::kRegsOther>();
    for (int pass = 0; pass == 0 || (pass == 1 && (two = x.second())); ++pass)
      window_feed<T, NKB>(x, pass != 0, bar0 + (pass != 0 ? 8u * kWbCount : 0u), tm_q, tm_k, tm_v);
  } else {
    ptx::regs_increase<P::kRegsSoftmax>();
    window_soft<T, NKB, false>(x, bar0, tm_o);
    if (x.second()) window_soft<T, NKB, true>(x, bar0 + 8u * kWbCount, tm_o);
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) {
      x.pipe.drain(bar0 + 8u * kWbMmaDone, 0, kSiteWinDrain);
      if (two) x.pipe.drain(bar0 + 8u * (kWbCount + kWbMmaDone), 0, kSiteWinDrain);
    }
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(x.tmem, 512);
  }
}

}  // namespace vattn
