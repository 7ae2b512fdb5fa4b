// window_bwd_kernel.cuh -- gradients of the windowed attention
// (vattn_backward_window) on the tensor cores.
//
// With s_ij = scale q_i . k_j, p_ij = exp(s_ij - lse_i) on the visible pairs
// (0 elsewhere) and delta_i = dout_i . out_i:
//   dp_ij = dout_i . v_j,   ds_ij = p_ij (dp_ij - delta_i),
//   dv_j = sum_i p_ij dout_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j.
// The sums of dk and dv run over queries (of all heads of the group), that of
// dq over keys.  Two walks recompute s and dp rather than share them: seven
// products instead of five, but no atomics, so the order of every sum is
// fixed and the same call gives the same bits.
//
// Both walks are one kernel body: a block keeps a 128-row tile X (keys: K
// and V; queries: Q and dout) and streams 128-row tiles Y of the other side
// that its rows see:
//   S = X1 Y1^T, G = X2 Y2^T           (128 x 128 each, f32 in TMEM)
//   P = 2^(S scale log2e - lse2), D = P (G - delta), rounded to the type
//   keys:     dV += P Y2, dK += D Y1     queries:  dQ += D Y1
// P and D overwrite S in TMEM and are the A operands of the second products;
// Y is read K-major for the first and MN-major for the second, so nothing is
// transposed.  The grid is one block per multiprocessor.  Each takes X tiles
// from a counter, key tiles (longer) first (with tiles dealt out in turn, the
// blocks that got one more key tile ended last: 30 us of 190):
//   warp 0   X and Y tiles by TMA; Y through a ring of half tiles (64 rows),
//            ahead across X tiles
//   warp 1   issues G, then S of each tile (128 columns a product: a 128 x 64
//            one takes 50 cycles, a 128 x 128 one 65)
//   warp 2   issues the second products once P and D are there; an issuing
//            thread is held while its products run, so with two of them the
//            next tile's G and S run between
//   warp 3   takes the next X tile and tells the others, and the power of its D
//   warps 4-7, 8-11   P and D of columns 0..63, 64..127 of every tile, then
//            the X tile's results
// G is overwritten as soon as it is in registers, S once its P and D have
// been used.  TMEM columns (512), A: S, then P and D; B: G:
//   head_dim <= 64         A 0 and 128 in turn, B 256, dV 384, dK / dQ 448
//   above, X of keys       A 0, B 128, dV 256, dK 384
//   above, X of queries    A 0 and 256 in turn, B 128, dQ 384
//
// A key tile's walk is cut into chunks (f32 partial sums in a workspace,
// added in order by vattn_window_join_kernel) where tiles are few or, for the
// tiles of the first keys, the walk is long.
//
// Rounding: P and D go to the tensors' type for the second products, as these
// need (relative 2^-9 / 2^-12 at most of each term), and delta comes from `out` as
// rounded; all sums, lse and delta are f32.  For long rows that stays below the
// rounding of the results; for rows of a few keys dq and dk are off by up to twice
// as much as their own rounding.
//
// f16 keeps that relative error down to 2^-14 only, which a weight p of a long row
// and a D of an ordinary gradient (dout of 1e-3 over 4096 keys) are below, and ends
// at 65504.  So P is held as 2^15 p <= 2^15, and D as 2^e D with the power e of the
// walk that takes the largest value it can have, |dout_i| |v_j| + |delta_i| over
// the rows and keys of the walk, to 2^14 .. 2^15: no D overflows, and terms keep
// their digits down to 2^-29 of the largest.  The results are divided by 2^15 and
// 2^e in f32.  The statistics kernel leaves the largest |dout|^2, |delta| and |v|^2 of
// every 64 rows, and warp 3 looks up those of an X tile's walk while the tile
// before is worked on.  (2 x 16(4) x 4096 x 64, window 1024: 153 us, bf16, which
// needs none of it, 140.)
//
// What bounds it: for a tile of 128 x 128 pairs the products take 2080 cycles at
// head_dim 128 (keys; queries 1560) and half of that at 64, the arithmetic on
// the pairs about 1100 a warpgroup, and S, G, P, D and the sums follow each
// other through TMEM, where head_dim 128 leaves one pair of S and G.  2 x 16(4) x
// 4096 x 64, window 1024, 4 first keys: 140 us, 537 TFLOP/s counted as 10 D flops
// a visible pair, 751 with the products that are computed twice.
#pragma once

#include "window_pipe.cuh"

namespace vattn {

constexpr int kGradCols = 64;                // columns of a math warpgroup, rows of half a Y tile
constexpr int kGradBlock = kGradCols * 128;  // 64 rows x 64 elements, 128-byte swizzle
constexpr int kGradStat = 2 * kGradCols;     // floats of half a tile's -lse2, -delta
constexpr int kGradPBits = 15;               // f16: P is held as 2^15 p

struct WindowGradParams {
  WindowParams w;
  RowsTensor q, k, v, out, dout, dq, dk, dv;
  const float* lse;
  float* stat;     // [batch * heads][stat_tiles][-lse2 x 64 | -delta x 64] (f16: -lse2 + 15)
  float2* peak;    // f16: [batch * heads][stat_tiles] largest |dout|^2 and |delta| of the 64 rows
  float* v_peak;   // f16: [batch * kv_heads][2 key_tiles] largest |v|^2 of the 64 rows
  float* part;     // [slot][dv, dk][128][dim] partial sums of the chunks
  uint32_t* next;  // X tiles taken from the counter so far; zeroed by the statistics kernel
  uint32_t* status;
  MapMul mq, mg, mk, mv;  // q, dout, k, v
  int stat_tiles;  // half tiles (64 rows) of the queries, an even number
  int key_tiles;   // ceil(n_keys / 128)
  int sink_tiles;  // of these, the first with keys < sinks, cut into sink_chunks
  int sink_chunks, chunks;
  int sink_blocks, key_blocks, blocks;  // X tiles: the first keys' (with their chunks), all keys', all
  FastDiv d_sink_chunks, d_chunks, d_seqs, d_kv_heads, d_bhs, d_heads, d_stat_tiles;
  float scale_log2;
};

// -lse2 = -lse log2(e) and -delta of every query row; rows that see nothing
// (and those that fill the last tile) get -infinity and 0, hence weights 0.
// A block has half a tile, 64 rows; LR lanes, 16 bytes each, hold one row, and
// the loads of a lane's LR / 4 rows are all in flight before the sums.  f16: the
// blocks behind those have 64 rows of V each, of which they leave the largest
// square.  A row that is not finite counts as 0 there.
template <typename T, int LR>
__global__ void __launch_bounds__(256) vattn_window_stat_kernel(const __grid_constant__ WindowGradParams p) {
  constexpr int R = kGradCols * LR / 256;
  ptx::grid_dep_launch();  // the gradient kernel sets itself up meanwhile, and waits for this one's end
  if (blockIdx.x == 0 && threadIdx.x == 0) *p.next = 0;
  constexpr bool kPowers = !Elem<T>::kBf16;
  __shared__ float2 peak_s[8];
  const int lane = threadIdx.x % LR, c = lane * 8;
  auto leave = [&](float2 top, float2* to_pair, float* to_one) {  // the block's largest
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      top.x = fmaxf(top.x, __shfl_xor_sync(0xffffffffu, top.x, o));
      top.y = fmaxf(top.y, __shfl_xor_sync(0xffffffffu, top.y, o));
    }
    if (threadIdx.x % 32 == 0) peak_s[threadIdx.x / 32] = top;
    __syncthreads();
    if (threadIdx.x != 0) return;
#pragma unroll
    for (int w = 1; w < 8; ++w) top = make_float2(fmaxf(top.x, peak_s[w].x), fmaxf(top.y, peak_s[w].y));
    if (to_pair != nullptr) *to_pair = top;
    else *to_one = top.x;
  };
  auto finite = [](float x) { return x - x == 0.0f ? x : 0.0f; };
  const long long stat_blocks = static_cast<long long>(p.w.batch) * p.w.heads * p.stat_tiles;
  if (blockIdx.x >= stat_blocks) {
    if (!kPowers) return;
    const long long at = blockIdx.x - stat_blocks;
    if (at >= static_cast<long long>(p.w.batch) * p.w.kv_heads * 2 * p.key_tiles) return;
    const int half = static_cast<int>(at % (2 * p.key_tiles));
    const uint32_t bk = static_cast<uint32_t>(at / (2 * p.key_tiles));
    uint32_t kh;
    const int b = static_cast<int>(p.d_kv_heads.div(bk, &kh));
    const Seq s = window_seq(p.w, b);
    Vec<T, 8> x[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int j = half * kGradCols + threadIdx.x / LR + k * (256 / LR);
      const bool on = j < s.len && c < p.w.dim;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k].e[e] = Elem<T>::narrow(0.0f);
      if (on) x[k] = *reinterpret_cast<const Vec<T, 8>*>(rows_at<T>(p.v, b, kh, j) + c);
    }
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < R; ++k) {
      float f[8], sum = 0.0f;
      x[k].widen(f);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(f[e], f[e], sum);
#pragma unroll
      for (int o = LR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      top = fmaxf(top, finite(sum));
    }
    leave(make_float2(top, 0.0f), nullptr, p.v_peak + at);
    return;
  }
  uint32_t tile, h;
  const uint32_t bh = p.d_stat_tiles.div(blockIdx.x, &tile);
  const int b = static_cast<int>(p.d_heads.div(bh, &h));
  const Seq s = window_seq(p.w, b);
  Vec<T, 8> x[R], y[R];
  bool on[R];
#pragma unroll
  for (int k = 0; k < R; ++k) {
    const int i = static_cast<int>(tile) * kGradCols + threadIdx.x / LR + k * (256 / LR);
    const int pos = s.start + i;
    on[k] = i < p.w.n_queries && pos >= 0 && pos < s.len;
    if (on[k] && c < p.w.dim) {
      x[k] = *reinterpret_cast<const Vec<T, 8>*>(rows_at<T>(p.dout, b, h, i) + c);
      y[k] = *reinterpret_cast<const Vec<T, 8>*>(rows_at<T>(p.out, b, h, i) + c);
    }
  }
  float2 top = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int k = 0; k < R; ++k) {
    float sum = 0.0f, square = 0.0f;
    if (on[k] && c < p.w.dim) {
      float fx[8], fy[8];
      x[k].widen(fx);
      y[k].widen(fy);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum = fmaf(fx[e], fy[e], sum);
        if (kPowers) square = fmaf(fx[e], fx[e], square);
      }
    }
#pragma unroll
    for (int o = LR / 2; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (kPowers) square += __shfl_xor_sync(0xffffffffu, square, o);
    }
    top = make_float2(fmaxf(top.x, finite(square)), fmaxf(top.y, finite(fabsf(sum))));
    if (lane != 0) continue;
    const int r = threadIdx.x / LR + k * (256 / LR), i = static_cast<int>(tile) * kGradCols + r;
    const float lse = on[k] ? p.lse[static_cast<long long>(bh) * p.w.n_queries + i] : -INFINITY;
    const bool empty = lse == -INFINITY;
    float* to = p.stat + static_cast<long long>(blockIdx.x) * kGradStat + r;
    to[0] = empty ? -INFINITY : fmaf(-lse, kLog2E, kPowers ? static_cast<float>(kGradPBits) : 0.0f);
    to[kGradCols] = empty ? 0.0f : -sum;
  }
  if (kPowers) leave(top, p.peak + blockIdx.x, nullptr);
}

template <int NKB>
struct GradPlan {
  static constexpr int kXBytes = NKB * kBlockBytes;
  static constexpr int kYBytes = NKB * kBlockBytes;       // a Y tile: per 64 columns, 128 rows of 128 bytes
  static constexpr int kSlotBytes = 2 * kYBytes + 1024;   // Y1, Y2, the queries' stats
  static constexpr int kSlots = NKB == 1 ? 4 : 2;
  static constexpr int kHalves = 2 * kSlots;              // ring entries: half h of slot e / 2
  static constexpr int kOffX = 0;
  static constexpr int kOffY = 2 * kXBytes;
  static constexpr int kOffBar = kOffY + kSlots * kSlotBytes;
  static constexpr int kSmemBytes = kOffBar + 512 + 1024;
  static constexpr int kThreads = 384;
  static constexpr uint32_t kRegsOther = 72, kRegsMath = 216;  // 72 + 2 x 216 = 3 x 168
  static constexpr uint32_t kColG = NKB == 1 ? 256 : 128;
  static constexpr uint32_t kColDv = NKB == 1 ? 384 : 256;
  static constexpr uint32_t kColD = NKB == 1 ? 448 : 384;     // dK or dQ
  // two A columns in turn, or one
  template <bool kKeys> static constexpr bool kTurns = NKB == 1 || !kKeys;
  template <bool kKeys> static __device__ __forceinline__ uint32_t col_a(uint32_t tile) {
    return kTurns<kKeys> && (tile & 1u) ? (NKB == 1 ? 128u : 256u) : 0u;
  }
  static_assert(kSmemBytes <= 232448, "shared memory");
};

enum GradBar : int {
  kGbXFull = 0, kGbXEmpty = 1, kGbYFull = 2, kGbYEmpty = 10, kGbSFull = 18, kGbGFree = 19, kGbPFull = 20,
  kGbPFree = 22, kGbSum = 24, kGbSumFree = 25, kGbNext = 27, kGbTaken = 29, kGbDone = 31, kGbPower = 32, kGbCount = 36,
};
// A wait names a phase by its parity, so whoever waits on a barrier has seen
// the phase before the one it waits for.  The score issuer does not look at
// every X tile's sums, hence two SumFree barriers in turn: when it waits for
// the last tile's, those of the tile two before are done (the last tile's first
// S needed the tile before to have used P and D, whose sums needed them).

// What a block walks over: Y tiles 0 .. n - 1 of its share.
template <bool kKeys>
struct GradWalk {
  int b, h;         // h: key head (keys) or query head (queries)
  int row0;         // first row of the X tile
  Seq s;
  int slot;   // of the partial sums, -1: none
  // (tiles of 128 rows) keys: item -> head g of the group and query tile; queries: key tiles [0, ns) and [first, ..)
  int first, per_head, begin, n, ns;

};

// Item x of a walk: its Y tile and query head of the group.
template <bool kKeys>
struct GradItem {
  int x, g, tile;
  __device__ __forceinline__ GradItem(const GradWalk<kKeys>& w, int x0) : x(x0), g(0), tile(0) {
    if (kKeys) {
      const int i = w.begin + x0;
      g = i / w.per_head;
      tile = w.first + (i - g * w.per_head);
    } else {
      tile = x0 < w.ns ? x0 : w.first + (x0 - w.ns);
    }
  }
  __device__ __forceinline__ void step(const GradWalk<kKeys>& w, int by) {
    x += by;
    if (kKeys) {
      tile += by;
      while (tile >= w.first + w.per_head) {
        tile -= w.per_head;
        ++g;
      }
    } else {
      tile = x < w.ns ? x : w.first + (x - w.ns);
    }
  }
};

template <bool kKeys>
__device__ __forceinline__ GradWalk<kKeys> grad_walk(const WindowGradParams& p, int block);

template <>
__device__ __forceinline__ GradWalk<true> grad_walk<true>(const WindowGradParams& p, int block) {
  GradWalk<true> k;
  const bool sink = block < p.sink_blocks;
  const int at = sink ? block : block - p.sink_blocks;
  const int chunks = sink ? p.sink_chunks : p.chunks;
  uint32_t chunk, bk, kh;
  const uint32_t t = (sink ? p.d_sink_chunks : p.d_chunks).div(static_cast<uint32_t>(at), &chunk);
  const int tile = static_cast<int>(p.d_seqs.div(t, &bk)) + (sink ? 0 : p.sink_tiles);
  k.b = static_cast<int>(p.d_kv_heads.div(bk, &kh));
  k.h = static_cast<int>(kh);
  k.row0 = tile * kTile;
  k.s = window_seq(p.w, k.b);
  // slots: those of the first keys' tiles, then the others' (where cut)
  k.slot = chunks == 1 ? -1 : (sink || p.sink_chunks == 1 ? at : p.sink_blocks + at);
  k.ns = 0;
  k.n = k.begin = k.first = 0;
  k.per_head = 1;
  const int hi_pos = k.row0 < p.w.sinks ? k.s.len - 1 : min(k.s.len - 1, k.row0 + kTile - 1 + p.w.window - 1);
  const int lo = max(0, k.row0 - k.s.start), hi = min(p.w.n_queries - 1, hi_pos - k.s.start);
  if (k.row0 < k.s.len && hi >= lo) {
    k.first = lo / kTile;
    k.per_head = hi / kTile - k.first + 1;
    const long long all = static_cast<long long>(k.per_head) * p.w.group;
    k.begin = static_cast<int>(all * chunk / chunks);
    k.n = static_cast<int>(all * (chunk + 1LL) / chunks) - k.begin;
  }
  return k;
}

template <>
__device__ __forceinline__ GradWalk<false> grad_walk<false>(const WindowGradParams& p, int block) {
  GradWalk<false> k;
  uint32_t bh, h;
  const int tile = static_cast<int>(p.d_bhs.div(static_cast<uint32_t>(block - p.key_blocks), &bh));
  k.row0 = (p.stat_tiles / 2 - 1 - tile) * kTile;  // late rows see most: first
  k.b = static_cast<int>(p.d_heads.div(bh, &h));
  k.h = static_cast<int>(h);
  k.s = window_seq(p.w, k.b);
  k.slot = -1;
  k.begin = 0;
  k.per_head = 1;
  k.n = k.ns = k.first = 0;
  const int lo = max(0, k.s.start + k.row0);
  const int hi = min(k.s.start + min(k.row0 + kTile, p.w.n_queries), k.s.len) - 1;
  if (hi >= lo) {
    k.first = max(0, lo - p.w.window + 1) / kTile;
    k.ns = min((min(p.w.sinks, k.s.len) + kTile - 1) / kTile, k.first);
    k.n = k.ns + hi / kTile - k.first + 1;
  }
  return k;
}

// f16: 2^(e - 15) of the walk's D (a whole warp): e takes the bound |dout| |v| +
// |delta| over the walk's rows and keys to 2^14 .. 2^15.
template <bool kKeys>
__device__ __forceinline__ float grad_power(const WindowGradParams& p, const GradWalk<kKeys>& wk, int lane) {
  float2 g = make_float2(0.0f, 0.0f);
  float v = 0.0f;
  auto rows = [&](long long bh, int half) {
    const float2 x = p.peak[bh * p.stat_tiles + half];
    g = make_float2(fmaxf(g.x, x.x), fmaxf(g.y, x.y));
  };
  auto keys = [&](long long bk, int half) { v = fmaxf(v, p.v_peak[bk * 2 * p.key_tiles + half]); };
  if constexpr (kKeys) {
    const long long bk = static_cast<long long>(wk.b) * p.w.kv_heads + wk.h;
    for (int i = lane; i < 2 * wk.n; i += 32) {
      const GradItem<true> it(wk, i >> 1);
      rows(bk * p.w.group + it.g, 2 * it.tile + (i & 1));
    }
    if (lane < 2) keys(bk, wk.row0 / kGradCols + lane);
  } else {
    const long long bh = static_cast<long long>(wk.b) * p.w.heads + wk.h;
    for (int i = lane; i < 2 * wk.n; i += 32)
      keys(static_cast<long long>(wk.b) * p.w.kv_heads + wk.h / p.w.group, 2 * GradItem<false>(wk, i >> 1).tile + (i & 1));
    if (lane < 2) rows(bh, wk.row0 / kGradCols + lane);
  }
  const float most = sqrtf(warp_max(g.x)) * sqrtf(warp_max(v)) + warp_max(g.y);
  int k = 0;
  if (most > 0.0f) (void)frexpf(most, &k);  // most < 2^k
  return __int_as_float((127 + min(max(-k, -60), 60)) << 23);
}

// The block's roles, one X tile at a time; `at` counts the Y tiles of the
// block so far, `tiles` its X tiles with items.
struct GradCtx {
  const WindowGradParams& p;
  Pipe pipe;
  uint32_t base_s, bar0, tmem;
  int warp, lane;
  __device__ __forceinline__ uint32_t bar(int i) const { return bar0 + 8u * static_cast<uint32_t>(i); }
};

template <int NKB, bool kKeys>
__device__ __forceinline__ bool grad_load(const GradCtx& x, const CUtensorMap* tm_x1, const CUtensorMap* tm_x2,
                                          const CUtensorMap* tm_y1, const CUtensorMap* tm_y2, const MapMul& mx1,
                                          const MapMul& mx2, const MapMul& my1, const MapMul& my2, int block,
                                          uint32_t& at, uint32_t& tiles) {
  using P = GradPlan<NKB>;
  const WindowGradParams& p = x.p;
  const GradWalk<kKeys> wk = grad_walk<kKeys>(p, block);
  if (wk.n == 0) return true;
  const uint64_t keep = ptx::policy_evict_last(), once = ptx::policy_evict_first();
  GradItem<kKeys> it(wk, 0);
  for (int n = 0; n < wk.n; ++n, it.step(wk, 1)) {
    const int h = kKeys ? wk.h * p.w.group + it.g : wk.h / p.w.group;
    for (int half = 0; half < 2; ++half, ++at) {  // at: halves here
      const uint32_t e = at % P::kHalves;
      if (!x.pipe.wait(x.bar(kGbYEmpty + e), ((at / P::kHalves) & 1u) ^ 1u, kSiteGradLoad)) return false;
      ptx::mbar_arrive_expect_tx(x.bar(kGbYFull + e), 2 * NKB * kGradBlock + (kKeys ? kGradStat * 4 : 0));
      const uint32_t slot = x.base_s + P::kOffY + (e >> 1) * P::kSlotBytes;
      const int row = it.tile * kTile + half * kGradCols;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int kb = 0; kb < NKB; ++kb) {
          const MapMul m = i ? my2 : my1;
          ptx::tma_load_4d_hint(slot + i * P::kYBytes + kb * kBlockBytes + half * kGradBlock, i ? tm_y2 : tm_y1,
                                x.bar(kGbYFull + e), kb * 64, row, h * m.h, wk.b * m.b, keep);
        }
      if (kKeys)
        ptx::bulk_load(slot + 2 * P::kYBytes + half * kGradStat * 4,
                       p.stat + ((static_cast<long long>(wk.b) * p.w.heads + h) * p.stat_tiles + 2 * it.tile + half) *
                                    kGradStat,
                       kGradStat * 4, x.bar(kGbYFull + e));
    }
    if (n > 0) continue;
    // X behind the first Y: it waits for the last X tile's S and G
    if (!x.pipe.wait(x.bar(kGbXEmpty), (tiles & 1u) ^ 1u, kSiteGradLoad)) return false;
    ptx::mbar_arrive_expect_tx(x.bar(kGbXFull), 2 * P::kXBytes);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int kb = 0; kb < NKB; ++kb) {
        const MapMul m = i ? mx2 : mx1;
        ptx::tma_load_4d_hint(x.base_s + P::kOffX + i * P::kXBytes + kb * kBlockBytes, i ? tm_x2 : tm_x1,
                              x.bar(kGbXFull), kb * 64, wk.row0, wk.h * m.h, wk.b * m.b, once);
      }
    ++tiles;
  }
  return true;
}

// G = X2 Y2^T and S = X1 Y1^T of every tile (a whole warp; one lane issues).
// `keys_before`: the last X tile with items was one of keys.
template <typename T, int NKB, bool kKeys>
__device__ __forceinline__ bool grad_scores(const GradCtx& x, int block, uint32_t& at, uint32_t& tiles,
                                            bool& keys_before) {
  using P = GradPlan<NKB>;
  const WindowGradParams& p = x.p;
  const GradWalk<kKeys> wk = grad_walk<kKeys>(p, block);
  if (wk.n == 0) return true;
  const int ksteps = (p.w.dim + 15) >> 4;
  constexpr uint32_t idesc = ptx::idesc_16bit_f32(kTile, kTile, false, Elem<T>::kBf16);
  constexpr uint32_t hi = ptx::smem_desc_hi(1024, ptx::kSwizzle128B);
  const uint32_t x_lo = ptx::smem_desc_lo(x.base_s + P::kOffX, 16);
  if (!x.pipe.wait_warp(x.bar(kGbXFull), tiles & 1u, kSiteGradMma)) return false;
  // from keys to queries the second A column takes dV's place: its last sums have been read
  if (NKB == 2 && !kKeys && keys_before &&
      !x.pipe.wait_warp(x.bar(kGbSumFree + ((tiles - 1) & 1u)), ((tiles - 1) >> 1) & 1u, kSiteGradMma))
    return false;
  keys_before = kKeys;
  ++tiles;
  GradItem<kKeys> it(wk, 0);
  for (int n = 0; n < wk.n; ++n, ++at, it.step(wk, 1)) {
    const uint32_t slot = at % P::kSlots, turn = (at / P::kSlots) & 1u;
    const uint32_t y = x.base_s + P::kOffY + slot * P::kSlotBytes;
    if (!x.pipe.wait_warp(x.bar(kGbYFull + 2 * slot), turn, kSiteGradMma) ||
        !x.pipe.wait_warp(x.bar(kGbYFull + 2 * slot + 1), turn, kSiteGradMma))
      return false;
    // Y rows outside the sequence may hold anything: zero, so that they add
    // nothing to the second products
    const int row0 = it.tile * kTile;
    const int first = kKeys ? -wk.s.start - row0 : 0;  // rows of the sequence: [first, last)
    const int last = (kKeys ? wk.s.len - wk.s.start : wk.s.len) - row0;
    if (first > 0 || last < kTile) {
      for (int kb = 0; kb < 2 * NKB; ++kb)
        for (int i = x.lane; i < kTile * 8; i += 32)
          if ((i >> 3) < first || (i >> 3) >= last)
            ptx::st_shared_v4(y + kb * kBlockBytes + i * 16, 0.0f, 0.0f, 0.0f, 0.0f);
      ptx::fence_proxy_async_smem();
      __syncwarp();
    }
    const uint32_t y_lo = ptx::smem_desc_lo(y, 16);
    // i = 1: G, once the last one is in registers; i = 0: S, once the P and D there have been used
#pragma unroll
    for (int i = 1; i >= 0; --i) {
      if (i == 1) {
        if (at > 0 && !x.pipe.wait_warp(x.bar(kGbGFree), (at - 1) & 1u, kSiteGradMma)) return false;
      } else {
        const uint32_t before = P::template kTurns<kKeys> ? 2u : 1u;  // tile `before` back used these columns
        if (at >= before && !x.pipe.wait_warp(x.bar(kGbPFree + ((at - before) & 1u)), ((at - before) >> 1) & 1u, kSiteGradMma))
          return false;
      }
      ptx::tc_fence_after();
      const uint32_t d = x.tmem + (i == 1 ? P::kColG : P::template col_a<kKeys>(at));
      if (ptx::elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4 * NKB; ++ks) {
          const uint32_t off = (i * P::kXBytes + (ks >> 2) * kBlockBytes + (ks & 3) * 32) >> 4;
          if (ks < ksteps)
            ptx::mma_ss(d, ptx::smem_desc_join(x_lo + off, hi), ptx::smem_desc_join(y_lo + off, hi), idesc, ks > 0);
        }
        if (i == 0) {
          ptx::mma_commit(x.bar(kGbSFull));
          // the issuer's own arrival: what it saw of Y (the stats that the math warps
          // read) and wrote there (zeros, which the second products read) goes with it
          ptx::mbar_arrive(x.bar(kGbSFull));
          if (n + 1 == wk.n) ptx::mma_commit(x.bar(kGbXEmpty));
        }
      }
    }
  }
  return true;
}

// keys: dV += P Y2, dK += D Y1;  queries: dQ += D Y1.
template <typename T, int NKB, bool kKeys>
__device__ __forceinline__ bool grad_sums(const GradCtx& x, int block, uint32_t& at, uint32_t& tiles) {
  using P = GradPlan<NKB>;
  const WindowGradParams& p = x.p;
  const GradWalk<kKeys> wk = grad_walk<kKeys>(p, block);
  if (wk.n == 0) return true;
  const uint32_t idesc =
      ptx::idesc_16bit_f32(kTile, static_cast<uint32_t>((p.w.dim + 15) >> 4) * 16u, true, Elem<T>::kBf16);
  constexpr uint32_t hi = ptx::smem_desc_hi(1024, ptx::kSwizzle128B);
  // the last X tile's sums have been read
  if (tiles > 0 && !x.pipe.wait_warp(x.bar(kGbSumFree + ((tiles - 1) & 1u)), ((tiles - 1) >> 1) & 1u, kSiteGradMma))
    return false;
  ++tiles;
  for (int n = 0; n < wk.n; ++n, ++at) {
    const uint32_t slot = at % P::kSlots, turn = (at / P::kSlots) & 1u;
    if (!x.pipe.wait_warp(x.bar(kGbYFull + 2 * slot), turn, kSiteGradMma) ||
        !x.pipe.wait_warp(x.bar(kGbYFull + 2 * slot + 1), turn, kSiteGradMma) ||
        !x.pipe.wait_warp(x.bar(kGbPFull + (at & 1u)), (at >> 1) & 1u, kSiteGradMma))
      return false;
    ptx::tc_fence_after();
    const uint32_t y1 = ptx::smem_desc_lo(x.base_s + P::kOffY + slot * P::kSlotBytes, kBlockBytes);
    const uint32_t y2 = y1 + (P::kYBytes >> 4);
    const uint32_t a = x.tmem + P::template col_a<kKeys>(at);
    if (ptx::elect_one()) {
#pragma unroll
      for (int ks = 0; ks < kTile / 16; ++ks) {
        const uint32_t a_ks = a + (ks >> 2) * 64u + (ks & 3) * 8u;  // P of columns 16 ks ..; D 32 further
        if (kKeys)
          ptx::mma_ts(x.tmem + P::kColDv, a_ks, ptx::smem_desc_join(y2 + ks * (2048u >> 4), hi), idesc,
                      n > 0 || ks > 0);
        ptx::mma_ts(x.tmem + P::kColD, a_ks + 32u, ptx::smem_desc_join(y1 + ks * (2048u >> 4), hi), idesc,
                    n > 0 || ks > 0);
        if (ks == 3) ptx::mma_commit(x.bar(kGbYEmpty + 2 * slot));
      }
      ptx::mma_commit(x.bar(kGbYEmpty + 2 * slot + 1));
      ptx::mma_commit(x.bar(kGbPFree + (at & 1u)));
      if (n + 1 == wk.n) ptx::mma_commit(x.bar(kGbSum));
    }
  }
  return true;
}

// P and D of 64 columns of every tile, then the X tile's results (one warpgroup).
template <typename T, int NKB, bool kKeys>
__device__ __forceinline__ bool grad_math(const GradCtx& x, int block, uint32_t& at, uint32_t& tiles, float power) {
  constexpr bool kPowers = !Elem<T>::kBf16;
  using P = GradPlan<NKB>;
  const WindowGradParams& p = x.p;
  const GradWalk<kKeys> wk = grad_walk<kKeys>(p, block);
  const int wg = (x.warp - 4) >> 2;
  const int r = (x.warp & 3) * 32 + x.lane;
  const uint32_t lanes = static_cast<uint32_t>((x.warp & 3) * 32) << 16;
  const int row = wk.row0 + r;  // key, or query row of the call
  const int W = p.w.window;
  float row_lse = -INFINITY, row_delta = 0.0f;
  if (!kKeys && wk.n > 0) {
    const float* st = p.stat + ((static_cast<long long>(wk.b) * p.w.heads + wk.h) * p.stat_tiles + row / kGradCols) *
                                   kGradStat + row % kGradCols;
    row_lse = st[0];
    row_delta = kPowers ? st[kGradCols] * power : st[kGradCols];
  }
  const float2 power2 = make_float2(power, power);
  const float2 scale = make_float2(p.scale_log2, p.scale_log2);
  if (wk.n > 0) {
    GradItem<kKeys> it(wk, 0);
    for (int n = 0; n < wk.n; ++n, ++at, it.step(wk, 1)) {
      const uint32_t s_addr = x.tmem + lanes + P::template col_a<kKeys>(at) + wg * 64u;
      const uint32_t g_addr = x.tmem + lanes + P::kColG + wg * 64u;
      const int y0 = it.tile * kTile + wg * kGradCols;
      if (!x.pipe.wait_warp(x.bar(kGbSFull), at & 1u, kSiteGradSoft)) return false;
      ptx::tc_fence_after();
      uint32_t s[2][32], g[2][32];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        ptx::tmem_ld_32x32b_x32(s_addr + c * 32, s[c]);
        ptx::tmem_ld_32x32b_x32(g_addr + c * 32, g[c]);
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        ptx::tmem_wait_ld_dep(s[c]);
        ptx::tmem_wait_ld_dep(g[c]);
      }
      ptx::tc_fence_before();
      pipe_warp_arrive(x.bar(kGbGFree));
      // columns [c_lo, c_hi] of the row are visible, and those <= c_sink
      int c_lo, c_hi, c_sink = -1;
      bool full;
      if (kKeys) {
        const int p0 = wk.s.start + y0;
        c_lo = row < wk.s.len ? row - p0 : kGradCols;
        c_hi = row < p.w.sinks ? kGradCols - 1 : row + W - 1 - p0;
        full = p0 >= wk.row0 + kTile - 1 && p0 + kGradCols <= wk.s.len &&
               (p0 + kGradCols - 1 < wk.row0 + W || wk.row0 + kTile <= p.w.sinks);
      } else {
        const int pos = wk.s.start + row, p0 = wk.s.start + wk.row0;
        c_hi = pos >= 0 && pos < wk.s.len ? pos - y0 : -1;
        c_lo = pos - W + 1 - y0;
        c_sink = min(p.w.sinks - 1 - y0, c_hi);
        full = p0 >= y0 + kGradCols - 1 && p0 + kTile <= wk.s.len &&
               (p0 + kTile - 1 - W < y0 || y0 + kGradCols <= p.w.sinks);
      }
      if (!full) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const uint32_t see = (bits_upto(c_hi, c) & ~bits_upto(c_lo - 1, c)) | bits_upto(c_sink, c);
          if (__all_sync(0xffffffffu, see == 0xffffffffu)) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!((see >> e) & 1u)) {
              s[c][e] = 0xff800000u;
              g[c][e] = 0u;
            }
        }
      }
      const uint32_t stats = x.base_s + P::kOffY + (at % P::kSlots) * P::kSlotBytes + 2 * P::kYBytes + wg * kGradStat * 4;
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float4 nl, nd;
          if (kKeys) {
            nl = ptx::ld_shared_v4(stats + (c * 32 + e * 4) * 4);
            nd = ptx::ld_shared_v4(stats + (kGradCols + c * 32 + e * 4) * 4);
          } else {
            nl = make_float4(row_lse, row_lse, row_lse, row_lse);
            nd = make_float4(row_delta, row_delta, row_delta, row_delta);
          }
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const int i = e * 4 + f * 2;
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1])), scale,
                                        f ? make_float2(nl.z, nl.w) : make_float2(nl.x, nl.y));
            const float2 w = make_float2(ptx::ex2_approx(y.x), ptx::ex2_approx(y.y));
            const float2 dp = make_float2(__uint_as_float(g[c][i]), __uint_as_float(g[c][i + 1]));
            const float2 delta = f ? make_float2(nd.z, nd.w) : make_float2(nd.x, nd.y);
            const float2 d = __fmul2_rn(w, !kPowers ? __fadd2_rn(dp, delta)
                                           : kKeys  ? __fmul2_rn(__fadd2_rn(dp, delta), power2)
                                                    : __ffma2_rn(dp, power2, delta));
            if (kKeys) s[c][i / 2] = pack2<T>(w.x, w.y);
            g[c][i / 2] = pack2<T>(d.x, d.y);
          }
        }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (kKeys) ptx::tmem_st_32x32b_x16(s_addr + c * 16, *reinterpret_cast<uint32_t(*)[16]>(s[c]));
        ptx::tmem_st_32x32b_x16(s_addr + 32 + c * 16, *reinterpret_cast<uint32_t(*)[16]>(g[c]));
      }
      ptx::tmem_wait_st();
      ptx::tc_fence_before();
      pipe_warp_arrive(x.bar(kGbPFull + (at & 1u)));
    }
  }
  // keys: warpgroup 0 stores dV (unscaled), 1 dK; queries: each every other 16 columns of dQ
  if (wk.n > 0) {
    if (!x.pipe.wait_warp(x.bar(kGbSum), tiles & 1u, kSiteGradOut)) return false;
    ++tiles;
    ptx::tc_fence_after();
  }
  const int D = p.w.dim;
  const uint32_t a_addr = x.tmem + lanes + (kKeys && wg == 0 ? P::kColDv : P::kColD);
  const bool live = wk.n > 0 && (kKeys ? row < wk.s.len : (wk.s.start + row >= 0 && wk.s.start + row < wk.s.len));
  constexpr float kBack = kPowers ? 0x1p-15f : 1.0f;
  static_assert(kGradPBits == 15, "kBack");
  const float f = kKeys && wg == 0 ? kBack : (kPowers ? p.w.scale * (kBack / power) : p.w.scale);
  const bool store = row < (kKeys ? p.w.n_keys : p.w.n_queries);
  T* to = nullptr;
  float* part = nullptr;
  if (wk.slot >= 0) part = p.part + ((wk.slot * 2LL + wg) * kTile + r) * D;
  else if (store) to = rows_at_mut<T>(kKeys ? (wg == 0 ? p.dv : p.dk) : p.dq, wk.b, wk.h, row);
  for (int c = kKeys ? 0 : wg * 16; c < D; c += kKeys ? 16 : 32) {
    uint32_t y[16];
    if (wk.n > 0) {
      ptx::tmem_ld_32x32b_x16(a_addr + c, y);
      ptx::tmem_wait_ld_dep16(y);
    }
#pragma unroll
    for (int e = 0; e < 16; ++e) y[e] = live ? __float_as_uint(__uint_as_float(y[e]) * f) : 0u;
    if (part != nullptr) {
#pragma unroll
      for (int e = 0; e < 16; e += 4)
        if (c + e < D) *reinterpret_cast<uint4*>(part + c + e) = make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
    } else if (to != nullptr) {
#pragma unroll
      for (int e = 0; e < 16; e += 8)
        if (c + e < D) {
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            h[k] = pack2<T>(__uint_as_float(y[e + 2 * k]), __uint_as_float(y[e + 2 * k + 1]));
          *reinterpret_cast<uint4*>(to + c + e) = make_uint4(h[0], h[1], h[2], h[3]);
        }
    }
  }
  if (wk.n > 0) {
    ptx::tc_fence_before();
    pipe_warp_arrive(x.bar(kGbSumFree + ((tiles - 1) & 1u)));
  }
  return true;
}

// X tiles: blockIdx.x, then from the counter: key tiles first, then the query
// tiles, which are shorter and even out what the key tiles leave.  tm_*:
// boxes of 128 rows (x) and of 64 (y).
template <typename T, int NKB>
__global__ void __launch_bounds__(GradPlan<NKB>::kThreads, 1)
    vattn_window_bwd_kernel(const __grid_constant__ CUtensorMap tm_qx, const __grid_constant__ CUtensorMap tm_gx,
                            const __grid_constant__ CUtensorMap tm_kx, const __grid_constant__ CUtensorMap tm_vx,
                            const __grid_constant__ CUtensorMap tm_qy, const __grid_constant__ CUtensorMap tm_gy,
                            const __grid_constant__ CUtensorMap tm_ky, const __grid_constant__ CUtensorMap tm_vy,
                            const __grid_constant__ WindowGradParams p) {
  using P = GradPlan<NKB>;
  constexpr bool kPowers = !Elem<T>::kBf16;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = ptx::smem_addr(smem_raw);
  const uint32_t base_s = (raw_s + 1023u) & ~1023u;
  uint8_t* const base = smem_raw + (base_s - raw_s);
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(base + P::kOffBar + 8 * kGbCount);
  const Pipe pipe{base_s + P::kOffBar + 8 * kGbCount + 8};
  volatile int* taken = reinterpret_cast<volatile int*>(tmem_slot + 2 + kPipeBytes / 4);  // [2] X tiles handed out
  volatile float* powers = reinterpret_cast<volatile float*>(taken + 2);                  // [4] and their grad_power
  const uint32_t bar0 = base_s + P::kOffBar;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    auto init = [bar0](int i, uint32_t count) { ptx::mbar_init(bar0 + 8u * static_cast<uint32_t>(i), count); };
    init(kGbXFull, 1);
    init(kGbXEmpty, 1);
    for (int i = 0; i < P::kHalves; ++i) {
      init(kGbYFull + i, 1);
      init(kGbYEmpty + i, 1);
    }
    init(kGbSFull, 2);  // the products, and their issuer
    init(kGbGFree, 8);
    for (int i = 0; i < 2; ++i) {
      init(kGbPFull + i, 8);
      init(kGbPFree + i, 1);
      init(kGbSumFree + i, 8);
      init(kGbNext + i, 1);
      init(kGbTaken + i, 11);  // loader, two issuers, eight math warps
    }
    for (int i = 0; i < 4; ++i) init(kGbPower + i, 1);
    init(kGbSum, 1);
    init(kGbDone, 2);
    pipe.init(p.w, p.status);
    ptx::fence_mbar_init();
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(const_cast<uint32_t*>(tmem_slot)), 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const GradCtx x{p, pipe, base_s, bar0, *tmem_slot, warp, lane};
  ptx::grid_dep_wait();
  uint32_t at = 0, tiles = 0;
  bool ok = true;
  // The block's next X tile (its first is blockIdx.x), -1 after the last: by
  // one thread, or by all lanes of a warp.
  uint32_t n_taken = 0;
  auto next = [&](bool whole_warp) -> int {
    const uint32_t i = n_taken & 1u, phase = (n_taken >> 1) & 1u;
    ++n_taken;
    if (whole_warp ? !x.pipe.wait_warp(x.bar(kGbNext + i), phase, kSiteGradNext)
                   : !x.pipe.wait(x.bar(kGbNext + i), phase, kSiteGradNext))
      return -1;
    const int block = taken[i];
    if (whole_warp) pipe_warp_arrive(x.bar(kGbTaken + i));
    else ptx::mbar_arrive(x.bar(kGbTaken + i));
    return block < p.blocks ? block : -1;
  };
  if (warp < 4) {
    ptx::regs_decrease<P::kRegsOther>();
    if (warp == 0 && lane == 0) {
      for (int block = next(false); ok && block >= 0; block = ok ? next(false) : -1) {
        if (block < p.key_blocks)
          ok = grad_load<NKB, true>(x, &tm_kx, &tm_vx, &tm_qy, &tm_gy, p.mk, p.mv, p.mq, p.mg, block, at, tiles);
        else
          ok = grad_load<NKB, false>(x, &tm_qx, &tm_gx, &tm_ky, &tm_vy, p.mq, p.mg, p.mk, p.mv, block, at, tiles);
      }
      // every copy has landed before the block exits
      if (tiles > 0) x.pipe.drain(x.bar(kGbXFull), (tiles - 1) & 1u, kSiteGradDrain);
      for (uint32_t d = at > P::kHalves ? at - P::kHalves : 0; d < at; ++d)
        x.pipe.drain(x.bar(kGbYFull + d % P::kHalves), (d / P::kHalves) & 1u, kSiteGradDrain);
    } else if (warp == 1) {
      bool keys_before = false;
      for (int block = next(true); ok && block >= 0; block = ok ? next(true) : -1)
        ok = block < p.key_blocks ? grad_scores<T, NKB, true>(x, block, at, tiles, keys_before)
                                  : grad_scores<T, NKB, false>(x, block, at, tiles, keys_before);
      if (ptx::elect_one()) ptx::mma_commit(x.bar(kGbDone));
    } else if (warp == 2) {
      for (int block = next(true); ok && block >= 0; block = ok ? next(true) : -1)
        ok = block < p.key_blocks ? grad_sums<T, NKB, true>(x, block, at, tiles)
                                  : grad_sums<T, NKB, false>(x, block, at, tiles);
      if (ptx::elect_one()) ptx::mma_commit(x.bar(kGbDone));
    } else if (warp == 3) {
      int block = static_cast<int>(blockIdx.x);
      for (uint32_t i = 0;; ++i) {
        if (!x.pipe.wait_warp(x.bar(kGbTaken + (i & 1u)), ((i >> 1) & 1u) ^ 1u, kSiteGradNext)) break;
        if (lane == 0) taken[i & 1u] = block;
        pipe_warp_arrive(x.bar(kGbNext + (i & 1u)));
        if (block >= p.blocks) break;
        if (kPowers) {
          const float power = block < p.key_blocks ? grad_power<true>(p, grad_walk<true>(p, block), lane)
                                                   : grad_power<false>(p, grad_walk<false>(p, block), lane);
          if (lane == 0) powers[i & 3u] = power;
          pipe_warp_arrive(x.bar(kGbPower + (i & 3u)));
        }
        int taken_now = 0;
        if (lane == 0) taken_now = static_cast<int>(gridDim.x + atomicAdd(p.next, 1u));
        block = __shfl_sync(0xffffffffu, taken_now, 0);
      }
    }
  } else {
    ptx::regs_increase<P::kRegsMath>();
    for (int block = next(true); ok && block >= 0; block = ok ? next(true) : -1) {
      float power = 1.0f;
      if (kPowers) {  // (of four in turn: that of the tile after next is not written over one being read)
        const uint32_t i = n_taken - 1;
        if (!x.pipe.wait_warp(x.bar(kGbPower + (i & 3u)), (i >> 2) & 1u, kSiteGradNext)) break;
        power = powers[i & 3u];
      }
      ok = block < p.key_blocks ? grad_math<T, NKB, true>(x, block, at, tiles, power)
                                : grad_math<T, NKB, false>(x, block, at, tiles, power);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    if (lane == 0) x.pipe.drain(x.bar(kGbDone), 0, kSiteGradDrain);
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(x.tmem, 512);
  }
}

// dk and dv of the key tiles that were cut: their chunks' partial sums added
// in order.  blockIdx.x = (tile, sequence and key head); a thread takes 8
// consecutive elements of one row.
template <typename T>
__global__ void __launch_bounds__(256) vattn_window_join_kernel(const __grid_constant__ WindowGradParams p) {
  const long long seqs = static_cast<long long>(p.w.batch) * p.w.kv_heads;
  const long long bk = blockIdx.x % seqs;
  const int tile = static_cast<int>(blockIdx.x / seqs) + (p.sink_chunks > 1 ? 0 : p.sink_tiles);
  const bool sink = tile < p.sink_tiles;
  const int chunks = sink ? p.sink_chunks : p.chunks;
  if (chunks == 1) return;
  const long long at = ((static_cast<long long>(tile) - (sink ? 0 : p.sink_tiles)) * seqs + bk) * chunks;
  const long long slot = sink || p.sink_chunks == 1 ? at : p.sink_blocks + at;
  const int b = static_cast<int>(bk / p.w.kv_heads), h = static_cast<int>(bk - static_cast<long long>(b) * p.w.kv_heads);
  const int D = p.w.dim, per_row = D / 8;
  const int e = blockIdx.y * 256 + threadIdx.x;
  if (e >= 2 * kTile * per_row) return;
  const int which = e / (kTile * per_row), r = e / per_row % kTile, d = e % per_row * 8;
  const int row = tile * kTile + r;
  if (row >= p.w.n_keys) return;
  ptx::grid_dep_wait();
  const float* from = p.part + ((slot * 2 + which) * kTile + r) * static_cast<long long>(D) + d;
  float x[8] = {};
  for (int c = 0; c < chunks; ++c, from += 2 * kTile * static_cast<long long>(D)) {
    const float4 lo = *reinterpret_cast<const float4*>(from), hi = *reinterpret_cast<const float4*>(from + 4);
    x[0] += lo.x; x[1] += lo.y; x[2] += lo.z; x[3] += lo.w;
    x[4] += hi.x; x[5] += hi.y; x[6] += hi.z; x[7] += hi.w;
  }
  reinterpret_cast<Vec<T, 8>*>(rows_at_mut<T>(which ? p.dk : p.dv, b, h, row) + d)->narrow(x);
}

}  // namespace vattn
