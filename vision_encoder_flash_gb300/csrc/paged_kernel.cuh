// paged_kernel.cuh -- attention of a few new tokens over the 8-bit paged cache
// (vattn_forward_paged).
//
// Memory bound: every visible key and value, one byte an element, is read once for
// all rows (new token, query head of the group) of its key head together.  A
// block takes up to 8 NB RW rows and a share of the keys.  Its four math warps are
// RW groups of rows times 4 / RW groups of keys, each with 32 of a step's keys.
// Four more warps fill a ring of steps by TMA, two of them K and two V, in boxes of
// 128 to 16 rows of one page (what divides the page and the step), with the table's
// entries of the next 32 boxes in their lanes, and give most of their registers to
// the math warps.  (Copies from the math warps took 370 of the 1700 cycles of a step.)
//
// The products are mma.sync m16n8k16 in f16 with the keys, or the dims of values,
// as the 16 rows and NB times 8 query rows as columns: few query rows leave little
// of a product unused, and what was converted once serves all NB.  An e4m3 value
// is an f16 value, so keys and values enter exactly, converted in registers; so
// does q, a bf16 row times the power of two that takes its largest to 2^14 .. 2^15
// (f16 as it is).  K: the four consecutive bytes that ldmatrix gives a lane are
// taken as elements 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of the product's 16 (c = lane %
// 4), and q is laid out alike, so nothing moves between lanes.  V: ldmatrix.trans
// gives bytes of two keys and two dims; a byte permutation makes them pairs of
// keys, and a product's rows g and g + 8 are dims 2 g and 2 g + 1 of 16.  The
// weights, keys by rows, turn into the second product's operand by movmatrix.
// (With query rows as the 16 and keys as columns the same bytes took 159 us where
// this takes 107, see below: half of each product idle, twice the accumulators.)
//
// Scales: those of keys multiply the scores.  Those of values, vs, join the
// exponent: t = score + log2(vs) for each key, m the running maximum of t, w = 2^(t
// - m) the weight in the second product, O = sum w x, and l = sum w / vs, so out = O
// / l.  One exponential a pair, and w has its digits relative to what the key may
// add to the result, however far the pages' scales are apart (within 2^100).  w is
// 2^15 at most, so over 2^29 keys with scales of 2^-100 l would pass 2^128: it is held
// times 2^-18, which leaves it between 2^-111 and 2^126, and O / l below 2^127.
//
// Shares of the keys, their joins by a cluster (up to four) or through a workspace,
// as in cached_kernel.cuh.  Masks are made where a step holds the sequence's end, the
// first keys' end, the window's edge or new tokens: one lane looks up 16 keys of one
// row.  Values of keys that none of a warp's rows sees are cleared in registers; a NaN
// in one that some see and others do not sends the step through loops over visible
// pairs.  A value whose scale is 0 counts as one that no row sees, but for its weight in
// l: log2(vs) is -infinity, which marks it, and 2^-100 in its place.
//
// 32 sequences x 8 key heads x up to 16385 keys of 128, one token of 32 heads, bf16:
// 106 us, 6.8 TB/s, the measured copy rate.  One sequence of 200003 keys, one key head
// of 8: 13.7 us, 3.7 TB/s: 3 us before the first products, 4 for the join.  Where a
// call is small a step is latency (1200 cycles alone on its scheduler), and so is the
// code that runs once: rolled loops for q took 1 us off a call.  With many rows the
// bound is the two warps a scheduler has: 22 cycles a product of 16 keys x 8 rows x 16
// dims whatever else a step does, where the tensor core needs 8 (11 tokens of 4 heads,
// 13 x 4 x 38131 keys of 128: 150 us, 2.3 TB/s).
#pragma once

#include "cached_kernel.cuh"
#include "e4m3.cuh"

namespace vattn {

constexpr int kPagedKeys = 32;  // keys of a warp's part of a step
constexpr int kPagedWarps = 4;  // math warps
constexpr int kPagedCluster = 4;  // shares that a cluster of blocks joins by itself
constexpr float kPagedSumScale = 0x1p-18f;  // l is held times this (above)
constexpr float kPagedZeroLog2 = -100.0f;   // of the scale that counts for values of zeros

struct PagedParams {
  WindowParams w;  // n_keys: rows that the table has room for; kv_len: the cache's
  RowsTensor q, out;
  const uint8_t* pool[2];  // k, v (kDim), and from page to page, head to head
  long long ps[2][2];
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  uint32_t* status;
  float* part_o;   // [sequence and key head][row block][split][8 NB RW][dim]
  float* part_ml;  // ... [8 NB RW][2]: maximum (log2 units) and sum
  long long n_pages;
  int max_pages, page;
  int box, log_box;  // rows of a box
  int rows;          // group * n_queries
  int row_blocks;
  int splits;
  float scale_log2;
  FastDiv d_page, d_splits, d_row_blocks, d_kv_heads, d_group;
};

// The keys of one sequence, in boxes: those of the first keys, then those from the
// lowest window to the end; and a split's share of them.
struct PagedSpan {
  int base, len;    // new token t is row base + t; rows in use
  int first;        // no row sees keys in [sinks, first)
  int heads, begin; // listed: boxes [0, heads) and [begin, ..)
  int per, n;       // boxes of a share (whole steps), of all

  __device__ __forceinline__ static PagedSpan make(const WindowParams& w, int log_box, int groups, int b, const FastDiv& splits) {
    PagedSpan s;
    const int box = 1 << log_box;
    s.len = min(max(w.kv_len[b], 0), w.n_keys);
    s.base = s.len - w.n_queries;
    s.first = max(0, s.base - w.window + 1);
    s.begin = s.first >> log_box;
    s.heads = min((min(w.sinks, s.len) + box - 1) >> log_box, s.begin);
    s.n = s.heads + ((s.len + box - 1) >> log_box) - s.begin;
    const int unit = (groups * kPagedKeys) >> log_box;  // a step
    const int some = static_cast<int>(splits.div(static_cast<uint32_t>(s.n) + splits.d - 1));
    s.per = (some + unit - 1) & ~(unit - 1);  // (a power of two)
    return s;
  }
  __device__ __forceinline__ int box(int i) const { return i < heads ? i : begin + (i - heads); }
  __device__ __forceinline__ bool has(int split) const { return split == 0 || split * per < n; }
  __device__ __forceinline__ bool one() const { return per >= n; }
  __device__ __forceinline__ int shares() const { return n == 0 ? 1 : (n + per - 1) / per; }
};

// Place of 16-byte chunk c in shared row r of CH chunks, as TMA's swizzle of rows of
// 16 CH bytes has it.
template <int CH>
__device__ __forceinline__ int paged_swizzled(int r, int c) {
  return c ^ (CH == 8 ? r & 7 : CH == 4 ? (r >> 1) & 3 : (r >> 2) & 1);
}

// The same in a row of q, 2 DP bytes.
template <int DP>
__device__ __forceinline__ int paged_swizzled_q(int r, int c) {
  return c ^ (DP >= 64 ? r & 7 : (r >> 1) & 3);
}

template <int DP, int NB, int RW>
struct PagedPlan {
  static constexpr int kThreads = 256;
  static constexpr int kKw = kPagedWarps / RW;  // groups of keys
  static constexpr int kRows = 8 * NB * RW;
  static constexpr int kStepKeys = kKw * kPagedKeys, kLogStep = RW == 1 ? 7 : (RW == 2 ? 6 : 5);
  static_assert(kStepKeys == 1 << kLogStep, "a power of two");
  static constexpr int kTileBytes = kStepKeys * DP;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = DP == 128 ? 3 : (DP == 64 ? 4 : 6);
  static constexpr int kResultStride = DP + 4;  // floats of a row: O, maximum, sum
  static constexpr int kResultBytes = kPagedWarps * 8 * NB * kResultStride * 4;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kOffRows = kRingBytes > kResultBytes ? kRingBytes : kResultBytes;  // what each row sees
  static constexpr int kOffQ = kOffRows + kRows * 16;  // q as f16, rows of 2 DP bytes, and behind it each row's factor
  static constexpr int kOffMeta = kOffQ + kRows * (2 * DP + 16);  // [stage][8] scales and places of a step's boxes
  static constexpr int kOffBar = kOffMeta + kStages * 128;
  static constexpr int kSmemBytes = kOffBar + 16 * kStages + 32 + 1024;  // + alignment slack
  static constexpr uint32_t kRegsOther = 40, kRegsMath = 216;  // their sum: what two blocks' launches have
};

// 8 x 8 16-bit elements, two neighbours of a row a lane, transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// What a row sees: new token u by bit u, and of the rows before the new tokens (before
// old_end; 0: it sees nothing at all) what lies above lo or among the first keys.
struct PagedRow {
  uint64_t news;
  int lo, old_end;
};

__device__ __forceinline__ uint64_t bits64_upto(int hi) { return hi >= 63 ? ~0ull : (hi < 0 ? 0ull : (2ull << hi) - 1); }
// Keys j .. j + 15 of these, bit i key j + i.
__device__ __forceinline__ uint32_t paged_sees(const PagedRow& y, int j, int base, int sinks) {
  const uint32_t old = bits_upto(y.old_end - 1 - j, 0) & (~bits_upto(y.lo - j, 0) | bits_upto(sinks - 1 - j, 0));
  const int d = j - base;
  const uint64_t at = d >= 0 ? (d < 64 ? y.news >> d : 0) : (d > -16 ? y.news << -d : 0);
  return (old | static_cast<uint32_t>(at)) & 0xffffu;
}

// Are rows of kDim bytes copied untiled (see the kernel)?
__host__ __device__ constexpr bool paged_tight(int kDim) { return kDim % 32 == 16; }

// The math warps: all of the share's keys, then their results, joined.
template <typename T, int DP, int NB, int RW, int kDim>
__device__ __forceinline__ void paged_math(const PagedParams& p, const Pipe& pipe, uint8_t* smem, uint32_t smem_s,
                                           const PagedRow* rows, const PagedSpan& sp, uint32_t bk, int b,
                                           int kh, int rb, int split) {
  using P = PagedPlan<DP, NB, RW>;
  constexpr bool kTight = paged_tight(kDim);
  constexpr int CH = (kDim != 0 ? kDim : DP) / 16;  // 16-byte chunks of a row, 16-element steps of a product
  constexpr int RS = P::kResultStride, S = P::kStages;
  const int tid = static_cast<int>(threadIdx.x), warp = tid >> 5, lane = tid & 31;
  const int rw = warp % RW, kw = warp / RW;
  const uint32_t bar0 = smem_s + P::kOffBar;
  auto full = [bar0](int st) -> uint32_t { return bar0 + 8u * st; };
  auto empty = [bar0](int st) -> uint32_t { return bar0 + 8u * (S + st); };
  const WindowParams& w = p.w;
  const int D = w.dim, log_boxes = P::kLogStep - p.log_box;
  // a shared row of K or V: DP bytes, swizzled, or just those that there are
  constexpr int pitch = kTight ? kDim : DP;
  auto tile_at = [](int r, int c) {
    return static_cast<uint32_t>(kTight ? r * kDim + c * 16 : r * DP + (paged_swizzled<DP / 16>(r, c) << 4));
  };
  const bool clustered = p.splits > 1 && p.splits <= kPagedCluster;
  float* const res = reinterpret_cast<float*>(smem);  // results, over the ring: [group of keys][kRows][RS]
  const int g = lane >> 2, c4 = lane & 3;
  // ---- q to f16 in shared memory, DP / 8 lanes a row, the 16 elements of a product's
  // step in the order of K's bytes: 4 c, 4 c + 1 of c = 0 .. 3, then 4 c + 2, 4 c + 3
  // (rolled loops: this runs once, and most of its time was that of fetching its code)
  const uint32_t q_s = smem_s + P::kOffQ;
  float* const row_factor = reinterpret_cast<float*>(smem + P::kOffQ + P::kRows * 2 * DP);
#pragma unroll 1
  for (int i = tid; i < P::kRows * (DP / 8); i += 32 * kPagedWarps) {
    const int r = i / (DP / 8), d = i % (DP / 8);  // 8 elements from 8 d on
    const int rr = rb * P::kRows + r;
    uint32_t head;
    const int t = static_cast<int>(p.d_group.div(static_cast<uint32_t>(rr), &head));
    Vec<T, 8> x;
#pragma unroll
    for (int f = 0; f < 8; ++f) x.e[f] = Elem<T>::narrow(0.0f);
    if (rr < p.rows && d * 8 < D)
      x = *reinterpret_cast<const Vec<T, 8>*>(rows_at<T>(p.q, b, kh * w.group + static_cast<int>(head), t) + d * 8);
    float y[8], factor = p.scale_log2;
    x.widen(y);
    if constexpr (Elem<T>::kBf16) {
      float most = 0.0f;
#pragma unroll
      for (int f = 0; f < 8; ++f) most = fmaxf(most, fabsf(y[f]) < INFINITY ? fabsf(y[f]) : 0.0f);
#pragma unroll
      for (int o = DP / 16; o > 0; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
      // 2^k most in 2^14 .. 2^15 (2^127 takes k = -113); of small rows 2^k is 2^110, with
      // which bf16's smallest step, 2^-133, is f16's 2^-23, so nothing is lost either
      const int k = most == 0.0f ? 0 : min(14 + 127 - static_cast<int>(__float_as_uint(most) >> 23), 110);
      const float by = __int_as_float((127 + k) << 23);
      factor = p.scale_log2 * __int_as_float((127 - k) << 23);
#pragma unroll
      for (int f = 0; f < 8; ++f) y[f] *= by;
    }
    if (d == 0) row_factor[r] = factor;
    const uint32_t at = q_s + static_cast<uint32_t>(r * 2 * DP + (d & 1) * 8);  // of the step's two 16-byte chunks
    const int c = d & ~1;
    ptx::st_shared_v2(at + (paged_swizzled_q<DP>(r, c) << 4), pack2<__half>(y[0], y[1]), pack2<__half>(y[4], y[5]));
    ptx::st_shared_v2(at + (paged_swizzled_q<DP>(r, c + 1) << 4), pack2<__half>(y[2], y[3]), pack2<__half>(y[6], y[7]));
  }
  const int v0 = split * sp.per, v1 = min(sp.n, v0 + sp.per);
  const int steps = (max(v1 - v0, 0) + (1 << log_boxes) - 1) >> log_boxes;
  ptx::named_barrier_sync(1, P::kThreads);  // barriers and rows are there

  // ---- q as columns: lane / 4 of each eight rows; held in registers where there is room
  constexpr bool kHoldQ = NB <= 2;
  constexpr int CQ = kHoldQ ? (CH + 1) / 2 * 2 : 2;
  uint32_t qf[CQ][NB][2];
  auto load_q = [&](int ks) {  // of steps ks and ks + 1
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
      uint32_t x[4];  // matrices: the two halves of step ks, and of the next
      const int r = rw * 8 * NB + nb * 8 + (lane & 7);
      ldmatrix_x4(q_s + static_cast<uint32_t>(r * 2 * DP + (paged_swizzled_q<DP>(r, 2 * ks + (lane >> 3)) << 4)), x);
      qf[ks % CQ][nb][0] = x[0];
      qf[ks % CQ][nb][1] = x[1];
      qf[(ks + 1) % CQ][nb][0] = x[2];
      qf[(ks + 1) % CQ][nb][1] = x[3];
    }
  };
  float row_c[NB][2];  // of rows 2 c4 and 2 c4 + 1: from a product's sum to log2 units, but for the key's scale
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) row_c[nb][e] = row_factor[rw * 8 * NB + nb * 8 + 2 * c4 + e];
  if constexpr (kHoldQ) {
#pragma unroll
    for (int ks = 0; ks < CH; ks += 2) load_q(ks);
  }

  float m[NB][2], l[NB][2];
  float o[CH][NB][4];  // dims 16 ch + 2 g, + 1 (e / 2) of rows 2 c4, + 1 (e % 2)
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      m[nb][e] = -INFINITY;
      l[nb][e] = 0.0f;
    }
#pragma unroll
    for (int n = 0; n < CH; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][nb][e] = 0.0f;
  }

  // keys j .. j + 15 need no mask: all rows see them
  const int free_end = w.n_queries > 1 ? sp.base : sp.len;
  const int free_begin = w.n_queries > 1 ? max(0, sp.base + w.n_queries - w.window) : sp.first;
  int step = 0, st = 0;
  uint32_t turn = 0;
  for (; step < steps; ++step) {
    if (!pipe.wait_warp(full(st), turn, kSitePagedMath)) break;
    const uint32_t ks_s = smem_s + static_cast<uint32_t>(st * P::kStageBytes + kw * kPagedKeys * pitch);
    const uint32_t vs_s = ks_s + P::kTileBytes;
    uint32_t kf[CH][4];
#pragma unroll
    for (int ks = 0; ks < CH; ++ks)  // matrices: keys 0-7, 8-15, 16-23, 24-31 by the 16 dims of chunk ks
      ldmatrix_x4(ks_s + tile_at(lane, ks), kf[ks]);
    // the warp's keys by 16: first of each in the sequence (behind it if they are not
    // there), scales; those that not all rows see count as masked, and those whose
    // values are zeros (meta.x < 0)
    int j0[2];
    float4 meta[2];
    bool masked[2];
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
      const int at = kw * kPagedKeys + mb * 16;
      meta[mb] = ptx::ld_shared_v4(smem_s + P::kOffMeta + static_cast<uint32_t>((st * 8 + (at >> p.log_box)) * 16));
      const int j = __float_as_int(meta[mb].w) + (at & (p.box - 1));
      j0[mb] = j;
      masked[mb] = (meta[mb].x < 0.0f) | (j + 15 >= free_end) | ((j < free_begin) & (j + 15 >= w.sinks));
    }
    const bool some = masked[0] || masked[1];
    // ---- S = K Q^T, over the even and the odd chunks by themselves where that
    // leaves the tensor core fewer products in a row on one sum
    constexpr int PART = NB == 1 ? 2 : 1;
    float s[2][NB][4], s_odd[2][NB][4];  // keys 16 mb + g, + 8 (e / 2) of rows 2 c4, + 1 (e % 2)
#pragma unroll
    for (int mb = 0; mb < 2; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mb][nb][e] = s_odd[mb][nb][e] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < CH; ++ks) {
      if (!kHoldQ && ks % 2 == 0) load_q(ks);
#pragma unroll
      for (int mb = 0; mb < 2; ++mb) {
        const uint32_t a[4] = {e4m3_half2_lo(kf[ks][2 * mb]), e4m3_half2_lo(kf[ks][2 * mb + 1]),
                               e4m3_half2_hi(kf[ks][2 * mb]), e4m3_half2_hi(kf[ks][2 * mb + 1])};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          mma_16816<__half>(ks % PART ? s_odd[mb][nb] : s[mb][nb], a, qf[ks % CQ][nb][0], qf[ks % CQ][nb][1]);
      }
    }
    if (PART == 2) {
#pragma unroll
      for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mb][nb][e] += s_odd[mb][nb][e];
    }
    uint32_t vf[CH][4];  // the same matrices of V, transposed by pairs of dims, ahead of their use
#pragma unroll
    for (int n = 0; n < CH; ++n) ldmatrix_x4_trans(vs_s + tile_at(lane, n), vf[n]);
    // ---- masks: at the sequence's end, the first keys' end, the window's edge, among
    // the new tokens.  Lane i looks up rows i % 16 (+ 16) of the warp and keys i / 16.
    bool loops = false;
    uint32_t see[2][NB][2];  // of rows 2 c4 + e: 16 keys a word, where masked
    uint32_t any_w = 0;      // keys whose values some row takes
    if (some) {
      const int mb = lane >> 4, j = mb ? j0[1] : j0[0];
      uint32_t mine[(NB + 1) / 2], any = 0, every = 0xffffu;
#pragma unroll
      for (int q = 0; q < (NB + 1) / 2; ++q) {
        const int r = 16 * q + (lane & (NB - 2 * q == 1 ? 7 : 15));
        const PagedRow y = rows[rw * 8 * NB + r];
        mine[q] = paged_sees(y, j, sp.base, w.sinks);
        const bool live = y.old_end != 0 || y.news != 0;
        any |= live ? mine[q] : 0u;
        every &= live ? mine[q] : 0xffffu;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            see[k][nb][e] = __shfl_sync(0xffffffffu, mine[nb / 2], 16 * k + nb % 2 * 8 + 2 * c4 + e) >> g;  // its keys g and g + 8
#pragma unroll
            for (int h = 0; h < 2; ++h)
              if (!((see[k][nb][e] >> (8 * h)) & 1u)) s[k][nb][2 * h + e] = -INFINITY;
          }
      if ((mb ? meta[1].y : meta[0].y) == -INFINITY) any = 0;
      const uint32_t half = mb ? 0xffff0000u : 0x0000ffffu;
      any_w = __reduce_or_sync(0xffffffffu, (any << (16 * mb)) & half);
      const uint32_t every_w = __reduce_and_sync(0xffffffffu, (every << (16 * mb)) | ~half);
      // V of keys that none of the warp's rows sees may hold anything: zeros; and so may
      // the scales of 16 such keys (c below has bounds of its own)
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (((any_w >> (16 * k)) & 0xffffu) == 0) {
          meta[k].y = kPagedZeroLog2;
          meta[k].z = kPagedSumScale * 0x1p100f;
        }
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // keys 8 q + 2 c4, + 1: low and high halves
        const uint32_t a = any_w >> (8 * q + 2 * c4);
        const uint32_t keep = (a & 1u ? 0xffffu : 0u) | (a & 2u ? 0xffff0000u : 0u);
#pragma unroll
        for (int n = 0; n < CH; ++n) vf[n][q] &= keep;
      }
      // a NaN in a key that some rows see and others do not: loops over the visible pairs
      if ((any_w & ~every_w) != 0) {
        uint32_t bad = 0;
#pragma unroll
        for (int n = 0; n < CH; ++n)
#pragma unroll
          for (int q = 0; q < 4; ++q)  // a byte's low seven bits all ones: a carry out of them
            bad |= ((vf[n][q] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
        loops = __any_sync(0xffffffffu, bad != 0);
      }
    }
    // ---- online softmax, two rows a lane for each eight, eight lanes a row; a row is
    // rescaled once its maximum grew by more than 2^8 (exact after the final 1 / l),
    // and only then is the maximum over its lanes wanted
    float c[2][NB][2], top[NB][2];
    bool grew = false;
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int mb = 0; mb < 2; ++mb)  // not 0 or infinity, which -infinity or 0 make NaN
          c[mb][nb][e] = fminf(fmaxf(row_c[nb][e] * fabsf(meta[mb].x), 0x1p-126f), 0x1p127f);
        top[nb][e] = fmaxf(fmaf(fmaxf(s[0][nb][e], s[0][nb][e + 2]), c[0][nb][e], meta[0].y),
                           fmaf(fmaxf(s[1][nb][e], s[1][nb][e + 2]), c[1][nb][e], meta[1].y));
        grew |= top[nb][e] > m[nb][e] + kLazyLog2;
      }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float y = top[nb][e];
#pragma unroll
          for (int x = 4; x < 32; x *= 2) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, x));
          const bool more = y > m[nb][e] + kLazyLog2;
          const float alpha = more ? ptx::ex2_approx(m[nb][e] - y) : 1.0f;
          if (more) m[nb][e] = y;
          l[nb][e] *= alpha;
#pragma unroll
          for (int n = 0; n < CH; ++n) {
            o[n][nb][e] *= alpha;
            o[n][nb][e + 2] *= alpha;
          }
        }
    }
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float ref = kWeightLog2<__half> - (m[nb][e] == -INFINITY ? 0.0f : m[nb][e]);
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          const float shift = ref + meta[mb].y;
          s[mb][nb][e] = ptx::ex2_approx(fmaf(s[mb][nb][e], c[mb][nb][e], shift));
          s[mb][nb][e + 2] = ptx::ex2_approx(fmaf(s[mb][nb][e + 2], c[mb][nb][e], shift));
          l[nb][e] = fmaf(s[mb][nb][e] + s[mb][nb][e + 2], meta[mb].z, l[nb][e]);  // of this lane's keys
        }
      }
    // ---- O += V P
    if (!loops) {
      uint32_t pf[2][NB][2];
#pragma unroll
      for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            pf[mb][nb][e] = movmatrix_trans(pack2<__half>(s[mb][nb][2 * e], s[mb][nb][2 * e + 1]));
#pragma unroll
      for (int n = 0; n < CH; ++n) {
#pragma unroll
        for (int y = 0; y < 4; ++y) vf[n][y] = __byte_perm(vf[n][y], 0u, 0x3120);
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          const uint32_t a[4] = {e4m3_half2_lo(vf[n][2 * mb]), e4m3_half2_hi(vf[n][2 * mb]),
                                 e4m3_half2_lo(vf[n][2 * mb + 1]), e4m3_half2_hi(vf[n][2 * mb + 1])};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma_16816<__half>(o[n][nb], a, pf[mb][nb][0], pf[mb][nb][1]);
        }
      }
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((see[k][nb][e & 1] >> (8 * (e >> 1))) & 1u) || ((any_w >> (16 * k)) & 0xffffu) == 0) s[k][nb][e] = -1.0f;
#pragma unroll 1
      for (int y = 0; y < 8; ++y)
#pragma unroll
        for (int h = 0; h < 4; ++h) {  // key 8 h + y: its weights are with lanes 4 y ..
          float u[NB][2];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int e = 0; e < 2; ++e) u[nb][e] = __shfl_sync(0xffffffffu, s[h >> 1][nb][2 * (h & 1) + e], 4 * y + c4);
          const int r = 8 * h + y;
#pragma unroll
          for (int n = 0; n < CH; ++n) {
            const uint32_t z = *reinterpret_cast<const uint16_t*>(smem + (vs_s - smem_s) + tile_at(r, n) + g * 2);
            const uint32_t z2 = e4m3_half2_lo(z);
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&z2));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (!(u[nb][e] < 0.0f)) {
                  o[n][nb][e] = fmaf(u[nb][e], v.x, o[n][nb][e]);
                  o[n][nb][e + 2] = fmaf(u[nb][e], v.y, o[n][nb][e + 2]);
                }
          }
        }
    }
    pipe_warp_arrive(empty(st));
    if (++st == S) {
      st = 0;
      turn ^= 1;
    }
  }
  ptx::named_barrier_sync(2, 32 * kPagedWarps);  // the ring is free: the warps' results go there
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
#pragma unroll
      for (int x = 4; x < 32; x *= 2) l[nb][e] += __shfl_xor_sync(0xffffffffu, l[nb][e], x);
      float* to = res + (kw * P::kRows + rw * 8 * NB + nb * 8 + 2 * c4 + e) * RS;
#pragma unroll
      for (int n = 0; n < CH; ++n) *reinterpret_cast<float2*>(to + n * 16 + 2 * g) = make_float2(o[n][nb][e], o[n][nb][e + 2]);
      if (g == 0) *reinterpret_cast<float2*>(to + DP) = make_float2(m[nb][e], l[nb][e]);
    }
  ptx::named_barrier_sync(2, 32 * kPagedWarps);
  // ---- join the warps that shared the keys
  auto write = [&](int rr, int d, float sum, float (&acc)[8]) {
    uint32_t head;
    const int t = static_cast<int>(p.d_group.div(static_cast<uint32_t>(rr), &head));
    const bool none = sum == 0.0f || cached_word(w, b, t, sp.base) == 0;
    const float inv = 1.0f / sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = none ? 0.0f : acc[e] * inv * kPagedSumScale;
    reinterpret_cast<Vec<T, 8>*>(rows_at_mut<T>(p.out, b, kh * w.group + static_cast<int>(head), t) + d)->narrow(acc);
  };
  const bool alone = p.splits == 1 || (sp.one() && !clustered);
  const int per_row = D / 8;
  for (int x = tid; x < P::kRows * per_row; x += 32 * kPagedWarps) {
    const int r = x / per_row, d = (x - r * per_row) * 8;
    const int rr = rb * P::kRows + r;
    if (rr >= p.rows) continue;
    float* from = res + r * RS;  // + kRows for the next group of keys
    float mx = -INFINITY;
#pragma unroll
    for (int y = 0; y < P::kKw; ++y) mx = fmaxf(mx, from[y * P::kRows * RS + DP]);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f, acc[8] = {};
#pragma unroll
    for (int y = 0; y < P::kKw; ++y) {
      const float* f = from + y * P::kRows * RS;
      const float a = ptx::ex2_approx(f[DP] - ref);
      sum = fmaf(a, f[DP + 1], sum);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(a, f[d + e], acc[e]);
    }
    if (clustered) {  // in place of the first group's
#pragma unroll
      for (int e = 0; e < 8; e += 4) *reinterpret_cast<float4*>(from + d + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
    } else if (alone) {
      write(rr, d, sum, acc);
    } else {
      const long long at = ((static_cast<long long>(bk) * p.row_blocks + rb) * p.splits + split) * P::kRows + r;
      float4* to = reinterpret_cast<float4*>(p.part_o + at * D + d);
      to[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
      to[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
      if (d == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(mx, sum);
    }
  }
  if (!clustered) {
    ptx::grid_dep_launch();
    return;
  }
  ptx::named_barrier_sync(2, 32 * kPagedWarps);
  if (tid < P::kRows) {
    float* row = res + tid * RS;
    float mx = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int y = 0; y < P::kKw; ++y) mx = fmaxf(mx, row[y * P::kRows * RS + DP]);
    const float ref = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
    for (int y = 0; y < P::kKw; ++y) {
      const float* f = row + y * P::kRows * RS + DP;
      sum = fmaf(ptx::ex2_approx(f[0] - ref), f[1], sum);
    }
    *reinterpret_cast<float2*>(row + DP) = make_float2(mx, sum);
  }
  ptx::cluster_sync();
  const int shares = sp.shares();
  for (int x = split * 32 * kPagedWarps + tid; x < P::kRows * per_row; x += p.splits * 32 * kPagedWarps) {
    const int r = x / per_row, d = (x - r * per_row) * 8;
    const int rr = rb * P::kRows + r;
    if (rr >= p.rows) continue;
    const uint32_t row = smem_s + static_cast<uint32_t>(r * RS * 4);
    float2 ml[kPagedCluster];
    float mx = -INFINITY;
#pragma unroll
    for (int s = 0; s < kPagedCluster; ++s) {
      ml[s] = s < shares ? ptx::ld_cluster_v2(ptx::cluster_map(row + DP * 4, s)) : make_float2(-INFINITY, 0.0f);
      mx = fmaxf(mx, ml[s].x);
    }
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f, acc[8] = {};
#pragma unroll
    for (int s = 0; s < kPagedCluster; ++s) {
      if (s >= shares) break;
      const float a = ptx::ex2_approx(ml[s].x - ref);
      sum = fmaf(a, ml[s].y, sum);
      const uint32_t from = ptx::cluster_map(row + static_cast<uint32_t>(d) * 4, s);
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 f = ptx::ld_cluster_v2(from + e * 4);
        acc[e] = fmaf(a, f.x, acc[e]);
        acc[e + 1] = fmaf(a, f.y, acc[e + 1]);
      }
    }
    write(rr, d, sum, acc);
  }
  ptx::cluster_sync();  // before the shared memory that others read goes
  ptx::grid_dep_launch();
}

// kDim: 0, or 48, 80 or 112 dims whose rows are one behind the other in a page: boxes as
// untiled copies, and shared rows as they are.  As tiles of 64 or 128 columns such rows
// begin and end inside the sectors that a copy reads: 32 x 8 key heads x up to 16000 keys
// x 80 took 127 us and now 79, of 112 101 and 99, of 48 75 and 60 (96 and 64 dims take 84
// and 62), and the products skip the chunks that are not there (200003 keys of one head x
// 80 17.5 and 11.8).  An odd number of 16-byte chunks a row leaves ldmatrix without a
// conflict, unswizzled.  96: tiles, with the products of the chunks that are there.
template <typename T, int DP, int NB, int RW, int kDim>
__global__ void __launch_bounds__(PagedPlan<DP, NB, RW>::kThreads, 2)
    vattn_paged_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ PagedParams p) {
  using P = PagedPlan<DP, NB, RW>;
  constexpr bool kTight = paged_tight(kDim);
  constexpr int S = P::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int kpos[VATTN_MAX_NEW_TOKENS];
  const uint32_t raw_s = ptx::smem_addr(smem_raw);
  const uint32_t smem_s = (raw_s + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (smem_s - raw_s);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = smem_s + P::kOffBar;
  auto full = [bar0](int st) -> uint32_t { return bar0 + 8u * st; };
  auto empty = [bar0](int st) -> uint32_t { return bar0 + 8u * (S + st); };
  const Pipe pipe{bar0 + 16u * S};
  const WindowParams& w = p.w;
  uint32_t split_u, rb_u, kh_u;
  const uint32_t bk = p.d_row_blocks.div(p.d_splits.div(blockIdx.x, &split_u), &rb_u);
  const int b = static_cast<int>(p.d_kv_heads.div(bk, &kh_u));
  const int split = static_cast<int>(split_u), rb = static_cast<int>(rb_u), kh = static_cast<int>(kh_u);
  const bool clustered = p.splits > 1 && p.splits <= kPagedCluster;

  PagedRow* const rows = reinterpret_cast<PagedRow*>(smem + P::kOffRows);
  const int log_boxes = P::kLogStep - p.log_box, boxes = 1 << log_boxes;  // of a step
  if (warp == kPagedWarps && lane == 0) {
    for (int i = 0; i < S; ++i) {
      ptx::mbar_init(full(i), boxes > 1 ? 4 : 2);  // the loaders that have boxes
      ptx::mbar_init(empty(i), kPagedWarps);
    }
    pipe.init(w, p.status);
    ptx::fence_mbar_init();
    if (!kTight) {
      ptx::prefetch_tensormap(&tm_k);
      ptx::prefetch_tensormap(&tm_v);
    }
  }
  ptx::grid_dep_wait();
  const PagedSpan sp = PagedSpan::make(w, p.log_box, P::kKw, b, p.d_splits);
  if (!clustered && !sp.has(split)) return;  // (in a cluster: with no keys, but at its barriers)
  if (warp >= kPagedWarps) {
    ptx::regs_decrease<P::kRegsOther>();
    const int v0 = split * sp.per, v1 = min(sp.n, v0 + sp.per);
    const int steps = (max(v1 - v0, 0) + boxes - 1) >> log_boxes;
    // ------------------------------------------------------ boxes into the ring
    // lane i has what box i of 32 needs, and of the 32 after
    const int loader = warp - kPagedWarps, mine = boxes - (loader >> 1);  // boxes loader / 2, + 2, ... of a step's K or V
    struct Box {
      int page, row, key0;          // page: behind the last if it is not there, and reads as zeros
      float k, log2_v, inv_v;       // k < 0: the values are zeros
    };
    auto place = [&](int i, Box& x) {  // of the share's box i
      x.key0 = sp.box(v0 + i) << p.log_box;
      x.page = static_cast<int>(p.n_pages);
      uint32_t row = 0;
      if (v0 + i < v1) {
        const uint32_t lp = p.d_page.div(static_cast<uint32_t>(x.key0), &row);
        const int id = p.table[static_cast<long long>(b) * p.max_pages + lp];
        if (id >= 0 && id < p.n_pages) x.page = id;
      }
      x.row = static_cast<int>(row);
      if (x.page >= p.n_pages) x.key0 = 1 << 30;
    };
    auto scales = [&](Box& x) {  // (the first loader's)
      x.k = x.inv_v = 1.0f;
      x.log2_v = 0.0f;
      if (loader != 0 || x.page >= p.n_pages) return;
      const long long at = static_cast<long long>(x.page) * w.kv_heads + kh;
      const float v = p.v_scale[at];
      x.k = p.k_scale[at];
      if (v == 0.0f) x.k = -fmaxf(x.k, 0x1p-126f);
      x.log2_v = log2f(v);
      x.inv_v = kPagedSumScale / v;
    };
    Box now{}, next{};
    const uint64_t once = ptx::policy_evict_first();
    const CUtensorMap* const tm = (loader & 1) != 0 ? &tm_v : &tm_k;
    const int box_bytes = (kTight ? kDim : DP) << p.log_box;
    // The copies of a step, whose boxes are with lanes l0, l0 + 1, ..., to place st.
    auto copies = [&](int st, int l0) {
      for (int i = loader >> 1; i < boxes; i += 2) {
        const int pg = __shfl_sync(0xffffffffu, now.page, l0 + i), row = __shfl_sync(0xffffffffu, now.row, l0 + i);
        const uint32_t to = smem_s + static_cast<uint32_t>(st * P::kStageBytes + (loader & 1) * P::kTileBytes + i * box_bytes);
        if constexpr (kTight) {  // (a page that is not there leaves the place as it was: its keys are masked)
          const uint8_t* from = p.pool[loader & 1] + pg * p.ps[loader & 1][0] + kh * p.ps[loader & 1][1] + row * kDim;
          if (pg < p.n_pages && ptx::elect_one())
            ptx::bulk_load_hint(to, from, static_cast<uint32_t>(box_bytes), full(st), once);
        } else if (ptx::elect_one()) {
          ptx::tma_load_4d_hint(to, tm, full(st), 0, row, kh, pg, once);
        }
      }
    };
    // What the products need beside them, and the barrier's count, which the copies may be ahead of.
    auto announce = [&](int st, int l0) {
      const int which = lane - l0;
      if (loader == 0 && which >= 0 && which < boxes)
        ptx::st_shared_v4(smem_s + P::kOffMeta + static_cast<uint32_t>((st * 8 + which) * 16), now.k, now.log2_v, now.inv_v,
                          __int_as_float(now.key0));
      int copied = (mine + 1) >> 1;
      if constexpr (kTight) {
        const uint32_t here = __ballot_sync(0xffffffffu, now.page < p.n_pages) >> l0;
        copied = __popc(here & ((1u << boxes) - 1u) & (loader >> 1 != 0 ? 0xaaaaaaaau : 0x55555555u));
      }
      __syncwarp();
      if (mine > 0 && ptx::elect_one()) ptx::mbar_arrive_expect_tx(full(st), static_cast<uint32_t>(copied * box_bytes));
    };
    place(lane, now);
    ptx::named_barrier_sync(3, P::kThreads - 32 * kPagedWarps);  // the barriers
    const int first = min(min(S, steps), 32 >> log_boxes);
    for (int i = 0; i < first; ++i) copies(i, i << log_boxes);
    scales(now);
    place(32 + lane, next);
    // positions of the new tokens of a tree, then what each row sees
    constexpr int kLoaderThreads = P::kThreads - 32 * kPagedWarps;
    const int lt = tid - 32 * kPagedWarps;
    if (w.tree != nullptr) {
      if (lt < w.n_queries) kpos[lt] = sp.base + __popcll(cached_word(w, b, lt, sp.base)) - 1;
      ptx::named_barrier_sync(3, kLoaderThreads);
    }
    static_assert(P::kRows <= kLoaderThreads && VATTN_MAX_NEW_TOKENS <= kLoaderThreads, "a thread each");
    if (lt < P::kRows) {
      const int rr = rb * P::kRows + lt;
      const int t = static_cast<int>(p.d_group.div(static_cast<uint32_t>(rr)));
      PagedRow y{rr < p.rows ? cached_word(w, b, t, sp.base) : 0, 0x7fffffff, 0};
      if (y.news != 0) {
        y.old_end = max(0, sp.base);
        y.lo = sp.base + __popcll(y.news) - 1 - w.window;
        if (w.tree == nullptr) {
          y.news &= ~bits64_upto(t - w.window) | bits64_upto(w.sinks - 1 - sp.base);
        } else if (y.lo >= sp.base - 1) {  // a window inside the tree (tokens without bits are at base - 1)
          for (uint64_t left = y.news; left != 0; left &= left - 1) {
            const int u = __ffsll(static_cast<long long>(left)) - 1, at = kpos[u];
            if (at <= y.lo && at >= w.sinks) y.news &= ~(1ull << u);
          }
        }
      }
      rows[lt] = y;
    }
    for (int i = 0; i < first; ++i) announce(i, i << log_boxes);
    ptx::named_barrier_sync(1, P::kThreads);
    int step = first, st = first == S ? 0 : first;
    uint32_t turn = first == S ? 0u : 1u;  // of the place's last use, which is awaited
    bool ok = true;
    for (; step < steps; ++step) {
      const int i0 = step << log_boxes, l0 = i0 & 31;
      if (l0 == 0) {
        now = next;
        scales(now);
        place(i0 + 32 + lane, next);
      }
      if (!(ok = pipe.wait_warp(empty(st), turn, kSitePagedLoad))) break;
      announce(st, l0);
      copies(st, l0);
      if (++st == S) {
        st = 0;
        turn ^= 1u;
      }
    }
    if (!ok && lane == 0)  // the copies in flight land before the block exits
      for (int d = max(0, step - S); d < step; ++d)
        pipe.drain(full(d % S), static_cast<uint32_t>((d / S) & 1), kSitePagedDrain);
    __syncwarp();
  } else {
    ptx::regs_increase<P::kRegsMath>();
    paged_math<T, DP, NB, RW, kDim>(p, pipe, smem, smem_s, rows, sp, bk, b, kh, rb, split);
  }
}

// Merges the shares of 32 dims of a row, one block each: the weight of every share
// first, then eight lanes a share, 16 bytes a lane, add up every 32nd one, and the
// block their sums, in a fixed order.
template <typename T, int ROWS, int KW>
__global__ void __launch_bounds__(256) vattn_paged_join_kernel(const __grid_constant__ PagedParams p) {
  __shared__ float weight[kCachedMaxSplits];
  __shared__ float red[16];
  __shared__ float4 acc_s[8][8];
  const WindowParams& w = p.w;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = w.dim;
  const long long bk = blockIdx.x / p.rows;
  const int rr = static_cast<int>(blockIdx.x - bk * p.rows);
  const int b = static_cast<int>(bk / w.kv_heads), kh = static_cast<int>(bk - static_cast<long long>(b) * w.kv_heads);
  const int t = rr / w.group, d = static_cast<int>(blockIdx.y) * 32 + (lane & 7) * 4;
  ptx::grid_dep_wait();
  const PagedSpan sp = PagedSpan::make(w, p.log_box, KW, b, p.d_splits);
  const int shares = sp.shares();
  if (shares == 1) return;  // written by its block
  const bool none = cached_word(w, b, t, sp.base) == 0;
  const long long at0 = (bk * p.row_blocks + rr / ROWS) * p.splits * ROWS + rr % ROWS;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + at0;
  static_assert(kCachedMaxSplits <= 512, "two shares a thread, 16 of its dims");
  // all that the thread adds up, on its way while the weights are formed
  float4 y[kCachedMaxSplits / 32];
  {
    const float* from = p.part_o + at0 * D + d;
#pragma unroll
    for (int i = 0; i < kCachedMaxSplits / 32; ++i) {
      const int s = warp * 4 + (lane >> 3) + 32 * i;
      y[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (d < D && s < shares) y[i] = *reinterpret_cast<const float4*>(from + s * static_cast<long long>(ROWS) * D);
    }
  }
  float2 f[2];
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = tid + 256 * i;
    f[i] = s < shares ? ml[s * static_cast<long long>(ROWS)] : make_float2(-INFINITY, 0.0f);
    mx = fmaxf(mx, f[i].x);
  }
  mx = warp_max(mx);
  if (lane == 0) red[warp] = mx;
  __syncthreads();
  mx = red[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, red[i]);
  const float ref = mx == -INFINITY ? 0.0f : mx;
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float a = ptx::ex2_approx(f[i].x - ref);
    weight[tid + 256 * i] = a;
    sum = fmaf(a, f[i].y, sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) red[8 + warp] = sum;
  __syncthreads();
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < kCachedMaxSplits / 32; ++i) {  // (weights behind the last share are 0)
    const float a = weight[warp * 4 + (lane >> 3) + 32 * i];
    acc.x = fmaf(a, y[i].x, acc.x);
    acc.y = fmaf(a, y[i].y, acc.y);
    acc.z = fmaf(a, y[i].z, acc.z);
    acc.w = fmaf(a, y[i].w, acc.w);
  }
#pragma unroll
  for (int o = 8; o < 32; o *= 2) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
  }
  if (lane < 8) acc_s[warp][lane] = acc;
  __syncthreads();
  if (tid >= 8 || d >= D) return;
  sum = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) sum += red[8 + i];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    const float4 y = acc_s[i][lane];
    acc.x += y.x;
    acc.y += y.y;
    acc.z += y.z;
    acc.w += y.w;
  }
  const float inv = 1.0f / sum;
  const bool zero = none || sum == 0.0f;
  const float out[4] = {zero ? 0.0f : acc.x * inv * kPagedSumScale, zero ? 0.0f : acc.y * inv * kPagedSumScale,
                        zero ? 0.0f : acc.z * inv * kPagedSumScale, zero ? 0.0f : acc.w * inv * kPagedSumScale};
  reinterpret_cast<Vec<T, 4>*>(rows_at_mut<T>(p.out, b, kh * w.group + (rr - t * w.group), t) + d)->narrow(out);
}

// The same for few shares (32 at most): a warp has a row, lane i the weight of share i.
template <typename T, int ROWS, int KW>
__global__ void __launch_bounds__(256) vattn_paged_join_few_kernel(const __grid_constant__ PagedParams p) {
  const WindowParams& w = p.w;
  const int lane = static_cast<int>(threadIdx.x) & 31, D = w.dim;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= static_cast<long long>(w.batch) * w.kv_heads * p.rows) return;
  const long long bk = row / p.rows;
  const int rr = static_cast<int>(row - bk * p.rows);
  const int b = static_cast<int>(bk / w.kv_heads), kh = static_cast<int>(bk - static_cast<long long>(b) * w.kv_heads);
  const int t = rr / w.group;
  ptx::grid_dep_wait();
  const PagedSpan sp = PagedSpan::make(w, p.log_box, KW, b, p.d_splits);
  const int shares = sp.shares();
  if (shares == 1) return;  // written by its block
  const bool none = cached_word(w, b, t, sp.base) == 0;
  const long long at0 = (bk * p.row_blocks + rr / ROWS) * p.splits * ROWS + rr % ROWS;
  const float* from = p.part_o + at0 * D + (lane * 4 < D ? lane * 4 : 0);
  constexpr int kAhead = 12;  // shares on their way while the weights are formed
  float4 ahead[kAhead];
#pragma unroll
  for (int s = 0; s < kAhead; ++s)
    ahead[s] = s < shares ? *reinterpret_cast<const float4*>(from + s * static_cast<long long>(ROWS) * D)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float2 ml = lane < shares ? reinterpret_cast<const float2*>(p.part_ml)[at0 + lane * static_cast<long long>(ROWS)]
                                  : make_float2(-INFINITY, 0.0f);
  const float mx = warp_max(ml.x), ref = mx == -INFINITY ? 0.0f : mx;
  const float weight = ptx::ex2_approx(ml.x - ref);
  float sum = weight * ml.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](int s, const float4& y) {
    const float a = __shfl_sync(0xffffffffu, weight, s);  // (0 behind the last share)
    acc.x = fmaf(a, y.x, acc.x);
    acc.y = fmaf(a, y.y, acc.y);
    acc.z = fmaf(a, y.z, acc.z);
    acc.w = fmaf(a, y.w, acc.w);
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) add(s, ahead[s]);
#pragma unroll 4
  for (int s = kAhead; s < shares; ++s) add(s, *reinterpret_cast<const float4*>(from + s * static_cast<long long>(ROWS) * D));
  if (lane * 4 >= D) return;
  const float inv = 1.0f / sum;
  const bool zero = none || sum == 0.0f;
  const float out[4] = {zero ? 0.0f : acc.x * inv * kPagedSumScale, zero ? 0.0f : acc.y * inv * kPagedSumScale,
                        zero ? 0.0f : acc.z * inv * kPagedSumScale, zero ? 0.0f : acc.w * inv * kPagedSumScale};
  reinterpret_cast<Vec<T, 4>*>(rows_at_mut<T>(p.out, b, kh * w.group + (rr - t * w.group), t) + lane * 4)->narrow(out);
}

}  // namespace vattn
