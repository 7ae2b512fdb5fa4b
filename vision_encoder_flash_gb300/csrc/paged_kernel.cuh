// paged_kernel.cuh -- attention of a few new tokens over the 8-bit paged cache
// (vattn_forward_paged).
//
// Memory bound: every visible key and value, one byte an element, is read once for
// all rows (new token, query head of the group) of its key head together.  A
// block takes up to 8 NB RW rows and a share of the keys.  Its four warps are RW
// groups of rows times 4 / RW groups of keys; a group of keys takes every 4 / RW-th
// 32 keys of the share through a ring of its own, filled by TMA in boxes of 32 or
// 16 rows of one page (what divides the page) from the group's first warp, which
// has the table's entries and the scales of its next 32 boxes in its lanes.
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
//
// Scales: those of keys multiply the scores.  Those of values, vs, join the
// exponent: t = score + log2(vs) for each key, m the running maximum of t, w = 2^(t
// - m) the weight in the second product, O = sum w x, and l = sum w / vs, so out = O
// / l.  One exponential a pair, and w has its digits relative to what the key may
// add to the result, however far the pages' scales are apart (within 2^100).
//
// Shares of the keys, their joins by a cluster (up to four) or through a
// workspace, masks and values that are not finite: as in cached_kernel.cuh.
#pragma once

#include "cached_kernel.cuh"
#include "e4m3.cuh"

namespace vattn {

constexpr int kPagedKeys = 32;  // keys of a step
constexpr int kPagedWarps = 4;
#ifndef PCL
#define PCL 4
#endif
constexpr int kPagedCluster = PCL;

struct PagedParams {
  WindowParams w;  // n_keys: rows that the table has room for; kv_len: the cache's
  RowsTensor q, out;
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
  int per, n;       // boxes of a share (whole steps of all its groups of keys), of all

  __device__ __forceinline__ static PagedSpan make(const WindowParams& w, int log_box, int groups, int b, int splits) {
    PagedSpan s;
    const int box = 1 << log_box;
    s.len = min(max(w.kv_len[b], 0), w.n_keys);
    s.base = s.len - w.n_queries;
    s.first = max(0, s.base - w.window + 1);
    s.begin = s.first >> log_box;
    s.heads = min((min(w.sinks, s.len) + box - 1) >> log_box, s.begin);
    s.n = s.heads + ((s.len + box - 1) >> log_box) - s.begin;
    const int unit = (groups * kPagedKeys) >> log_box;
    s.per = ((s.n + splits - 1) / splits + unit - 1) / unit * unit;
    return s;
  }
  __device__ __forceinline__ int box(int i) const { return i < heads ? i : begin + (i - heads); }
  __device__ __forceinline__ int shares() const { return n == 0 ? 1 : (n + per - 1) / per; }
};

// Place of 16-byte chunk c in shared row r of CH chunks, as TMA's swizzle of rows of
// 16 CH bytes has it.
template <int CH>
__device__ __forceinline__ int paged_swizzled(int r, int c) {
  return c ^ (CH == 8 ? r & 7 : CH == 4 ? (r >> 1) & 3 : (r >> 2) & 1);
}

template <int DP, int NB, int RW>
struct PagedPlan {
  static constexpr int kThreads = 32 * kPagedWarps;
  static constexpr int kKw = kPagedWarps / RW;  // groups of keys
  static constexpr int kRows = 8 * NB * RW;
  static constexpr int kTileBytes = kPagedKeys * DP;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = DP == 128 ? 3 : (DP == 64 ? 4 : 6);
  static constexpr int kResultStride = DP + 4;  // floats of a row: O, maximum, sum
  static constexpr int kResultBytes = kPagedWarps * 8 * NB * kResultStride * 4;
  static constexpr int kRingBytes = kKw * kStages * kStageBytes;
  static constexpr int kOffRows = kRingBytes > kResultBytes ? kRingBytes : kResultBytes;  // what each row sees
  static constexpr int kOffMeta = kOffRows + kRows * 16;  // [group][stage][2] scales of a step's boxes
  static constexpr int kOffBar = kOffMeta + kKw * kStages * 32;
  static constexpr int kSmemBytes = kOffBar + 16 * kKw * kStages + 32 + 1024;  // + alignment slack
};

// 8 x 8 16-bit elements, two neighbours of a row a lane, transposed.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// What a row sees: new tokens by the word's bits, others above lo or below sinks.
struct PagedRow {
  uint64_t word;  // 0: nothing
  int lo, sinks;
};

template <typename T, int DP, int NB, int RW>
__global__ void __launch_bounds__(PagedPlan<DP, NB, RW>::kThreads)
    vattn_paged_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ PagedParams p) {
  using P = PagedPlan<DP, NB, RW>;
  constexpr int CH = DP / 16;  // 16-byte chunks of a shared row, 16-element steps of a product
  constexpr int RS = P::kResultStride, S = P::kStages;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int kpos[VATTN_MAX_NEW_TOKENS];
  const uint32_t raw_s = ptx::smem_addr(smem_raw);
  const uint32_t smem_s = (raw_s + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (smem_s - raw_s);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rw = warp % RW, kw = warp / RW;
  const uint32_t bar0 = smem_s + P::kOffBar;
  auto full = [bar0, kw](int st) -> uint32_t { return bar0 + 8u * (kw * S + st); };
  auto empty = [bar0, kw](int st) -> uint32_t { return bar0 + 8u * ((P::kKw + kw) * S + st); };
  const Pipe pipe{bar0 + 16u * P::kKw * S};
  const WindowParams& w = p.w;
  const int D = w.dim;
  uint32_t split_u, rb_u, kh_u;
  const uint32_t bk = p.d_row_blocks.div(p.d_splits.div(blockIdx.x, &split_u), &rb_u);
  const int b = static_cast<int>(p.d_kv_heads.div(bk, &kh_u));
  const int split = static_cast<int>(split_u), rb = static_cast<int>(rb_u), kh = static_cast<int>(kh_u);
  const bool clustered = p.splits > 1 && p.splits <= kPagedCluster;

  if (tid == 0) {
    for (int i = 0; i < P::kKw * S; ++i) {
      ptx::mbar_init(bar0 + 8u * i, 1);
      ptx::mbar_init(bar0 + 8u * (P::kKw * S + i), RW);
    }
    pipe.init(w, p.status);
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_k);
    ptx::prefetch_tensormap(&tm_v);
  }
  ptx::grid_dep_wait();
  const PagedSpan sp = PagedSpan::make(w, p.log_box, P::kKw, b, p.splits);
  const int v0 = split * sp.per, v1 = min(sp.n, v0 + sp.per);
  const int shares = sp.shares();
  if (!clustered && split >= shares) return;  // (in a cluster: with no keys, but at its barriers)
  if (tid < w.n_queries) kpos[tid] = sp.base + __popcll(cached_word(w, b, tid, sp.base)) - 1;
  PagedRow* const rows = reinterpret_cast<PagedRow*>(smem + P::kOffRows);
  if (tid < P::kRows) {
    const int rr = rb * P::kRows + tid;
    PagedRow y{0, 0x7fffffff, 0};
    if (rr < p.rows) y.word = cached_word(w, b, static_cast<int>(p.d_group.div(static_cast<uint32_t>(rr))), sp.base);
    if (y.word != 0) {
      y.lo = sp.base + __popcll(y.word) - 1 - w.window;
      y.sinks = w.sinks;
    }
    rows[tid] = y;
  }
  __syncthreads();

  // ---- the group's steps: 32 keys each, as one box or two; its boxes numbered through
  const int log_boxes = 5 - p.log_box, boxes = 1 << log_boxes;
  static_assert(kPagedKeys == 32, "log_boxes");
  const int all_steps = (max(v1 - v0, 0) + boxes - 1) >> log_boxes;
  const int steps = (all_steps - kw + P::kKw - 1) / P::kKw;
  auto box_of = [&](int i) -> int { return v0 + ((((i >> log_boxes) * P::kKw + kw) << log_boxes) | (i & (boxes - 1))); };

  // ---- loads (the group's first warp): lane i has what box i of 32 needs, page, row
  // and scales, and of the 32 after (half way on: the scales too)
  struct Box {
    int page, row, key0;          // page: behind the last if it is not there, and reads as zeros
    float k, log2_v, inv_v;       // k < 0: the keys are not there
  };
  auto place = [&](int i, Box& x) {  // of the group's box i
    const int at = box_of(i);
    x.key0 = sp.box(at) << p.log_box;
    x.page = static_cast<int>(p.n_pages);
    uint32_t row = 0;
    if (at < v1) {
      const uint32_t lp = p.d_page.div(static_cast<uint32_t>(x.key0), &row);
      const int id = p.table[static_cast<long long>(b) * p.max_pages + lp];
      if (id >= 0 && id < p.n_pages) x.page = id;
    }
    x.row = static_cast<int>(row);
  };
  auto scales = [&](Box& x) {
    x.k = -1.0f;
    x.log2_v = x.inv_v = 0.0f;
    if (x.page >= p.n_pages) return;
    const long long at = static_cast<long long>(x.page) * w.kv_heads + kh;
    const float v = p.v_scale[at];
    x.k = p.k_scale[at];
    x.log2_v = log2f(v);
    x.inv_v = 1.0f / v;
  };
  int issued = 0, issue_st = 0;  // steps, and the next one's place in the ring
  Box now{}, next{};
  const uint64_t once = ptx::policy_evict_first();
  // The copies of a step's boxes, lanes l0 and l0 + 1 of `now`, to place st.
  auto copies = [&](int st, int l0) {
    const int pg = __shfl_sync(0xffffffffu, now.page, l0), row = __shfl_sync(0xffffffffu, now.row, l0);
    const uint32_t to = smem_s + static_cast<uint32_t>((kw * S + st) * P::kStageBytes);
    if (ptx::elect_one()) {
      ptx::tma_load_4d_hint(to, &tm_k, full(st), 0, row, kh, pg, once);
      ptx::tma_load_4d_hint(to + P::kTileBytes, &tm_v, full(st), 0, row, kh, pg, once);
    }
    if (log_boxes == 0) return;
    const int pg1 = __shfl_sync(0xffffffffu, now.page, l0 + 1), row1 = __shfl_sync(0xffffffffu, now.row, l0 + 1);
    if (ptx::elect_one()) {  // (of a box behind the share: zeros)
      ptx::tma_load_4d_hint(to + 16 * DP, &tm_k, full(st), 0, row1, kh, pg1, once);
      ptx::tma_load_4d_hint(to + P::kTileBytes + 16 * DP, &tm_v, full(st), 0, row1, kh, pg1, once);
    }
  };
  // What the products need beside them, and the barrier's count, which the copies may be ahead of.
  auto announce = [&](int st, int l0) {
    const int which = lane - l0;
    if (which >= 0 && which < boxes)
      ptx::st_shared_v4(smem_s + P::kOffMeta + static_cast<uint32_t>(((kw * S + st) * 2 + which) * 16), now.k, now.log2_v,
                        now.inv_v, __int_as_float(now.key0));
    __syncwarp();
    if (ptx::elect_one()) ptx::mbar_arrive_expect_tx(full(st), P::kStageBytes);
  };
  auto issue = [&]() {
    const int st = issue_st, i0 = issued << log_boxes, l0 = i0 & 31;
    issue_st = st + 1 == S ? 0 : st + 1;
    if (l0 == 0) {
      now = next;
      place(i0 + 32 + lane, next);
    } else if (l0 == 16) {
      scales(next);
    }
    announce(st, l0);
    copies(st, l0);
    ++issued;
  };
  if (rw == 0 && steps > 0) {
    place(lane, now);
    const int first = min(S, steps);  // S steps are 12 boxes at most
    for (int i = 0; i < first; ++i) copies(i, i << log_boxes);
    scales(now);
    place(32 + lane, next);
    for (int i = 0; i < first; ++i) announce(i, i << log_boxes);
    issued = first;
    issue_st = first == S ? 0 : first;
  }

  // ---- q as columns: lane / 4 of each eight rows, in the order of K's bytes
  const int g = lane >> 2, c4 = lane & 3;
  uint32_t qf[CH][NB][2];
  float row_c[NB][2];  // of rows 2 c4 and 2 c4 + 1: from a product's sum to log2 units, but for the key's scale
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int r = rw * 8 * NB + nb * 8 + g;
    uint32_t head;
    const int t = static_cast<int>(p.d_group.div(static_cast<uint32_t>(rb * P::kRows + r), &head));
    const T* qrow = rows[r].word != 0 ? rows_at<T>(p.q, b, kh * w.group + static_cast<int>(head), t) : nullptr;
    float y[CH][4];
    float most = 0.0f, c = p.scale_log2;
#pragma unroll
    for (int ks = 0; ks < CH; ++ks) {
      Vec<T, 4> x;
#pragma unroll
      for (int f = 0; f < 4; ++f) x.e[f] = Elem<T>::narrow(0.0f);
      if (qrow != nullptr && ks * 16 < D) x = *reinterpret_cast<const Vec<T, 4>*>(qrow + ks * 16 + c4 * 4);
      x.widen(y[ks]);
      if constexpr (Elem<T>::kBf16)
#pragma unroll
        for (int f = 0; f < 4; ++f) most = fmaxf(most, fabsf(y[ks][f]) < INFINITY ? fabsf(y[ks][f]) : 0.0f);
    }
    if constexpr (Elem<T>::kBf16) {
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
      // 2^k most in 2^14 .. 2^15 (of rows near either end of the range, as far as f32 goes)
      const int k = most == 0.0f ? 0 : min(max(14 + 127 - static_cast<int>(__float_as_uint(most) >> 23), -110), 110);
      const float by = __int_as_float((127 + k) << 23);
      c = p.scale_log2 * __int_as_float((127 - k) << 23);
#pragma unroll
      for (int ks = 0; ks < CH; ++ks)
#pragma unroll
        for (int f = 0; f < 4; ++f) y[ks][f] *= by;
    }
#pragma unroll
    for (int ks = 0; ks < CH; ++ks) {
      qf[ks][nb][0] = pack2<__half>(y[ks][0], y[ks][1]);
      qf[ks][nb][1] = pack2<__half>(y[ks][2], y[ks][3]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) row_c[nb][e] = __shfl_sync(0xffffffffu, c, 8 * c4 + 4 * e);
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
    const uint32_t ks_s = smem_s + static_cast<uint32_t>((kw * S + st) * P::kStageBytes);
    const uint32_t vs_s = ks_s + P::kTileBytes;
    // the step's keys by 16: first of each in the sequence, scales; those that are
    // not there, or that no row sees, count as masked throughout
    int j0[2];
    float4 meta[2];
    bool masked[2];
    const uint32_t meta_s = smem_s + P::kOffMeta + static_cast<uint32_t>((kw * S + st) * 32);
    meta[0] = ptx::ld_shared_v4(meta_s);
    meta[1] = ptx::ld_shared_v4(meta_s + (log_boxes << 4));
#pragma unroll
    for (int mb = 0; mb < 2; ++mb) {
      const int j = __float_as_int(meta[mb].w) + (mb == 1 && log_boxes == 0 ? 16 : 0);
      const bool on = !(meta[mb].x < 0.0f);
      j0[mb] = on ? j : 0x7fffff00;
      if (!on) meta[mb] = make_float4(1.0f, 0.0f, 1.0f, 0.0f);
      masked[mb] = !on || j + 15 >= free_end || (j < free_begin && j + 15 >= w.sinks);
    }
    const bool some = masked[0] || masked[1];
    // ---- S = K Q^T
    float s[2][NB][4];  // keys 16 mb + g, + 8 (e / 2) of rows 2 c4, + 1 (e % 2)
#pragma unroll
    for (int mb = 0; mb < 2; ++mb)
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[mb][nb][e] = 0.0f;
#pragma unroll
    for (int ks = 0; ks < CH; ++ks) {
      // matrices: keys 0-7, 8-15, 16-23, 24-31 by the 16 dims of chunk ks
      uint32_t kf[4];
      ldmatrix_x4(ks_s + static_cast<uint32_t>(lane * DP + (paged_swizzled<CH>(lane, ks) << 4)), kf);
#pragma unroll
      for (int mb = 0; mb < 2; ++mb) {
        const uint32_t a[4] = {e4m3_half2_lo(kf[2 * mb]), e4m3_half2_lo(kf[2 * mb + 1]), e4m3_half2_hi(kf[2 * mb]),
                               e4m3_half2_hi(kf[2 * mb + 1])};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) mma_16816<__half>(s[mb][nb], a, qf[ks][nb][0], qf[ks][nb][1]);
      }
    }
    // ---- masks: at the sequence's end, the first keys' end, the window's edge, among the new tokens
    auto sees = [&](int r, int j) {
      const PagedRow y = rows[r];
      const int u = j - sp.base;
      const int at = u >= 0 && j < sp.len ? kpos[u] : j;
      return j < sp.len && (u < 0 || ((y.word >> u) & 1)) && (at > y.lo || at < y.sinks);
    };
    const int r0 = rw * 8 * NB + 2 * c4;
    if (some) {
#pragma unroll
      for (int mb = 0; mb < 2; ++mb) {
        if (!masked[mb]) continue;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!sees(r0 + nb * 8 + (e & 1), j0[mb] + g + 8 * (e >> 1))) s[mb][nb][e] = -INFINITY;
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
          c[mb][nb][e] = fminf(fmaxf(row_c[nb][e] * meta[mb].x, 0x1p-126f), 0x1p127f);
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
    bool loops = false;
    if (some) {
      // rows that no query sees may hold anything: zeros; a NaN in another that
      // some do not see: loops over the visible pairs
      bool bad = false;
#pragma unroll
      for (int y = lane; y < kPagedKeys * CH; y += 32) {
        const int r = y / CH, c = y % CH, mb = r >> 4, j = (mb ? j0[1] : j0[0]) + (r & 15);
        if (!(mb ? masked[1] : masked[0])) continue;
        const uint32_t at = vs_s + static_cast<uint32_t>(r * DP + (paged_swizzled<CH>(r, c) << 4));
        if (j >= sp.len || (j < sp.first && j >= w.sinks)) {
          ptx::st_shared_v4(at, 0.0f, 0.0f, 0.0f, 0.0f);
          continue;
        }
        const float4 z = ptx::ld_shared_v4(at);
        const uint32_t zs[4] = {__float_as_uint(z.x), __float_as_uint(z.y), __float_as_uint(z.z), __float_as_uint(z.w)};
#pragma unroll
        for (int f = 0; f < 4; ++f)  // a byte's low seven bits all ones: a carry out of them
          bad |= (((zs[f] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
      }
      ptx::fence_proxy_async_smem();  // before the ring's next copy there
      loops = __any_sync(0xffffffffu, bad);
      __syncwarp();
    }
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
        // matrices: keys 0-7, 8-15, 16-23, 24-31 by the 16 dims of chunk n, transposed by pairs of dims
        uint32_t vf[4];
        ldmatrix_x4_trans(vs_s + static_cast<uint32_t>(lane * DP + (paged_swizzled<CH>(lane, n) << 4)), vf);
#pragma unroll
        for (int y = 0; y < 4; ++y) vf[y] = __byte_perm(vf[y], 0u, 0x3120);
#pragma unroll
        for (int mb = 0; mb < 2; ++mb) {
          const uint32_t a[4] = {e4m3_half2_lo(vf[2 * mb]), e4m3_half2_hi(vf[2 * mb]), e4m3_half2_lo(vf[2 * mb + 1]),
                                 e4m3_half2_hi(vf[2 * mb + 1])};
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) mma_16816<__half>(o[n][nb], a, pf[mb][nb][0], pf[mb][nb][1]);
        }
      }
    } else {
#pragma unroll
      for (int mb = 0; mb < 2; ++mb)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!sees(r0 + nb * 8 + (e & 1), j0[mb] + g + 8 * (e >> 1))) s[mb][nb][e] = -1.0f;
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
            const uint32_t z = *reinterpret_cast<const uint16_t*>(smem + (vs_s - smem_s) + r * DP +
                                                                  (paged_swizzled<CH>(r, n) << 4) + g * 2);
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
    if (RW > 1) pipe_warp_arrive(empty(st));
    else __syncwarp();
    if (rw == 0 && issued < steps) {
      if (RW > 1 && !pipe.wait_warp(empty(st), turn, kSitePagedLoad)) {
        ++step;
        break;
      }
      issue();
    }
    if (++st == S) {
      st = 0;
      turn ^= 1;
    }
  }
  if (rw == 0 && lane == 0)  // after a wait that ran out: the copies in flight land before the block exits
    for (; step < issued; ++step) pipe.drain(full(step % S), static_cast<uint32_t>((step / S) & 1), kSitePagedDrain);
  __syncthreads();  // the rings are free: the warps' results go there

  // ---- join the warps that shared the keys
  float* res = reinterpret_cast<float*>(smem);  // [group of keys][kRows][RS]
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
  __syncthreads();
  auto write = [&](int rr, int d, float sum, float (&acc)[8]) {
    uint32_t head;
    const int t = static_cast<int>(p.d_group.div(static_cast<uint32_t>(rr), &head));
    const bool none = sum == 0.0f || cached_word(w, b, t, sp.base) == 0;
    const float inv = 1.0f / sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = none ? 0.0f : acc[e] * inv;
    reinterpret_cast<Vec<T, 8>*>(rows_at_mut<T>(p.out, b, kh * w.group + static_cast<int>(head), t) + d)->narrow(acc);
  };
  const bool alone = p.splits == 1 || (shares == 1 && !clustered);
  const int per_row = D / 8;
  for (int x = tid; x < P::kRows * per_row; x += P::kThreads) {
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
  __syncthreads();
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
  for (int x = split * P::kThreads + tid; x < P::kRows * per_row; x += p.splits * P::kThreads) {
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
  const PagedSpan sp = PagedSpan::make(w, p.log_box, KW, b, p.splits);
  const int shares = sp.shares();
  if (shares == 1) return;  // written by its block
  const bool none = cached_word(w, b, t, sp.base) == 0;
  const long long at0 = (bk * p.row_blocks + rr / ROWS) * p.splits * ROWS + rr % ROWS;
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + at0;
  static_assert(kCachedMaxSplits <= 512, "two shares a thread");
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
  if (d < D) {
    const float* from = p.part_o + at0 * D + d;
#pragma unroll 4
    for (int s = warp * 4 + (lane >> 3); s < shares; s += 32) {
      const float4 y = *reinterpret_cast<const float4*>(from + s * static_cast<long long>(ROWS) * D);
      const float a = weight[s];
      acc.x = fmaf(a, y.x, acc.x);
      acc.y = fmaf(a, y.y, acc.y);
      acc.z = fmaf(a, y.z, acc.z);
      acc.w = fmaf(a, y.w, acc.w);
    }
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
  const float out[4] = {zero ? 0.0f : acc.x * inv, zero ? 0.0f : acc.y * inv, zero ? 0.0f : acc.z * inv, zero ? 0.0f : acc.w * inv};
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
  const PagedSpan sp = PagedSpan::make(w, p.log_box, KW, b, p.splits);
  const int shares = sp.shares();
  if (shares == 1) return;  // written by its block
  const bool none = cached_word(w, b, t, sp.base) == 0;
  const long long at0 = (bk * p.row_blocks + rr / ROWS) * p.splits * ROWS + rr % ROWS;
  const float2 ml = lane < shares ? reinterpret_cast<const float2*>(p.part_ml)[at0 + lane * static_cast<long long>(ROWS)]
                                  : make_float2(-INFINITY, 0.0f);
  const float mx = warp_max(ml.x), ref = mx == -INFINITY ? 0.0f : mx;
  const float weight = ptx::ex2_approx(ml.x - ref);
  float sum = weight * ml.y;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float* from = p.part_o + at0 * D + (lane * 4 < D ? lane * 4 : 0);
#pragma unroll 8
  for (int s = 0; s < shares; ++s) {
    const float4 y = *reinterpret_cast<const float4*>(from + s * static_cast<long long>(ROWS) * D);
    const float a = __shfl_sync(0xffffffffu, weight, s);
    acc.x = fmaf(a, y.x, acc.x);
    acc.y = fmaf(a, y.y, acc.y);
    acc.z = fmaf(a, y.z, acc.z);
    acc.w = fmaf(a, y.w, acc.w);
  }
  if (lane * 4 >= D) return;
  const float inv = 1.0f / sum;
  const bool zero = none || sum == 0.0f;
  const float out[4] = {zero ? 0.0f : acc.x * inv, zero ? 0.0f : acc.y * inv, zero ? 0.0f : acc.z * inv, zero ? 0.0f : acc.w * inv};
  reinterpret_cast<Vec<T, 4>*>(rows_at_mut<T>(p.out, b, kh * w.group + (rr - t * w.group), t) + lane * 4)->narrow(out);
}

}  // namespace vattn
