// paged_append_kernel.cuh -- new keys and values into the 8-bit paged cache
// (vattn_append_paged).
//
// A block has one page of one sequence, for one head of k or of v: the scale
// of a page and head belongs to one block, which no other waits for.  It takes
// the largest finite magnitude of its new rows (keys turned by their angle
// first, in f32), the scale from that and from the old one, rescales the rows
// before the new ones where the scale grew, and rounds the new rows to e4m3.
// With scales that are powers of two, rescaling moves exponents only: what was
// rounded once stays as it is but for values that leave the normal range.
//
// A thread holds slots of 2 x 8 elements of a row, a rotation pair each, in
// registers between the two steps; what it has beyond kAppendHold of them it
// reads again.
#pragma once

#include "e4m3.cuh"
#include "ptx.cuh"
#include "rope_rows.cuh"
#include "window_common.cuh"

namespace vattn {

constexpr int kAppendThreads = 512;  // most
constexpr int kAppendHold = 4;       // slots a thread holds
constexpr int kMinScaleExponent = -32;

struct AppendParams {
  RowsTensor x[2];           // k, v
  uint8_t* pool[2];
  long long ps[2][3];        // page, head, row
  float* scale[2];
  const int32_t* table;
  const int32_t* kv_len;
  const int32_t* cu;         // or null: n_tokens rows of each sequence
  const int32_t* positions;
  const float* factors;
  long long n_pages;
  int batch, heads, n_tokens;
  int page, max_pages;
  int D, half, slots;        // slots of a row
  int items;                 // uniform: pages that a sequence's new rows may touch
  FastDiv d_heads, d_items, d_page, d_slots;
  double turns[kQkMaxDim / 2];
  float turns_rest[kQkMaxDim / 2];
};

// A sequence's new rows in x: [first, first + n) of it (packed), and how many pages.
struct AppendSeq {
  int b, first, n, nth;  // nth of the sequence's touched pages
};

// Packed: sequence b's pages are the items from cu[b] / page + 2 b on, which leaves
// room for all that its rows can touch, wherever the first of them is in its page.
__device__ __forceinline__ AppendSeq append_seq(const AppendParams& p, int item) {
  AppendSeq s;
  if (p.cu == nullptr) {
    uint32_t nth;
    s.b = static_cast<int>(p.d_items.div(static_cast<uint32_t>(item), &nth));
    s.nth = static_cast<int>(nth);
    s.first = 0;
    s.n = p.n_tokens;
    return s;
  }
  auto at = [&](int b) { return min(max(p.cu[b], 0), p.n_tokens); };
  auto begin = [&](int b) { return static_cast<int>(p.d_page.div(static_cast<uint32_t>(at(b)))) + 2 * b; };
  int lo = 0, hi = p.batch;  // begin(lo) <= item < begin(hi)
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (begin(mid) <= item) lo = mid;
    else hi = mid;
  }
  s.b = lo;
  s.first = at(lo);
  s.n = max(0, at(lo + 1) - s.first);
  s.nth = item - begin(lo);
  return s;
}

template <typename T, int V>
__global__ void __launch_bounds__(kAppendThreads) vattn_append_paged_kernel(const __grid_constant__ AppendParams p) {
  __shared__ uint64_t turn[kQkMaxDim / 2];
  __shared__ float top_s[kAppendThreads / 32];
  ptx::grid_dep_wait();
  const int tid = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x);
  uint32_t head;
  const uint32_t rest = p.d_heads.div(blockIdx.x, &head);
  const int which = static_cast<int>(rest & 1u), h = static_cast<int>(head);
  const AppendSeq s = append_seq(p, static_cast<int>(rest >> 1));
  // new rows of the sequence's cache, and those of this page: [lo, hi)
  const int limit = p.max_pages * p.page;
  const int len = min(max(p.kv_len[s.b], 0), limit);
  const long long start = static_cast<long long>(p.kv_len[s.b]) - s.n;  // row of the first new token
  const int begin = static_cast<int>(min(static_cast<long long>(limit), max(0LL, start)));
  const int lp = static_cast<int>(p.d_page.div(static_cast<uint32_t>(begin))) + s.nth;
  if (s.n <= 0 || s.nth < 0 || lp >= p.max_pages || static_cast<long long>(lp) * p.page >= len) return;
  const int row0 = lp * p.page, lo = max(begin, row0), hi = min(len, row0 + p.page);
  if (hi <= lo) return;
  const long long P = p.table[static_cast<long long>(s.b) * p.max_pages + lp];
  if (P < 0 || P >= p.n_pages) return;
  const bool keys = which == 0;
  const int half = keys ? p.half : 0;
  if (keys) {
    for (int i = tid; i < half; i += threads) turn[i] = qk_turn(p.turns, p.turns_rest, p.factors, i);
    __syncthreads();
  }
  const RowsTensor& x = keys ? p.x[0] : p.x[1];
  uint8_t* const page = (keys ? p.pool[0] : p.pool[1]) + P * p.ps[which][0] + h * p.ps[which][1];
  const long long row_stride = p.ps[which][2];
  float* const scale_at = (keys ? p.scale[0] : p.scale[1]) + P * p.heads + h;

  // the f32 values of slot `at` of the new rows
  const int all = (hi - lo) * p.slots;
  struct Slot {
    QkSlot<V> s;
    int row;
  };
  auto slot = [&](int at) {
    Slot t;
    uint32_t c;
    t.row = lo + static_cast<int>(p.d_slots.div(static_cast<uint32_t>(at), &c));
    t.s.set(p.D, half, p.slots, static_cast<int>(c));
    return t;
  };
  auto values = [&](int at, float (&a)[V], float (&b)[V]) {
    const Slot t = slot(at);
    const long long i = s.first + (t.row - start);
    const T* from = p.cu != nullptr ? rows_at<T>(x, 0, h, i) : rows_at<T>(x, s.b, h, i);
    qk_load<T, V>(from, t.s.ia, t.s.here).widen(a);
    qk_load<T, V>(from, t.s.ib, t.s.pair).widen(b);
    if (t.s.rot) {
      const long long pos =
          p.positions == nullptr ? t.row : p.positions[(p.cu != nullptr ? 0LL : static_cast<long long>(s.b) * p.n_tokens) + i];
      float cs[V], sn[V];
      uint32_t c;
      (void)p.d_slots.div(static_cast<uint32_t>(at), &c);
      qk_angles<V>(t.s, turn, static_cast<int>(c), pos, cs, sn);
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const float ya = fmaf(-b[e], sn[e], a[e] * cs[e]), yb = fmaf(a[e], sn[e], b[e] * cs[e]);
        a[e] = ya;
        b[e] = yb;
      }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {  // infinities become NaN
      a[e] = fmaf(a[e], 0.0f, a[e]);
      b[e] = fmaf(b[e], 0.0f, b[e]);
    }
  };
  auto largest = [](float m, const float (&a)[V], const float (&b)[V]) {
#pragma unroll
    for (int e = 0; e < V; ++e) m = fmaxf(m, fmaxf(fabsf(a[e]), fabsf(b[e])));  // (NaN is left out)
    return m;
  };

  const float old = *scale_at;
  float ha[kAppendHold][V], hb[kAppendHold][V], top = 0.0f;
#pragma unroll
  for (int n = 0; n < kAppendHold; ++n)
    if (tid + n * threads < all) {
      values(tid + n * threads, ha[n], hb[n]);
      top = largest(top, ha[n], hb[n]);
    }
#pragma unroll 1
  for (int at = tid + kAppendHold * threads; at < all; at += threads) {
    float a[V], b[V];
    values(at, a, b);
    top = largest(top, a, b);
  }
  top = warp_max(top);
  if (threads > 32) {
    if ((tid & 31) == 0) top_s[tid >> 5] = top;
    __syncthreads();
    for (int w = 0; w < threads / 32; ++w) top = fmaxf(top, top_s[w]);
  }
  const float need = __int_as_float((max(e4m3_scale_exponent(top), kMinScaleExponent) + 127) << 23);
  const float scale = lo == row0 ? need : fmaxf(old, need);
  if (threads > 32) __syncthreads();  // every thread has read the old scale
  else __syncwarp();
  if (tid == 0) *scale_at = scale;

  // the rows before the new ones, 16 bytes at a time
  if (lo > row0 && scale != old) {
    const float by = old / scale;
    const int chunks = p.D / 16;
    for (int at = tid; at < (lo - row0) * chunks; at += threads) {
      const int r = at / chunks;
      uint4* to = reinterpret_cast<uint4*>(page + r * row_stride + (at - r * chunks) * 16);
      uint4 y = *to;
      uint32_t* w = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t lo2 = e4m3_half2_lo(w[i]), hi2 = e4m3_half2_hi(w[i]);
        const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo2));
        const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi2));
        w[i] = e4m3_pack4(a.x * by, a.y * by, b.x * by, b.y * by);
      }
      *to = y;
    }
  }
  const float by = 1.0f / scale;
  auto store = [&](int at, const float (&a)[V], const float (&b)[V]) {
    const Slot t = slot(at);
    uint8_t* to = page + (t.row - row0) * row_stride;
    if constexpr (V == 8) {
      *reinterpret_cast<uint2*>(to + t.s.ia) = make_uint2(e4m3_pack4(a[0] * by, a[1] * by, a[2] * by, a[3] * by),
                                                          e4m3_pack4(a[4] * by, a[5] * by, a[6] * by, a[7] * by));
      *reinterpret_cast<uint2*>(to + t.s.ib) = make_uint2(e4m3_pack4(b[0] * by, b[1] * by, b[2] * by, b[3] * by),
                                                          e4m3_pack4(b[4] * by, b[5] * by, b[6] * by, b[7] * by));
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        const uint32_t y = e4m3_pack(a[e] * by, b[e] * by);
        to[t.s.ia + e] = static_cast<uint8_t>(y);
        to[t.s.ib + e] = static_cast<uint8_t>(y >> 8);
      }
    }
  };
#pragma unroll
  for (int n = 0; n < kAppendHold; ++n)
    if (tid + n * threads < all) store(tid + n * threads, ha[n], hb[n]);
#pragma unroll 1
  for (int at = tid + kAppendHold * threads; at < all; at += threads) {
    float a[V], b[V];
    values(at, a, b);
    store(at, a, b);
  }
}

}  // namespace vattn
