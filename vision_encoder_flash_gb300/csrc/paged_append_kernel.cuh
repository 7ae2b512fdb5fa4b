// paged_append_kernel.cuh -- new keys and values into the 8-bit paged cache
// (vattn_append_paged).
//
// A page and head of k or of v is a unit, whose scale belongs to one block, which no
// other waits for; a block has consecutive ones, all heads of a page behind each
// other.  For each it takes the largest finite magnitude of the new rows (keys turned by
// their angle first, in f32), the scale from that and from the old one, rescales the
// rows before the new ones where the scale grew, and rounds the new rows to e4m3.  With
// scales that are powers of two, rescaling moves exponents only: what was rounded
// once stays as it is but for values that leave the normal range.
//
// A thread holds slots of 2 x 8 elements of a row, a rotation pair each, in
// registers between the two steps (what it has beyond kAppendHold of them it reads
// again), and the next heads' come through a cp.async ring of its own in shared
// memory.  The angles' sines and cosines serve all heads of the page, likewise from
// shared memory that only their thread uses.
//
// 6 prompts of 16384 tokens together, 8 heads x 128 bf16, pages of 64: 23.1 us, 4.4
// TB/s (65 % of the measured copy rate; 49.3 us with a block for each unit and its own
// angles; 25.9 with a block for a page, in two rounds).  Without the rotation 21.1: the
// bound is latency, of some 300 instructions a head at 5 cycles each, twice a barrier
// and the block's start, with 24 warps a multiprocessor.  Two slots a thread and 256
// threads for a page of 64: with four 35 us, with one 37.  Pages of 128 26.2 us (blocks
// of 512 threads, alone on their multiprocessor), of 256 42.2 (what the threads do not
// hold is read and turned twice, its angles kept as far as twice the held slots; with
// angles of the held slots only 56, parted over a cluster that joins its maxima head by
// head 61).  8 heads x 1 token: 3.5 us.
//
// V, elements of a slot's halves: 8, or 4 where the rotated dims or the strides do not
// divide into 16 bytes (80 dims of which 40 are rotated), or 1, which reads all of
// its rows twice.
#pragma once

#include "e4m3.cuh"
#include "ptx.cuh"
#include "rope_rows.cuh"
#include "window_common.cuh"

namespace vattn {

// A page's new rows: all held by up to 256 threads, of which three blocks are resident,
// or by up to 512, or more than those can hold.
enum AppendForm : int { kAppendHeld256 = 0, kAppendHeld = 1, kAppendMore = 2 };
constexpr int kAppendThreads = 512;  // most
constexpr int kAppendFewThreads = 256;
constexpr int kAppendStages = 2;         // heads in its ring
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
  int units, per_block;      // pages times heads, of k and of v; consecutive ones a block
  FastDiv d_heads, d_items, d_page, d_slots;
  uint64_t turn[kQkMaxDim / 2];  // without factors: each frequency's fraction of a turn (qk_turn)
  double turns[kQkMaxDim / 2];   // with them: what qk_turn wants
  float turns_rest[kQkMaxDim / 2];
};

// A sequence's new rows in x: [first, first + n) of it (packed), rows of its cache in
// use, and which of the pages that it touches.
struct AppendSeq {
  int b, first, n, nth, kv_len;
};

// Row b of the starts, held to the rows that there are.
__device__ __forceinline__ int append_start(const AppendParams& p, int b) { return min(max(p.cu[b], 0), p.n_tokens); }

// Do the starts ascend?  Up to 32 each warp looks at by itself, more the block's threads
// together, with many loads in flight; in L1 they serve the searches that follow.  (The
// vote at the end tells the compiler that a warp's lanes agree.)  200 prompts of 8 tokens
// 17.2 us, 16.9 without; 1000 of 4 of two heads 10.7 and 9.1; 4096 of one 49 and 40.
__device__ __forceinline__ bool append_ascends(const AppendParams& p) {
  constexpr int kAhead = 16;
  const int tid = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x), lane = tid & 31;
  if (p.batch <= 32) return __all_sync(0xffffffffu, lane >= p.batch || p.cu[lane] <= p.cu[lane + 1]);
  bool yes = tid >= p.batch || p.cu[tid] <= p.cu[tid + 1];
#pragma unroll 1
  for (int b0 = tid + threads; b0 < p.batch; b0 += kAhead * threads) {
    int x[kAhead], y[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int b = b0 + i * threads;
      x[i] = b < p.batch ? p.cu[b] : 0;
      y[i] = b < p.batch ? p.cu[b + 1] : 0;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) yes &= x[i] <= y[i];
  }
  return __all_sync(0xffffffffu, __syncthreads_and(yes) != 0);
}

// Where they do not, item `item` by a look at every sequence: as if their rows, of which
// there are n, followed each other.  None if they are more than there are together.
static __device__ __noinline__ AppendSeq append_seq_any(const AppendParams& p, int item) {
  const int lane = static_cast<int>(threadIdx.x) & 31;
  AppendSeq s{0, 0, 0, 0, 0};
  uint32_t before = 0;  // rows of the sequences before these 32, at most 2^30
  constexpr uint32_t kMany = 1u << 30;
#pragma unroll 1
  for (int b0 = 0; b0 < p.batch; b0 += 32) {
    const int b = b0 + lane;
    const int first = b < p.batch ? append_start(p, b) : 0;
    const int n = b < p.batch ? max(0, append_start(p, b + 1) - first) : 0;
    uint32_t upto = static_cast<uint32_t>(n);
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto = min(upto + y, kMany);
    }
    const uint32_t row = min(before + upto, kMany) - static_cast<uint32_t>(n);  // (as long as it matters)
    const int begin = static_cast<int>(p.d_page.div(min(row, kMany))) + 2 * b;
    const uint32_t here = __ballot_sync(0xffffffffu, b < p.batch && begin <= item);
    if (here != 0) {
      const int k = 31 - __clz(static_cast<int>(here));
      s.b = b0 + k;
      s.first = __shfl_sync(0xffffffffu, first, k);
      s.n = __shfl_sync(0xffffffffu, n, k);
      s.nth = item - __shfl_sync(0xffffffffu, begin, k);
    }
    before = min(before + __shfl_sync(0xffffffffu, upto, 31), kMany);
  }
  if (before > static_cast<uint32_t>(p.n_tokens)) s.n = 0;
  s.kv_len = p.kv_len[s.b];
  return s;
}

// Packed: sequence b's pages are the items from cu[b] / page + 2 b on, which leaves
// room for all that its rows can touch, wherever the first of them is in its page.
// A warp looks at 32 sequences at a time, so that few loads wait for one another.
__device__ __forceinline__ AppendSeq append_seq(const AppendParams& p, int item, bool ascends) {
  AppendSeq s;
  if (p.cu == nullptr) {
    uint32_t nth;
    s.b = static_cast<int>(p.d_items.div(static_cast<uint32_t>(item), &nth));
    s.nth = static_cast<int>(nth);
    s.first = 0;
    s.n = p.n_tokens;
    s.kv_len = p.kv_len[s.b];
    return s;
  }
  if (!ascends) return append_seq_any(p, item);
  const int lane = static_cast<int>(threadIdx.x) & 31;
  auto begin = [&](int b, int row) { return static_cast<int>(p.d_page.div(static_cast<uint32_t>(row))) + 2 * b; };
  auto last = [](bool yes) { return max(0, 31 - __clz(static_cast<int>(__ballot_sync(0xffffffffu, yes)))); };
  int lo = 0, n = p.batch;  // begin(lo) <= item < begin(lo + n)
  while (n > 32) {
    const int step = (n + 31) / 32, b = lo + lane * step;
    const int k = last(lane * step < n && begin(b, append_start(p, b)) <= item) * step;
    lo += k;
    n = min(step, n - k);
  }
  const int b = lo + min(lane, n - 1);
  const int row = append_start(p, b), end = append_start(p, b + 1), len = p.kv_len[b];
  const int k = last(lane < n && begin(b, row) <= item);
  s.b = lo + k;
  s.first = __shfl_sync(0xffffffffu, row, k);
  s.n = max(0, __shfl_sync(0xffffffffu, end, k) - s.first);
  s.nth = item - begin(s.b, s.first);
  s.kv_len = __shfl_sync(0xffffffffu, len, k);
  return s;
}

// Slots that a thread holds.
template <int V>
constexpr int kAppendHold = V >= 4 ? 16 / V : 0;

// Slots of a thread whose angles it keeps, where it cannot hold all of their values too.
template <int V, int kForm>
constexpr int kAppendAngles = kForm == kAppendMore ? 2 * kAppendHold<V> : kAppendHold<V>;

// Shared memory of a block: V (cos, sin) of these, and the held slots' rows.
template <int V, int kForm>
constexpr int append_smem(int threads) {
  return threads * (kAppendAngles<V, kForm> * 8 * V + kAppendHold<V> * kAppendStages * 4 * V);
}

// V elements of 16 bits.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> append_shared(uint32_t addr) {
  if constexpr (V == 8) {
    const float4 y = ptx::ld_shared_v4(addr);
    return *reinterpret_cast<const Vec<T, V>*>(&y);
  } else {
    const float2 y = ptx::ld_shared_v2(addr);
    return *reinterpret_cast<const Vec<T, V>*>(&y);
  }
}

template <typename T, int V, int kForm>
__global__ void __launch_bounds__(kForm == kAppendHeld256 ? kAppendFewThreads : kAppendThreads,
                                  kForm == kAppendHeld256 ? 3 : 1)
    vattn_append_paged_kernel(const __grid_constant__ AppendParams p) {
  extern __shared__ float4 angle_s[];  // [V / 2][slot][thread]: cosines, then sines; then the rings
  __shared__ uint64_t turn[kQkMaxDim / 2];
  __shared__ __align__(16) float top_s[2][kAppendThreads / 32];
  constexpr int kHold = kAppendHold<V>, kAngles = kAppendAngles<V, kForm>;
  constexpr bool kHeld = kForm != kAppendMore;
  ptx::grid_dep_wait();
  const int tid = static_cast<int>(threadIdx.x), threads = static_cast<int>(blockDim.x);
  if (tid < kAppendThreads / 16) top_s[tid & 1][tid >> 1] = 0.0f;
  for (int i = tid; i < p.half; i += threads)
    turn[i] = p.factors == nullptr ? p.turn[i] : qk_turn(p.turns, p.turns_rest, p.factors, i);
  const bool ascends = p.cu == nullptr || append_ascends(p);
  __syncthreads();
  uint32_t parity = 0;  // of the heads so far
  int unit = static_cast<int>(blockIdx.x) * p.per_block;
  const int last_unit = min(p.units, unit + p.per_block);
#pragma unroll 1
  while (unit < last_unit) {
    uint32_t h_first;
    const uint32_t rest = p.d_heads.div(static_cast<uint32_t>(unit), &h_first);
    const int which = static_cast<int>(rest & 1u), h0 = static_cast<int>(h_first);
    const int h1 = min(p.heads, h0 + last_unit - unit);
    unit += h1 - h0;
    const AppendSeq s = append_seq(p, static_cast<int>(rest >> 1), ascends);
    // new rows of the sequence's cache, and those of this page: [lo, hi)
    const int limit = p.max_pages * p.page;
    const int len = min(max(s.kv_len, 0), limit);
    const long long start = static_cast<long long>(s.kv_len) - s.n;  // row of the first new token
    const int begin = static_cast<int>(min(static_cast<long long>(limit), max(0LL, start)));
    const int lp = static_cast<int>(p.d_page.div(static_cast<uint32_t>(begin))) + s.nth;
    if (s.n <= 0 || s.nth < 0 || lp >= p.max_pages || static_cast<long long>(lp) * p.page >= len) continue;
    const int row0 = lp * p.page, lo = max(begin, row0), hi = min(len, row0 + p.page);
    if (hi <= lo) continue;
    const long long P = p.table[static_cast<long long>(s.b) * p.max_pages + lp];
    if (P < 0 || P >= p.n_pages) continue;
    const bool keys = which == 0;
    const int half = keys ? p.half : 0;
    const RowsTensor& x = keys ? p.x[0] : p.x[1];
    uint8_t* const pool = (keys ? p.pool[0] : p.pool[1]) + P * p.ps[which][0];
    const long long head_stride = p.ps[which][1], row_stride = p.ps[which][2];
    float* const scales = (keys ? p.scale[0] : p.scale[1]) + P * p.heads;
    const T* const first_row = p.cu != nullptr ? rows_at<T>(x, 0, 0, s.first - start) : rows_at<T>(x, s.b, 0, -start);  // + row: its place

    // slot `at` of the new rows: row, place in it, and where it is in head 0
    const int all = (hi - lo) * p.slots;
    struct Slot {
      QkSlot<V> s;
      int row, c;
    };
    auto slot = [&](int at) {
      Slot t;
      uint32_t c;
      t.row = lo + static_cast<int>(p.d_slots.div(static_cast<uint32_t>(at), &c));
      t.c = static_cast<int>(c);
      t.s.set(p.D, half, p.slots, t.c);
      return t;
    };
    auto position = [&](int row) -> long long {
      if (p.positions == nullptr) return row;
      return p.positions[(p.cu != nullptr ? 0LL : static_cast<long long>(s.b) * p.n_tokens) + s.first + (row - start)];
    };
    auto rotate = [](float (&a)[V], float (&b)[V], const float (&cs)[V], const float (&sn)[V]) {
      float x[V], y[V], minus[V];
      vmul<V>(x, a, cs);
      vmul<V>(y, a, sn);
#pragma unroll
      for (int e = 0; e < V; ++e) minus[e] = -b[e];
      vfma<V>(a, minus, sn, x);
      vfma<V>(b, b, cs, y);
    };
    auto angles = [&](int n, float (&cs)[V], float (&sn)[V]) {  // of the thread's slot n
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        const float4 y = angle_s[(k * kAngles + n) * threads + tid], z = angle_s[((k + V / 4) * kAngles + n) * threads + tid];
        cs[4 * k] = y.x;
        cs[4 * k + 1] = y.y;
        cs[4 * k + 2] = y.z;
        cs[4 * k + 3] = y.w;
        sn[4 * k] = z.x;
        sn[4 * k + 1] = z.y;
        sn[4 * k + 2] = z.z;
        sn[4 * k + 3] = z.w;
      }
    };
    // the f32 values of a slot that no thread holds, the thread's n-th
    auto values = [&](const Slot& t, int n, int h, float (&a)[V], float (&b)[V]) {
      const T* from = first_row + t.row * x.s[2] + h * x.s[1];
      qk_load<T, V>(from, t.s.ia, t.s.here).widen(a);
      qk_load<T, V>(from, t.s.ib, t.s.pair).widen(b);
      if (!t.s.rot) return;
      float cs[V], sn[V];
      if (n < kAngles) angles(n, cs, sn);
      else qk_angles<V>(t.s, turn, t.c, position(t.row), cs, sn);
      rotate(a, b, cs, sn);
    };
    auto largest = [](float m, const float (&a)[V], const float (&b)[V]) {  // (NaN is left out)
#pragma unroll
      for (int e = 0; e < V; ++e) m = ptx::max3(m, fabsf(a[e]), fabsf(b[e]));
      return m;
    };
    auto largest_finite = [](float m, const float (&a)[V], const float (&b)[V]) {
#pragma unroll
      for (int e = 0; e < V; ++e) {
        if (fabsf(a[e]) < INFINITY) m = fmaxf(m, fabsf(a[e]));
        if (fabsf(b[e]) < INFINITY) m = fmaxf(m, fabsf(b[e]));
      }
      return m;
    };

    // ---- the first heads' rows on their way, then the angles
    const T* from[kHold + 1];
    long long to[kHold + 1];  // place in the page, from the head's first byte
    int apart[kHold + 1];     // elements from a slot's first half to its second
    bool rot[kHold + 1], on[kHold + 1];
    const uint32_t ring = ptx::smem_addr(angle_s) + static_cast<uint32_t>(threads * kAngles * 8 * V + tid * 2 * V);
    // a head's rows: ring[stage][slot][a, b]
    auto ask = [&](int h) {
      if (h < h1) {
#pragma unroll
        for (int n = 0; n < kHold; ++n) {
          const uint32_t at = ring + static_cast<uint32_t>((((h - h0) % kAppendStages * kHold + n) * 2) * threads * 2 * V);
          ptx::cp_async<V == 8 ? 16 : 8>(at, from[n], on[n]);
          ptx::cp_async<V == 8 ? 16 : 8>(at + threads * 2 * V, from[n] + apart[n], on[n]);
          from[n] += x.s[1];
        }
      }
      ptx::cp_async_commit();
    };
    if constexpr (kHold > 0) {
#pragma unroll
      for (int n = 0; n < kHold; ++n) {
        on[n] = tid + n * threads < all;
        const Slot t = slot(on[n] ? tid + n * threads : 0);
        from[n] = first_row + t.row * x.s[2] + h0 * x.s[1] + t.s.ia;
        to[n] = (t.row - row0) * row_stride + t.s.ia;
        apart[n] = t.s.ib - t.s.ia;
        rot[n] = t.s.rot;
      }
      for (int i = 0; i < kAppendStages; ++i) ask(h0 + i);
    }
    if (half > 0) {
      if constexpr (kHold > 0) {
#pragma unroll 1
        for (int n = 0; n < kAngles; ++n) {
          if (!kHeld && n * threads >= all) break;
          const Slot t = slot(min(tid + n * threads, all - 1));
          if (!t.s.rot) continue;
          float cs[V], sn[V];
          qk_angles<V>(t.s, turn, t.c, position(t.row), cs, sn);
#pragma unroll
          for (int k = 0; k < V / 4; ++k) {
            angle_s[(k * kAngles + n) * threads + tid] = make_float4(cs[4 * k], cs[4 * k + 1], cs[4 * k + 2], cs[4 * k + 3]);
            angle_s[((k + V / 4) * kAngles + n) * threads + tid] = make_float4(sn[4 * k], sn[4 * k + 1], sn[4 * k + 2], sn[4 * k + 3]);
          }
        }
      }
    }

#pragma unroll 1
    for (int h = h0; h < h1; ++h) {
      float* const scale_at = scales + h;
      const float old = *scale_at;
      uint8_t* const page = pool + h * head_stride;
      float a[kHold + 1][V], b[kHold + 1][V], top = 0.0f;
      if constexpr (kHold > 0) ptx::cp_async_wait<kAppendStages - 1>();
#pragma unroll
      for (int n = 0; n < kHold; ++n) {
        const uint32_t at = ring + static_cast<uint32_t>((((h - h0) % kAppendStages * kHold + n) * 2) * threads * 2 * V);
        append_shared<T, V>(at).widen(a[n]);
        append_shared<T, V>(at + threads * 2 * V).widen(b[n]);
        if (rot[n]) {
          float cs[V], sn[V];
          angles(n, cs, sn);
          rotate(a[n], b[n], cs, sn);
        }
        top = largest(top, a[n], b[n]);  // (zeros where there is no slot)
      }
      if constexpr (kHold > 0) ask(h + kAppendStages);
      if constexpr (!kHeld) {
#pragma unroll 1
        for (int at = tid + kHold * threads, n = kHold; at < all; at += threads, ++n) {
          float ya[V], yb[V];
          values(slot(at), n, h, ya, yb);
          top = largest(top, ya, yb);
        }
      }
      // two places by turns: the warps that are late still read the last head's
      float* const tops = top_s[parity & 1u];
      ++parity;
      auto over_block = [&](float m, float* to) {
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));  // (none is negative, or NaN)
        if (threads == 32) return m;
        if ((tid & 31) == 0) to[tid >> 5] = m;
        __syncthreads();
        const int warps = threads / 32;  // (others' places are zero)
        for (int w = 0; w < warps; w += 4) {
          const float4 y = *reinterpret_cast<const float4*>(to + w);
          m = ptx::max3(m, y.x, y.y);
          m = ptx::max3(m, y.z, y.w);
        }
        return m;
      };
      top = over_block(top, tops);
      const bool infinite = top == INFINITY;  // (the whole block's)
      if (infinite) {
        float m = 0.0f;
#pragma unroll
        for (int n = 0; n < kHold; ++n) m = largest_finite(m, a[n], b[n]);
        if constexpr (!kHeld) {
          for (int at = tid + kHold * threads, n = kHold; at < all; at += threads, ++n) {
            float ya[V], yb[V];
            values(slot(at), n, h, ya, yb);
            m = largest_finite(m, ya, yb);
          }
        }
        if (threads > 32) __syncthreads();
        top = over_block(m, tops);
      }
      const float need = __int_as_float((max(e4m3_scale_exponent(top), kMinScaleExponent) + 127) << 23);
      const float scale = lo == row0 ? need : fmaxf(old, need);
      __syncwarp();
      if (tid == 0) *scale_at = scale;  // every thread has read the old one

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
            const float2 u = __half22float2(*reinterpret_cast<const __half2*>(&lo2));
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&hi2));
            w[i] = e4m3_pack4(u.x * by, u.y * by, v.x * by, v.y * by);
          }
          *to = y;
        }
      }
      const uint32_t bits = __float_as_uint(scale);  // (a power of two, but for an old one that the caller made)
      const float by = (bits & 0x7fffffu) == 0 && bits < 254u << 23 ? __uint_as_float((254u << 23) - bits) : 1.0f / scale;
      auto store = [&](uint8_t* at_a, uint8_t* at_b, float (&ya)[V], float (&yb)[V]) {
        vscale<V>(ya, ya, by);
        vscale<V>(yb, yb, by);
        if (infinite) {  // infinities become NaN
#pragma unroll
          for (int e = 0; e < V; ++e) {
            ya[e] = fmaf(ya[e], 0.0f, ya[e]);
            yb[e] = fmaf(yb[e], 0.0f, yb[e]);
          }
        }
        if constexpr (V == 8) {
          *reinterpret_cast<uint2*>(at_a) =
              make_uint2(e4m3_pack4(ya[0], ya[1], ya[2], ya[3]), e4m3_pack4(ya[4], ya[5], ya[6], ya[7]));
          *reinterpret_cast<uint2*>(at_b) =
              make_uint2(e4m3_pack4(yb[0], yb[1], yb[2], yb[3]), e4m3_pack4(yb[4], yb[5], yb[6], yb[7]));
        } else if constexpr (V == 4) {
          *reinterpret_cast<uint32_t*>(at_a) = e4m3_pack4(ya[0], ya[1], ya[2], ya[3]);
          *reinterpret_cast<uint32_t*>(at_b) = e4m3_pack4(yb[0], yb[1], yb[2], yb[3]);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const uint32_t y = e4m3_pack(ya[e], yb[e]);
            at_a[e] = static_cast<uint8_t>(y);
            at_b[e] = static_cast<uint8_t>(y >> 8);
          }
        }
      };
#pragma unroll
      for (int n = 0; n < kHold; ++n)
        if (on[n]) store(page + to[n], page + to[n] + apart[n], a[n], b[n]);
      if constexpr (!kHeld) {
#pragma unroll 1
        for (int at = tid + kHold * threads, n = kHold; at < all; at += threads, ++n) {
          float ya[V], yb[V];
          const Slot t = slot(at);
          values(t, n, h, ya, yb);
          uint8_t* const to = page + (t.row - row0) * row_stride;
          store(to + t.s.ia, to + t.s.ib, ya, yb);
        }
      }
    }
  }
}

}  // namespace vattn
