// qk_norm_rope_kernel.cuh -- RMS norm of every q and k row with the NeoX
// rotation in the same pass, and its gradient.
//
// A row is one head of one token, x[0 .. D).  With r = 1 / sqrt(mean(x^2) +
// eps) and w the tensor's weight:
//   y = x r w,   out = R(theta) y,
// where R turns the pairs (y[i], y[i + half]), i < half = rope_dims / 2, by
// theta_i = position * base^(-2 i / rope_dims) (/ factors[i]) as
// rope_kernel.cuh does and leaves dims >= 2 * half alone.  Backward, from g
// = d out:
//   g' = R(-theta) g,   dw += g' x r,   dx = r (g' w) - x r^3 / D sum(g' w x).
//
// Angles: in turns, position * f_i only counts modulo 1, so f_i is held as a
// 64-bit binary fraction (from 77 digits, rope_turns.h: those of an f64 alone leave
// 2^-25 turns at positions near 2^31) and position * f_i is one wrapping
// integer product: within 2^-31 turns at any 32-bit position, where an f32
// product loses all digits.  The fraction is cut to the nearest quarter turn
// and the rest goes through two short polynomials (qk_sincos).
//
// Work split: a group of lanes holds one row, lane = slot of V pairs (two
// 16-byte accesses where the sizes allow), so the rotation needs no exchange
// and the sums a few shuffles.  A group walks over tokens, and for each over a
// slice of the heads of one tensor: the angles, multiplied with the weights,
// stay in registers meanwhile.  Each row is read once and written once.  What
// bounds it is bytes in flight: each thread keeps its next rows coming
// through a ring of its own in shared memory (cp.async; no barrier, a thread
// reads what it asked for).  4 x 40 heads x 4096 x 128 bf16: 52.3 us, 6.4 TB/s (94
// % of the measured copy rate), with two rows a thread in registers 74 us; its
// gradient at 4 x 20 heads 46.0 us, 5.5 TB/s, weight sums included, from 105
// us (48.3 with its two sums one after the other).  The arithmetic, in packed f32
// pairs, is about 80 instructions for the 64 bytes of a lane and row.  16 + 16 heads
// x 4100 x 72 f32, 32 bytes a lane and row: 13.7 us, 5.5 TB/s, at 2.5 instructions a
// cycle; with three blocks a multiprocessor and groups of 16 lanes 15.9 (2.7).
#pragma once

#include <cstdint>

#include "elem.cuh"
#include "ptx.cuh"
#include "window_common.cuh"

namespace vattn {

constexpr int kQkThreads = 256;
constexpr int kQkMaxDim = 128;
// Blocks a multiprocessor holds, by registers, for V pairs a lane.
constexpr int qk_resident(int v, bool backward) { return v == 8 ? 2 : (backward ? 3 : 4); }

struct QkTensor {
  const void* x;   // input rows
  const void* g;   // gradient of the output rows (backward)
  void* y;         // output rows, or gradient of the input rows
  const void* w;   // weight or null
  long long xs[3], gs[3], ys[3];  // strides (batch, head, row), elements
  int heads;
  int slices;           // blocks in y that share the heads
  int heads_per_slice;
};

struct QkParams {
  QkTensor t[2];  // q, k
  const int32_t* positions;
  const float* factors;
  float* part;  // backward: [gridDim.y * gridDim.x][D] weight gradient of each block
  long long tokens;
  long long pos0;
  FastDiv d_n;
  int n;  // rows of a sequence
  int D;
  int half;
  int slots;  // pair slots of a row
  int log_lanes;  // lanes of a row, where these are a power of two
  int w_f32;
  float eps;
  double turns[kQkMaxDim / 2];  // turns per position
  float turns_rest[kQkMaxDim / 2];  // what that rounds away
};

// One lane's place in a row: V pairs (a[ia ..], b[ib ..]).
template <int V>
struct QkSlot {
  int ia, ib;
  bool here, pair, rot;
  __device__ __forceinline__ void set(const QkParams& p, int c) {
    const int i = c * V, rest = p.D - 2 * p.half;
    here = c < p.slots;
    rot = here && i < p.half;
    const int r = i - p.half;
    ia = rot ? i : 2 * p.half + r;
    ib = rot ? i + p.half : 2 * p.half + (rest + 1) / 2 + r;
    pair = here && ib < p.D;  // V == 1 and an odd rest: the last slot has no partner
  }
};

template <int V>
__device__ __forceinline__ void qk_weight(const QkSlot<V>& s, const void* w, int w_f32, bool bf16,
                                          float (&wa)[V], float (&wb)[V]) {
  auto at = [&](int i) -> float {
    if (w == nullptr) return 1.0f;
    if (w_f32) return static_cast<const float*>(w)[i];
    return bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(w)[i])
                : __half2float(static_cast<const __half*>(w)[i]);
  };
#pragma unroll
  for (int e = 0; e < V; ++e) {
    wa[e] = s.here ? at(s.ia + e) : 0.0f;
    wb[e] = s.pair ? at(s.ib + e) : 0.0f;
  }
}

// sin and cos of a 32-bit fraction of a turn, to 1.3 x 2^-24: quadrant and
// remainder y in [-pi/4, pi/4] from the integer, then sin y = y + y^3 A(y^2) and
// cos y = 1 - y^2/2 + y^4 B(y^2) with A and B of degree 2, the interpolation of
// (sin y / y - 1) / y^2 and (cos y - 1 + y^2/2) / y^4 at the Chebyshev points
// of [0, (pi/4)^2].
__device__ __forceinline__ void qk_sincos(uint32_t phase, float& sn, float& cs) {
  const uint32_t k = (phase + 0x20000000u) >> 30;  // quarter turns
  const float y = static_cast<float>(static_cast<int32_t>(phase - (k << 30))) * 0x1.921fb6p-30f;  // 2 pi / 2^32
  const float z = y * y;
  const float a = fmaf(fmaf(-0.000195878909f, z, 0.00833274797f), z, -0.166666642f);
  const float b = fmaf(fmaf(2.45479423e-05f, z, -0.00138883025f), z, 0.0416666642f);
  const float s = fmaf(y * z, a, y);
  const float c = fmaf(z * z, b, fmaf(-0.5f, z, 1.0f));
  const float s1 = (k & 1u) ? c : s, c1 = (k & 1u) ? s : c;
  sn = (k & 2u) ? -s1 : s1;
  cs = ((k + 1u) & 2u) ? -c1 : c1;
}

template <int V>
__device__ __forceinline__ void qk_angles(const QkSlot<V>& s, const uint64_t* turn, int c,
                                          long long pos, float (&cs)[V], float (&sn)[V]) {
#pragma unroll
  for (int e = 0; e < V; ++e) {
    cs[e] = 1.0f;
    sn[e] = 0.0f;
    if (s.rot) qk_sincos(static_cast<uint32_t>((static_cast<uint64_t>(pos) * turn[c * V + e]) >> 32), sn[e], cs[e]);
  }
}

// d = a * b, d = a * b + c over V lanes' worth, in pairs where V is even.
template <int V>
__device__ __forceinline__ void vmul(float (&d)[V], const float (&a)[V], const float (&b)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 r = __fmul2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]));
      d[e] = r.x;
      d[e + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) d[e] = a[e] * b[e];
  }
}
template <int V>
__device__ __forceinline__ void vfma(float (&d)[V], const float (&a)[V], const float (&b)[V], const float (&c)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int e = 0; e < V; e += 2) {
      const float2 r = __ffma2_rn(make_float2(a[e], a[e + 1]), make_float2(b[e], b[e + 1]), make_float2(c[e], c[e + 1]));
      d[e] = r.x;
      d[e + 1] = r.y;
    }
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) d[e] = fmaf(a[e], b[e], c[e]);
  }
}
template <int V>
__device__ __forceinline__ void vscale(float (&d)[V], const float (&a)[V], float b) {
  float bb[V];
#pragma unroll
  for (int e = 0; e < V; ++e) bb[e] = b;
  vmul<V>(d, a, bb);
}
template <int V>
__device__ __forceinline__ float vsum(const float (&a)[V]) {
  float s = 0.0f;
#pragma unroll
  for (int e = 0; e < V; ++e) s += a[e];
  return s;
}

__device__ __forceinline__ void qk_turns(const QkParams& p, uint64_t* turn) {
  if (static_cast<int>(threadIdx.x) < p.half) {
    double f = p.turns[threadIdx.x];
    float rest = p.turns_rest[threadIdx.x];  // 24 of its digits are enough: f64 arithmetic is slow
    if (p.factors != nullptr) {
      const float by = p.factors[threadIdx.x];
      const double q = f / by;
      rest = (static_cast<float>(fma(-q, static_cast<double>(by), f)) + rest) / by;
      f = q;
    }
    // the fractions of both, times 2^64; their sum modulo that
    f -= floor(f);
    rest -= rintf(rest);
    turn[threadIdx.x] = static_cast<uint64_t>(f * 0x1p64) + static_cast<uint64_t>(static_cast<long long>(rest * 0x1p64f));
  }
  __syncthreads();
}

template <typename T, int V>
__device__ __forceinline__ Vec<T, V> qk_load(const T* row, int i, bool here) {
  Vec<T, V> v;
  if (here) {
    v = *reinterpret_cast<const Vec<T, V>*>(row + i);
  } else {
#pragma unroll
    for (int e = 0; e < V; ++e) v.e[e] = Elem<T>::narrow(0.0f);
  }
  return v;
}

// A thread's group (lanes that hold one row) and place in it.  kOdd: a group has
// as many lanes as the row has slots, 3 to 10; what is left of the warp is group
// -1 and has no slot.  Else a power of two.
template <bool kOdd>
struct QkLane {
  int lanes, c0, group, groups;  // groups of a block
  __device__ __forceinline__ explicit QkLane(const QkParams& p) {
    const int tid = static_cast<int>(threadIdx.x);
    if constexpr (kOdd) {
      lanes = p.slots;
      const int rows = 32 / lanes, row = (tid & 31) / lanes;
      groups = kQkThreads / 32 * rows;
      group = row < rows ? (tid >> 5) * rows + row : -1;
      c0 = row < rows ? (tid & 31) - row * lanes : 32;
    } else {
      lanes = 1 << p.log_lanes;
      groups = kQkThreads >> p.log_lanes;
      group = tid >> p.log_lanes;
      c0 = tid & (lanes - 1);
    }
  }
  // Sum over the group.  kOdd: down to its first lane (which adds, in each step,
  // what its partner had before it) and back; else xor, which stays inside.
  __device__ __forceinline__ float sum(float x) const {
    if constexpr (kOdd) {
      for (int o = lanes > 8 ? 8 : 4; o > 0; o >>= 1) {
        const float y = __shfl_down_sync(0xffffffffu, x, o);
        if (c0 + o < lanes) x += y;
      }
      return __shfl_sync(0xffffffffu, x, (static_cast<int>(threadIdx.x) & 31) - (c0 & 31));
    } else {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        if (o < lanes) x += __shfl_xor_sync(0xffffffffu, x, o);
      return x;
    }
  }
  // Two sums at once (a power of two of lanes).
  __device__ __forceinline__ void sum2(float& x, float& y) const {
    static_assert(!kOdd, "a power of two");
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o >= lanes) continue;
      const float a = __shfl_xor_sync(0xffffffffu, x, o), b = __shfl_xor_sync(0xffffffffu, y, o);
      x += a;
      y += b;
    }
  }
};

// The rows of a group in the order it takes them: tokens first, + stride, ...,
// for each the heads [h0, h1).  N tensors of one shape are read (x, or x and
// g), kStages rows ahead through the thread's ring where an access has 8 bytes
// or more, else in place.
template <typename T, int V, int SL, int N>
struct QkRing {
  static constexpr int kBytes = V * static_cast<int>(sizeof(T));
  static constexpr bool kAsync = kBytes >= 8 && SL == 1;
  static constexpr int kStages = kAsync ? (N == 1 && V == 8 ? 6 : 4) : 1;
  static constexpr int kSmemBytes = kAsync ? kStages * N * 2 * kBytes * kQkThreads : 0;

  const QkParams& p;
  const QkTensor& t;
  const QkSlot<V> (&s)[SL];
  int h0, h1;
  long long stride;
  uint32_t base;
  // the next row to ask for
  long long token;
  const T* row[N];
  int h, stage;

  __device__ __forceinline__ QkRing(const QkParams& p_, const QkTensor& t_, const QkSlot<V> (&s_)[SL], int h0_, int h1_,
                                    long long first, long long stride_, uint32_t smem)
      : p(p_), t(t_), s(s_), h0(h0_), h1(h1_), stride(stride_), base(smem + threadIdx.x * kBytes), token(first), h(h0_),
        stage(0) {
    rows(token);
    if constexpr (kAsync)
      for (int i = 0; i < kStages; ++i) ask();
  }
  // rows of a token's first head
  __device__ __forceinline__ void rows(long long tk) {
    if (tk >= p.tokens) tk = p.tokens - 1;
    const long long b = p.tokens <= 0x7fffffffLL ? static_cast<long long>(p.d_n.div(static_cast<uint32_t>(tk))) : tk / p.n;
    const long long n = tk - b * p.n;
    row[0] = static_cast<const T*>(t.x) + b * t.xs[0] + n * t.xs[2] + h0 * t.xs[1];
    if constexpr (N == 2) row[1] = static_cast<const T*>(t.g) + b * t.gs[0] + n * t.gs[2] + h0 * t.gs[1];
  }
  __device__ __forceinline__ void advance() {
    row[0] += t.xs[1];
    if constexpr (N == 2) row[1] += t.gs[1];
    if (++h == h1) {
      h = h0;
      token += stride;
      if (token < p.tokens) rows(token);
    }
  }
  // Asks for the next row (an empty group behind the last).
  __device__ __forceinline__ void ask() {
    static_assert(SL == 1, "one slot a lane");
    if (token < p.tokens) {
      const uint32_t at = base + static_cast<uint32_t>(stage) * (N * 2 * kBytes * kQkThreads);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        ptx::cp_async<kBytes>(at + (2 * i) * kBytes * kQkThreads, row[i] + (s[0].here ? s[0].ia : 0), s[0].here);
        ptx::cp_async<kBytes>(at + (2 * i + 1) * kBytes * kQkThreads, row[i] + (s[0].pair ? s[0].ib : 0), s[0].pair);
      }
      advance();
    }
    ptx::cp_async_commit();
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  // The oldest row asked for; more() once its values have been used.
  __device__ __forceinline__ void take(Vec<T, V> (&a)[N][SL], Vec<T, V> (&b)[N][SL]) {
    if constexpr (kAsync) {
      ptx::cp_async_wait<kStages - 1>();
      const uint32_t at = base + static_cast<uint32_t>(stage) * (N * 2 * kBytes * kQkThreads);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        get(a[i][0], at + (2 * i) * kBytes * kQkThreads);
        get(b[i][0], at + (2 * i + 1) * kBytes * kQkThreads);
      }
    } else {
      const bool on = token < p.tokens;
#pragma unroll
      for (int i = 0; i < N; ++i)
#pragma unroll
        for (int k = 0; k < SL; ++k) {
          a[i][k] = qk_load<T, V>(row[i], s[k].ia, on && s[k].here);
          b[i][k] = qk_load<T, V>(row[i], s[k].ib, on && s[k].pair);
        }
    }
  }
  __device__ __forceinline__ void more() {
    if constexpr (kAsync) ask();
    else if (token < p.tokens) advance();
  }
  static __device__ __forceinline__ void get(Vec<T, V>& v, uint32_t at) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&v);
    if constexpr (kBytes == 16)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
    else
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(at) : "memory");
  }
};

// A block's tensor, heads and tokens.
struct QkShare {
  int which, h0, h1;
  long long block_first, first, stride;  // tokens of the block, of this thread's group (p.tokens: none)
  template <bool kOdd>
  __device__ __forceinline__ QkShare(const QkParams& p, const QkLane<kOdd>& lane) {
    which = static_cast<int>(blockIdx.y) < p.t[0].slices ? 0 : 1;
    const int slice = static_cast<int>(blockIdx.y) - (which == 0 ? 0 : p.t[0].slices);
    h0 = slice * p.t[which].heads_per_slice;
    h1 = min(p.t[which].heads, h0 + p.t[which].heads_per_slice);
    block_first = static_cast<long long>(blockIdx.x) * lane.groups;
    first = kOdd && lane.group < 0 ? p.tokens : block_first + lane.group;
    stride = static_cast<long long>(gridDim.x) * lane.groups;
  }
};

// SL slots per lane (2 only where V == 1 needs up to 64 slots of a warp).
// All groups of a block take the same number of tokens: those past the end
// work on zeros and store nothing.
template <typename T, int V, int SL, bool kOdd>
__global__ void __launch_bounds__(kQkThreads, qk_resident(V, false))
    vattn_qk_norm_rope_kernel(const __grid_constant__ QkParams p) {
  extern __shared__ __align__(16) uint8_t qk_smem[];
  __shared__ uint64_t turn[kQkMaxDim / 2];
  const QkLane<kOdd> lane(p);
  const QkShare sh(p, lane);
  const QkTensor& t = p.t[sh.which];
  const int lanes = lane.lanes, c0 = lane.c0;
  QkSlot<V> s[SL];
#pragma unroll
  for (int k = 0; k < SL; ++k) s[k].set(p, c0 + k * lanes);
  QkRing<T, V, SL, 1> ring(p, t, s, sh.h0, sh.h1, sh.first, sh.stride, ptx::smem_addr(qk_smem));
  qk_turns(p, turn);
  float wa[SL][V], wb[SL][V];
#pragma unroll
  for (int k = 0; k < SL; ++k) qk_weight<V>(s[k], t.w, p.w_f32, Elem<T>::kBf16, wa[k], wb[k]);
  const float inv_d = 1.0f / static_cast<float>(p.D);
  long long token = sh.first;
  for (long long f = sh.block_first; f < p.tokens; f += sh.stride, token += sh.stride) {
    const bool valid = token < p.tokens;
    const long long tk = valid ? token : p.tokens - 1;
    const long long b = p.tokens <= 0x7fffffffLL ? static_cast<long long>(p.d_n.div(static_cast<uint32_t>(tk))) : tk / p.n;
    const long long n = tk - b * p.n;
    const long long pos = p.positions != nullptr ? p.positions[tk] : p.pos0 + n;
    // out_a = r (x_a [w_a cos] - x_b [w_b sin]), out_b = r (x_a [w_a sin] + x_b [w_b cos])
    float ac[SL][V], as[SL][V], bc[SL][V], bs[SL][V];
#pragma unroll
    for (int k = 0; k < SL; ++k) {
      float cs[V], sn[V];
      qk_angles<V>(s[k], turn, c0 + k * lanes, pos, cs, sn);
      vmul<V>(ac[k], wa[k], cs);
      vmul<V>(as[k], wa[k], sn);
      vmul<V>(bc[k], wb[k], cs);
      vscale<V>(sn, sn, -1.0f);
      vmul<V>(bs[k], wb[k], sn);
    }
    T* row = static_cast<T*>(t.y) + b * t.ys[0] + n * t.ys[2] + sh.h0 * t.ys[1];
    for (int h = sh.h0; h < sh.h1; ++h, row += t.ys[1]) {
      Vec<T, V> xa[1][SL], xb[1][SL];
      ring.take(xa, xb);
      float fa[SL][V], fb[SL][V], sq[V];
#pragma unroll
      for (int e = 0; e < V; ++e) sq[e] = 0.0f;
#pragma unroll
      for (int k = 0; k < SL; ++k) {
        xa[0][k].widen(fa[k]);
        xb[0][k].widen(fb[k]);
        vfma<V>(sq, fa[k], fa[k], sq);
        vfma<V>(sq, fb[k], fb[k], sq);
      }
      const float r = rsqrtf(fmaf(lane.sum(vsum<V>(sq)), inv_d, p.eps));
      ring.more();
      if (!valid) continue;
#pragma unroll
      for (int k = 0; k < SL; ++k) {
        float oa[V], ob[V], ta[V], tb[V];
        vscale<V>(ta, fa[k], r);
        vscale<V>(tb, fb[k], r);
        vmul<V>(oa, tb, bs[k]);
        vfma<V>(oa, ta, ac[k], oa);
        vmul<V>(ob, tb, bc[k]);
        vfma<V>(ob, ta, as[k], ob);
        Vec<T, V> va, vb;
        va.narrow(oa);
        vb.narrow(ob);
        if (s[k].here) *reinterpret_cast<Vec<T, V>*>(row + s[k].ia) = va;
        if (s[k].pair) *reinterpret_cast<Vec<T, V>*>(row + s[k].ib) = vb;
      }
    }
  }
}

// The gradient.  A block keeps its slice's share of dw in registers: lane
// sums, then the groups of a warp by shuffles, the warps through shared
// memory, and one row of `part` per block that vattn_qk_weight_sum_kernel
// adds in a fixed order.
template <typename T, int V, int SL>
__global__ void __launch_bounds__(kQkThreads, qk_resident(V, true))
    vattn_qk_norm_rope_backward_kernel(const __grid_constant__ QkParams p) {
  extern __shared__ __align__(16) uint8_t qk_smem[];
  __shared__ uint64_t turn[kQkMaxDim / 2];
  __shared__ float red[kQkThreads / 32][kQkMaxDim];
  const QkLane<false> lane(p);
  const QkShare sh(p, lane);
  const QkTensor& t = p.t[sh.which];
  const int lanes = lane.lanes, c0 = lane.c0;
  const float inv_d = 1.0f / static_cast<float>(p.D);
  QkSlot<V> s[SL];
#pragma unroll
  for (int k = 0; k < SL; ++k) s[k].set(p, c0 + k * lanes);
  QkRing<T, V, SL, 2> ring(p, t, s, sh.h0, sh.h1, sh.first, sh.stride, ptx::smem_addr(qk_smem));
  float wa[SL][V], wb[SL][V], da[SL][V], db[SL][V];
  qk_turns(p, turn);
#pragma unroll
  for (int k = 0; k < SL; ++k) {
    qk_weight<V>(s[k], t.w, p.w_f32, Elem<T>::kBf16, wa[k], wb[k]);
#pragma unroll
    for (int e = 0; e < V; ++e) da[k][e] = db[k][e] = 0.0f;
  }
  long long token = sh.first;
  for (long long f = sh.block_first; f < p.tokens; f += sh.stride, token += sh.stride) {
    const bool valid = token < p.tokens;
    const long long tk = valid ? token : p.tokens - 1;
    const long long b = p.tokens <= 0x7fffffffLL ? static_cast<long long>(p.d_n.div(static_cast<uint32_t>(tk))) : tk / p.n;
    const long long n = tk - b * p.n;
    const long long pos = p.positions != nullptr ? p.positions[tk] : p.pos0 + n;
    float cs[SL][V], sn[SL][V];
#pragma unroll
    for (int k = 0; k < SL; ++k) qk_angles<V>(s[k], turn, c0 + k * lanes, pos, cs[k], sn[k]);
    T* row = static_cast<T*>(t.y) + b * t.ys[0] + n * t.ys[2] + sh.h0 * t.ys[1];
    for (int h = sh.h0; h < sh.h1; ++h, row += t.ys[1]) {
      Vec<T, V> va[2][SL], vb[2][SL];
      ring.take(va, vb);
      // g' = R(-theta) g, and the row's two sums
      float xa[SL][V], xb[SL][V], ga[SL][V], gb[SL][V], sq[V], dt[V];
#pragma unroll
      for (int e = 0; e < V; ++e) sq[e] = dt[e] = 0.0f;
#pragma unroll
      for (int k = 0; k < SL; ++k) {
        float fa[V], fb[V], tmp[V];
        va[0][k].widen(xa[k]);
        vb[0][k].widen(xb[k]);
        va[1][k].widen(fa);
        vb[1][k].widen(fb);
        vmul<V>(tmp, fb, sn[k]);
        vfma<V>(ga[k], fa, cs[k], tmp);
        vscale<V>(fa, fa, -1.0f);
        vmul<V>(tmp, fa, sn[k]);
        vfma<V>(gb[k], fb, cs[k], tmp);
        vfma<V>(sq, xa[k], xa[k], sq);
        vfma<V>(sq, xb[k], xb[k], sq);
        vmul<V>(tmp, ga[k], wa[k]);
        vfma<V>(dt, tmp, xa[k], dt);
        vmul<V>(tmp, gb[k], wb[k]);
        vfma<V>(dt, tmp, xb[k], dt);
      }
      float sum = vsum<V>(sq), dot = vsum<V>(dt);
      lane.sum2(sum, dot);
      ring.more();
      if (!valid) continue;
      const float r = rsqrtf(fmaf(sum, inv_d, p.eps));
      const float back = -dot * inv_d * r * r * r;  // times x: the norm's own share
      float kk[V];
#pragma unroll
      for (int e = 0; e < V; ++e) kk[e] = back;
#pragma unroll
      for (int k = 0; k < SL; ++k) {
        // u = g' r, dw += u x, dx = u w + x back
        float tmp[V];
        Vec<T, V> oa, ob;
        vscale<V>(ga[k], ga[k], r);
        vscale<V>(gb[k], gb[k], r);
        vfma<V>(da[k], ga[k], xa[k], da[k]);
        vfma<V>(db[k], gb[k], xb[k], db[k]);
        vmul<V>(tmp, ga[k], wa[k]);
        vfma<V>(tmp, xa[k], kk, tmp);
        oa.narrow(tmp);
        vmul<V>(tmp, gb[k], wb[k]);
        vfma<V>(tmp, xb[k], kk, tmp);
        ob.narrow(tmp);
        if (s[k].here) *reinterpret_cast<Vec<T, V>*>(row + s[k].ia) = oa;
        if (s[k].pair) *reinterpret_cast<Vec<T, V>*>(row + s[k].ib) = ob;
      }
    }
  }
  ptx::grid_dep_launch();
  if (p.part == nullptr) return;
  const int warp = static_cast<int>(threadIdx.x) >> 5;
#pragma unroll
  for (int k = 0; k < SL; ++k)
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float a = da[k][e], c = db[k][e];
      for (int o = lanes; o < 32; o <<= 1) {
        a += __shfl_xor_sync(0xffffffffu, a, o);
        c += __shfl_xor_sync(0xffffffffu, c, o);
      }
      if ((threadIdx.x & 31) < static_cast<unsigned>(lanes)) {
        if (s[k].here) red[warp][s[k].ia + e] = a;
        if (s[k].pair) red[warp][s[k].ib + e] = c;
      }
    }
  __syncthreads();
  for (int d = threadIdx.x; d < p.D; d += kQkThreads) {
    float a = 0.0f;
#pragma unroll
    for (int w = 0; w < kQkThreads / 32; ++w) a += red[w][d];
    p.part[(static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x) * p.D + d] = a;
  }
}

// dw of one tensor (blockIdx.y) in 32 columns (blockIdx.x): the rows of
// `part` in order, 32 interleaved partial sums, then their sum.
struct QkWeightSum {
  const float* part;
  float* dw[2];
  long long row0[2], row1[2];
  int D;
};

__global__ void __launch_bounds__(1024) vattn_qk_weight_sum_kernel(const QkWeightSum p) {
  __shared__ float red[32][33];
  ptx::grid_dep_wait();
  const int which = blockIdx.y;
  const int d = blockIdx.x * 32 + threadIdx.x;
  if (p.dw[which] == nullptr) return;
  float a = 0.0f;
  if (d < p.D)
#pragma unroll 8
    for (long long r = p.row0[which] + threadIdx.y; r < p.row1[which]; r += 32) a += p.part[r * p.D + d];
  red[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  if (threadIdx.y == 0 && d < p.D) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) sum += red[i][threadIdx.x];
    p.dw[which][d] = sum;
  }
}

}  // namespace vattn
