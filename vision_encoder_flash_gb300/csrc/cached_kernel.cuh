// cached_kernel.cuh -- attention of a few new tokens over a cache
// (vattn_forward_cached): one token, a run of them, or a tree.
//
// Memory bound: every visible key and value is read once, for all rows (new
// token, query head of the group) of its key head together.  A block takes
// up to 16 RW rows and a share of the keys, 64 keys at a time, through a
// three-stage cp.async ring; the two products are mma.sync m16n8k16, whose 16
// rows fit the few that there are (a tcgen05 tile has 128).  RW groups of
// warps take 16 rows each, the warps of a group share the tile's keys:
//   rows <= 16: four warps, 16 keys of the tile each
//   rows <= 32: two groups of four, 16 keys each (above 64 dims of two, 32
//               keys: eight warps' registers would leave one block resident)
//   more:       four groups of two, 32 keys each (a tree of 31 tokens, 4 heads
//               a key head, over 4096 keys: see cached_launch)
//
// Rows of 32, 64 or 128 dims in shared memory and registers, zeros behind
// head_dim: loops without a bound in them are 5 to 20 % faster (32 x 8 key heads x
// 8000 keys: 72 dims 78.6 us, else 92.8; 80 dims in a tree 30.9, else 29.6).
//
// The keys that any row sees are numbered through: first the first keys that
// lie before the lowest window, then those from that window to the end.  The
// shares of the blocks are equal parts of that list, cut on the device from
// the sequence's own length.  Up to four shares are a cluster: each block
// leaves its unnormalised O, maximum and sum in its shared memory, and all of
// them merge a part of the rows from there, in the order of the shares.  More
// shares go through a workspace and vattn_cached_join_kernel, likewise in order.
//
// 32 sequences x 8 key heads x up to 16385 keys of 128 bf16: 201 us, 7.2 TB/s
// (the measured copy rate is 6.8; 217 us while every row's address was formed by
// itself, O rescaled in every tile, and the loops bounded by head_dim).  A tree of 31 tokens over 4 x 4 heads x 4100
// keys of 64 f16: 19.4 us, bound by latency: seven tiles a block of about 1.2 us,
// 2.3 us before the first, the rest the joins.
//
// Weights are rounded to the tensors' type for the second product, as in
// window_fwd_kernel.cuh; everything else is f32.  Rows differ in what they
// see only at the window's edge and among the new tokens: tiles there are
// masked element by element, and if such a tile holds a value that is not
// finite, its second product is done by loops over the visible pairs, since
// 0 x infinity is not 0.
#pragma once

#include "../../include/vattn_decoder.h"
#include "window_pipe.cuh"

namespace vattn {

constexpr int kCachedKeys = 64;  // keys of a tile
constexpr int kCachedStages = 3;
constexpr int kCachedMaxSplits = 512;
// Shares that a cluster of blocks joins by itself (4 x 4 key heads x 31 tokens in a
// tree over 200 keys of 64, two shares: 11.4 us, through a workspace 13.8; over 600
// keys, five shares: 16.4 and 15.5, since larger clusters find less room).
constexpr int kCachedCluster = 4;

struct CachedParams {
  WindowParams w;
  RowsTensor q, k, v, out;
  float* part_o;  // [sequence and key head][row block][split][16 RW][dim]
  float* part_ml;  // ... [16 RW][2]: maximum (log2 units) and sum
  int rows;        // group * n_queries
  int row_blocks;
  int splits;
  float scale_log2;
};

// The keys of one sequence and a split's share of them.
struct CachedSpan {
  int base, len;    // new token t is row base + t; rows in use
  int sinks, first; // listed: keys [0, sinks) and [first, len)
  int per, n;       // keys of a share, of all

  __device__ __forceinline__ static CachedSpan make(const WindowParams& w, int b, int splits) {
    CachedSpan s;
    s.len = min(max(w.kv_len[b], 0), w.n_keys);
    s.base = s.len - w.n_queries;
    s.first = max(0, s.base - w.window + 1);
    s.sinks = min(w.sinks, s.first);
    s.n = s.sinks + s.len - s.first;
    s.per = ((s.n + splits - 1) / splits + kCachedKeys - 1) / kCachedKeys * kCachedKeys;
    return s;
  }
  __device__ __forceinline__ int key(int i) const { return i < sinks ? i : first + (i - sinks); }
  __device__ __forceinline__ int shares() const { return n == 0 ? 1 : (n + per - 1) / per; }
};

// Ancestor bits of new token t; none if the token has no row.
__device__ __forceinline__ uint64_t cached_word(const WindowParams& w, int b, int t, int base) {
  if (base + t < 0) return 0;
  const uint64_t all = w.n_queries >= 64 ? ~0ull : (1ull << w.n_queries) - 1;
  if (w.tree == nullptr) return (2ull << t) - 1;
  return w.tree[static_cast<long long>(b) * w.n_queries + t] & all;
}

template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (Elem<T>::kBf16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// Place of 16-byte chunk c in shared row r of CH chunks: eight consecutive
// rows have it in eight different banks' groups.
template <int CH>
__device__ __forceinline__ int swizzled(int r, int c) {
  return CH >= 8 ? c ^ (r & 7) : c ^ ((r >> 1) & 3);
}

template <int DP, int RW>
struct CachedPlan {
  static constexpr int kWarps = RW == 1 || (RW == 2 && DP == 128) ? 4 : 8;
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kKw = kWarps / RW;              // warps that share a tile's keys
  static constexpr int kWarpKeys = kCachedKeys / kKw;
  static constexpr int kTileBytes = kCachedKeys * DP * 2;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kOffP = kCachedStages * kStageBytes;  // weights of the loops' path, per warp
  static constexpr int kSmemBytes = kOffP + kWarps * 16 * kWarpKeys * 4;
  // blocks a multiprocessor, by shared memory (4 warps) or registers (8)
  static constexpr int kResident = (kWarps == 4 ? 4 : 2) / (DP <= 64 ? 1 : 2);
  static_assert(kWarps * 16 * (DP + 2) * 4 <= kOffP, "the warps' results reuse the ring");
};

template <typename T, int DP, int RW>
__global__ void __launch_bounds__(CachedPlan<DP, RW>::kThreads)
    vattn_cached_kernel(const __grid_constant__ CachedParams p) {
  using P = CachedPlan<DP, RW>;
  constexpr int KN = P::kWarpKeys / 8;  // 8-key blocks of a warp's tile share
  constexpr int CH = DP / 8;            // 16-byte chunks of a shared row
  constexpr int kThreads = P::kThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int kpos[VATTN_MAX_NEW_TOKENS];
  const uint32_t smem_s = ptx::smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rw = warp % RW, kw = warp / RW;
  const WindowParams& w = p.w;
  const int D = w.dim;
  const int split = blockIdx.x, rb = blockIdx.y;
  const bool clustered = p.splits > 1 && p.splits <= kCachedCluster;
  ptx::grid_dep_wait();
  for (long long bk = blockIdx.z; bk < static_cast<long long>(w.batch) * w.kv_heads; bk += gridDim.z) {
    const int b = static_cast<int>(bk / w.kv_heads), kh = static_cast<int>(bk - static_cast<long long>(b) * w.kv_heads);
    const CachedSpan sp = CachedSpan::make(w, b, p.splits);
    const int v0 = split * sp.per, v1 = min(sp.n, v0 + sp.per);
    const int shares = sp.shares();
    if (!clustered && split >= shares) continue;  // (in a cluster: with no keys, but at its barriers)
    __syncthreads();  // the previous sequence's reads of the ring and kpos
    if (tid < w.n_queries) kpos[tid] = sp.base + __popcll(cached_word(w, b, tid, sp.base)) - 1;

    // ---- the ring: thread = 16-byte chunk tid % CH of rows tid / CH, + kThreads / CH, ...
    const T* kbase = rows_at<T>(p.k, b, kh, 0);
    const T* vbase = rows_at<T>(p.v, b, kh, 0);
    const int ch = tid % CH, tiles = (max(v1 - v0, 0) + kCachedKeys - 1) / kCachedKeys;
    auto load = [&](int tile) {
      if (tile < tiles) {
        constexpr int kStep = kThreads / CH;  // rows; a multiple of 8, so a thread's swizzle is one
        static_assert(kStep % 8 == 0, "rows of a thread");
        const int r0 = tid / CH, i0 = v0 + tile * kCachedKeys;
        const uint32_t at = smem_s + static_cast<uint32_t>(tile % kCachedStages) * P::kStageBytes +
                            static_cast<uint32_t>(r0 * DP * 2 + (swizzled<CH>(r0, ch) << 4));
        if (i0 >= sp.sinks && i0 + kCachedKeys <= v1) {  // rows that follow each other
          const bool on = ch * 8 < D;
          const long long j = sp.key(i0) + r0;
          const T* kr = kbase + j * p.k.s[2] + (on ? ch * 8 : 0);
          const T* vr = vbase + j * p.v.s[2] + (on ? ch * 8 : 0);
#pragma unroll
          for (int r = 0; r < kCachedKeys; r += kStep) {
            ptx::cp_async<16>(at + r * DP * 2, kr, on);
            ptx::cp_async<16>(at + P::kTileBytes + r * DP * 2, vr, on);
            kr += kStep * p.k.s[2];
            vr += kStep * p.v.s[2];
          }
        } else {
#pragma unroll 1
          for (int r = 0; r < kCachedKeys; r += kStep) {
            const int i = i0 + r0 + r;
            const bool on = i < v1 && ch * 8 < D;
            const long long j = sp.key(i < v1 ? i : v0);
            const int c = on ? ch * 8 : 0;
            ptx::cp_async<16>(at + r * DP * 2, kbase + j * p.k.s[2] + c, on);
            ptx::cp_async<16>(at + P::kTileBytes + r * DP * 2, vbase + j * p.v.s[2] + c, on);
          }
        }
      }
      ptx::cp_async_commit();
    };
    load(0);
    load(1);

    // ---- the warp's 16 rows: lane / 4 and lane / 4 + 8
    uint32_t qf[DP / 16][4];
    int lo[2], sk[2];
    uint64_t word[2];
    const T* qrow[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = rb * 16 * RW + rw * 16 + (lane >> 2) + 8 * e;
      const int t = rr / w.group;
      word[e] = rr < p.rows ? cached_word(w, b, t, sp.base) : 0;
      qrow[e] = word[e] != 0 ? rows_at<T>(p.q, b, kh * w.group + (rr - t * w.group), t) : nullptr;
      lo[e] = word[e] != 0 ? sp.base + __popcll(word[e]) - 1 - w.window : 0x7fffffff;
      sk[e] = word[e] != 0 ? w.sinks : 0;
    }
#pragma unroll
    for (int ks = 0; ks < DP / 16; ++ks)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = ks * 16 + (lane & 3) * 2 + (e >> 1) * 8;
        qf[ks][e] = qrow[e & 1] != nullptr && c < D ? *reinterpret_cast<const uint32_t*>(qrow[e & 1] + c) : 0u;
      }

    float o[DP / 8][4];
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    for (int tile = 0; tile < tiles; ++tile) {
      ptx::cp_async_wait<1>();
      __syncthreads();
      load(tile + 2);
      const uint32_t ks_s = smem_s + static_cast<uint32_t>(tile % kCachedStages) * P::kStageBytes;
      const uint32_t vs_s = ks_s + P::kTileBytes;
      const int key0 = kw * P::kWarpKeys;               // the warp's keys in the tile
      const int i0 = v0 + tile * kCachedKeys;           // the tile's keys in the list
      // ---- S = Q K^T
      float s[KN][4];
#pragma unroll
      for (int n = 0; n < KN; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
      for (int ks = 0; ks < DP / 16; ++ks) {
#pragma unroll
        for (int n = 0; n < KN; n += 2) {
          // rows: 16 keys; matrices (keys 0-7, dims 0-7), (0-7, 8-15), (8-15, 0-7), (8-15, 8-15)
          const int r = key0 + n * 8 + (lane & 7) + ((lane >> 4) & 1) * 8;
          const int c = ks * 2 + ((lane >> 3) & 1);
          uint32_t kf[4];
          ldmatrix_x4(ks_s + static_cast<uint32_t>(r * DP * 2 + (swizzled<CH>(r, c) << 4)), kf);
          mma_16816<T>(s[n], qf[ks], kf[0], kf[1]);
          mma_16816<T>(s[n + 1], qf[ks], kf[2], kf[3]);
        }
      }
      // ---- masks: rows differ in what they see at the window's edge and
      // among the new tokens; behind the share nothing is seen
      const int last = i0 + kCachedKeys - 1;
      const bool rows_differ = w.n_queries > 1 &&
          ((last >= sp.sinks && sp.key(last) >= sp.base) ||
           (last >= sp.sinks && sp.key(max(i0, sp.sinks)) <= sp.base + w.n_queries - 1 - w.window));
      if (rows_differ || last >= v1) {
#pragma unroll
        for (int n = 0; n < KN; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = i0 + key0 + n * 8 + (lane & 3) * 2 + (e & 1);
            bool see = i < v1;
            if (rows_differ && see) {
              const int j = sp.key(i), u = j - sp.base;
              const int at = u >= 0 ? kpos[u] : j;
              see = (u < 0 || ((word[e >> 1] >> u) & 1)) && (at > lo[e >> 1] || at < sk[e >> 1]);
            }
            if (!see) s[n][e] = -INFINITY;
          }
      }
      // ---- online softmax, two rows a thread, four threads a row; a row is
      // rescaled once its maximum grew by more than 2^8 (exact after the final 1 / l)
      float alpha[2];
      bool grew = false;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float a = -INFINITY;
#pragma unroll
        for (int n = 0; n < KN; ++n) a = ptx::max3(a, s[n][2 * e], s[n][2 * e + 1]);
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
        a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
        const bool more = a * p.scale_log2 > m[e] + kLazyLog2;
        const float mn = more ? a * p.scale_log2 : m[e];
        const float ref = mn == -INFINITY ? 0.0f : mn;
        alpha[e] = more ? ptx::ex2_approx(m[e] - ref) : 1.0f;
        m[e] = mn;
        grew |= more;
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < KN; ++n)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const float x = ptx::ex2_approx(fmaf(s[n][2 * e + f], p.scale_log2, kWeightLog2<T> - ref));
            sum += x;
            s[n][2 * e + f] = x;
          }
        l[e] = fmaf(l[e], alpha[e], sum);  // of this thread's columns
      }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int n = 0; n < DP / 8; ++n) {
          o[n][0] *= alpha[0];
          o[n][1] *= alpha[0];
          o[n][2] *= alpha[1];
          o[n][3] *= alpha[1];
        }
      }
      // ---- O += P V
      bool loops = false;
      if (rows_differ) {
        bool bad = false;
        constexpr uint32_t kExp = Elem<T>::kBf16 ? 0x7f80u : 0x7c00u;
        for (int x = lane; x < P::kWarpKeys * CH; x += 32) {
          const int r = key0 + x / CH, c = x % CH;
          if (c * 8 >= D) continue;
          const float4 y = ptx::ld_shared_v4(vs_s + static_cast<uint32_t>(r * DP * 2 + (swizzled<CH>(r, c) << 4)));
          const uint32_t z[4] = {__float_as_uint(y.x), __float_as_uint(y.y), __float_as_uint(y.z), __float_as_uint(y.w)};
#pragma unroll
          for (int f = 0; f < 4; ++f)
            bad |= (z[f] & kExp) == kExp || ((z[f] >> 16) & kExp) == kExp;
        }
        loops = __any_sync(0xffffffffu, bad);
      }
      if (!loops) {
#pragma unroll
        for (int kk = 0; kk < KN / 2; ++kk) {
          uint32_t pf[4] = {pack2<T>(s[2 * kk][0], s[2 * kk][1]), pack2<T>(s[2 * kk][2], s[2 * kk][3]),
                            pack2<T>(s[2 * kk + 1][0], s[2 * kk + 1][1]), pack2<T>(s[2 * kk + 1][2], s[2 * kk + 1][3])};
          // rows: 16 keys; matrices (keys 0-7, dims 0-7), (8-15, 0-7), (0-7, 8-15), (8-15, 8-15)
          const int r = key0 + kk * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
          for (int n = 0; n < DP / 8; n += 2) {
            const int c = n + (lane >> 4);
            uint32_t vf[4];
            ldmatrix_x4_trans(vs_s + static_cast<uint32_t>(r * DP * 2 + (swizzled<CH>(r, c) << 4)), vf);
            mma_16816<T>(o[n], pf, vf[0], vf[1]);
            mma_16816<T>(o[n + 1], pf, vf[2], vf[3]);
          }
        }
      } else {
        // weights by key in shared memory, -1 where a row does not see the key
        float* pw = reinterpret_cast<float*>(smem + P::kOffP) + warp * 16 * P::kWarpKeys;
#pragma unroll
        for (int n = 0; n < KN; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = i0 + key0 + n * 8 + (lane & 3) * 2 + (e & 1);
            bool see = i < v1;
            if (see) {
              const int j = sp.key(i), u = j - sp.base;
              const int at = u >= 0 ? kpos[u] : j;
              see = (u < 0 || ((word[e >> 1] >> u) & 1)) && (at > lo[e >> 1] || at < sk[e >> 1]);
            }
            pw[((lane >> 2) + 8 * (e >> 1)) * P::kWarpKeys + n * 8 + (lane & 3) * 2 + (e & 1)] = see ? s[n][e] : -1.0f;
          }
        __syncwarp();
        for (int x = 0; x < P::kWarpKeys; ++x) {
          const float pa = pw[(lane >> 2) * P::kWarpKeys + x], pb = pw[((lane >> 2) + 8) * P::kWarpKeys + x];
          const int r = key0 + x;
#pragma unroll
          for (int n = 0; n < DP / 8; ++n) {
            if (n * 8 >= D) break;
            const T* vv = reinterpret_cast<const T*>(smem + (vs_s - smem_s) + r * DP * 2 + (swizzled<CH>(r, n) << 4)) + (lane & 3) * 2;
            const float va = Elem<T>::widen(vv[0]), vb = Elem<T>::widen(vv[1]);
            if (!(pa < 0.0f)) {
              o[n][0] = fmaf(pa, va, o[n][0]);
              o[n][1] = fmaf(pa, vb, o[n][1]);
            }
            if (!(pb < 0.0f)) {
              o[n][2] = fmaf(pb, va, o[n][2]);
              o[n][3] = fmaf(pb, vb, o[n][3]);
            }
          }
        }
        __syncwarp();
      }
    }
    ptx::cp_async_wait<0>();
    __syncthreads();  // the ring is free: the warps' results go there

    // ---- join the warps that shared the keys
    float* res = reinterpret_cast<float*>(smem);  // [warp][16][DP + 2]
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      float* to = res + (warp * 16 + (lane >> 2) + 8 * e) * (DP + 2);
#pragma unroll
      for (int n = 0; n < DP / 8; ++n)
        *reinterpret_cast<float2*>(to + n * 8 + (lane & 3) * 2) = make_float2(o[n][2 * e], o[n][2 * e + 1]);
      if ((lane & 3) == 0) *reinterpret_cast<float2*>(to + DP) = make_float2(m[e], l[e]);
    }
    __syncthreads();
    const bool alone = p.splits == 1 || (shares == 1 && !clustered);
    for (int x = tid; x < 16 * RW * (D / 8); x += kThreads) {
      const int r = x / (D / 8), d = x % (D / 8) * 8;
      const int rr = rb * 16 * RW + r;
      if (rr >= p.rows) continue;
      float* from = res + r * (DP + 2);  // warp r / 16, + RW for the next key share
      float mx = -INFINITY;
#pragma unroll
      for (int y = 0; y < P::kKw; ++y) mx = fmaxf(mx, from[y * RW * 16 * (DP + 2) + DP]);
      const float ref = mx == -INFINITY ? 0.0f : mx;
      float sum = 0.0f, acc[8] = {};
#pragma unroll
      for (int y = 0; y < P::kKw; ++y) {
        const float* f = from + y * RW * 16 * (DP + 2);
        const float a = ptx::ex2_approx(f[DP] - ref);
        sum = fmaf(a, f[DP + 1], sum);
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(a, f[d + e], acc[e]);
      }
      if (clustered) {  // in place of the first key share's
#pragma unroll
        for (int e = 0; e < 8; e += 2) *reinterpret_cast<float2*>(from + d + e) = make_float2(acc[e], acc[e + 1]);
        continue;
      }
      const int t = rr / w.group;
      if (alone) {
        const bool none = sum == 0.0f || cached_word(w, b, t, sp.base) == 0;
        const float inv = 1.0f / sum;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = none ? 0.0f : acc[e] * inv;
        reinterpret_cast<Vec<T, 8>*>(rows_at_mut<T>(p.out, b, kh * w.group + (rr - t * w.group), t) + d)->narrow(acc);
      } else {
        const long long at = ((bk * p.row_blocks + rb) * p.splits + split) * 16 * RW + r;
        float4* to = reinterpret_cast<float4*>(p.part_o + at * D + d);
        to[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
        to[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (d == 0) *reinterpret_cast<float2*>(p.part_ml + at * 2) = make_float2(mx, sum);
      }
    }
    if (!clustered) continue;
    __syncthreads();
    if (tid < 16 * RW) {
      float* row = res + tid * (DP + 2);
      float mx = -INFINITY, sum = 0.0f;
#pragma unroll
      for (int y = 0; y < P::kKw; ++y) mx = fmaxf(mx, row[y * RW * 16 * (DP + 2) + DP]);
      const float ref = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
      for (int y = 0; y < P::kKw; ++y) {
        const float* f = row + y * RW * 16 * (DP + 2) + DP;
        sum = fmaf(ptx::ex2_approx(f[0] - ref), f[1], sum);
      }
      *reinterpret_cast<float2*>(row + DP) = make_float2(mx, sum);
    }
    ptx::cluster_sync();
    for (int x = split * kThreads + tid; x < 16 * RW * (D / 8); x += p.splits * kThreads) {
      const int r = x / (D / 8), d = x % (D / 8) * 8;
      const int rr = rb * 16 * RW + r;
      if (rr >= p.rows) continue;
      const uint32_t row = smem_s + static_cast<uint32_t>(r * (DP + 2) * 4);
      float2 ml[kCachedCluster];
      float mx = -INFINITY;
#pragma unroll
      for (int s = 0; s < kCachedCluster; ++s) {
        ml[s] = s < shares ? ptx::ld_cluster_v2(ptx::cluster_map(row + DP * 4, s)) : make_float2(-INFINITY, 0.0f);
        mx = fmaxf(mx, ml[s].x);
      }
      const float ref = mx == -INFINITY ? 0.0f : mx;
      float sum = 0.0f, acc[8] = {};
#pragma unroll
      for (int s = 0; s < kCachedCluster; ++s) {
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
      const int t = rr / w.group;
      const bool none = sum == 0.0f || cached_word(w, b, t, sp.base) == 0;
      const float inv = 1.0f / sum;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = none ? 0.0f : acc[e] * inv;
      reinterpret_cast<Vec<T, 8>*>(rows_at_mut<T>(p.out, b, kh * w.group + (rr - t * w.group), t) + d)->narrow(acc);
    }
    ptx::cluster_sync();  // before the shared memory that others read goes
  }
  ptx::grid_dep_launch();
}

// Merges the shares of a row, one block per row: the weight of every share
// first, then the four warps add a quarter of the shares each (4 dims a
// lane), in a fixed order.
template <typename T, int RW>
__global__ void __launch_bounds__(128) vattn_cached_join_kernel(const __grid_constant__ CachedParams p) {
  __shared__ float weight[kCachedMaxSplits];
  __shared__ float red[8];
  __shared__ float4 acc_s[4][32];
  const WindowParams& w = p.w;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, D = w.dim;
  const long long bk = blockIdx.x / p.rows;
  const int rr = static_cast<int>(blockIdx.x - bk * p.rows);
  const int b = static_cast<int>(bk / w.kv_heads), kh = static_cast<int>(bk - static_cast<long long>(b) * w.kv_heads);
  const int t = rr / w.group;
  ptx::grid_dep_wait();
  const CachedSpan sp = CachedSpan::make(w, b, p.splits);
  const int shares = sp.shares();
  if (shares == 1) return;  // written by its block
  const bool none = cached_word(w, b, t, sp.base) == 0;
  const long long at0 = (bk * p.row_blocks + rr / (16 * RW)) * p.splits * 16 * RW + rr % (16 * RW);
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + at0;
  float mx = -INFINITY;
  for (int s = tid; s < shares; s += 128) mx = fmaxf(mx, ml[s * 16LL * RW].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (lane == 0) red[warp] = mx;
  __syncthreads();
  mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float ref = mx == -INFINITY ? 0.0f : mx;
  float sum = 0.0f;
  for (int s = tid; s < shares; s += 128) {
    const float2 f = ml[s * 16LL * RW];
    const float a = ptx::ex2_approx(f.x - ref);
    weight[s] = a;
    sum = fmaf(a, f.y, sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if (lane == 0) red[4 + warp] = sum;
  __syncthreads();
  sum = (red[4] + red[5]) + (red[6] + red[7]);
  float acc[4] = {};
  if (lane * 4 < D) {
    const float* from = p.part_o + at0 * D + lane * 4;
#pragma unroll 8
    for (int s = warp; s < shares; s += 4) {
      const float4 f = *reinterpret_cast<const float4*>(from + s * 16LL * RW * D);
      const float a = weight[s];
      acc[0] = fmaf(a, f.x, acc[0]);
      acc[1] = fmaf(a, f.y, acc[1]);
      acc[2] = fmaf(a, f.z, acc[2]);
      acc[3] = fmaf(a, f.w, acc[3]);
    }
  }
  acc_s[warp][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
  __syncthreads();
  if (warp != 0 || lane * 4 >= D) return;
  const float inv = 1.0f / sum;
#pragma unroll
  for (int k = 1; k < 4; ++k) {
    const float4 f = acc_s[k][lane];
    acc[0] += f.x;
    acc[1] += f.y;
    acc[2] += f.z;
    acc[3] += f.w;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) acc[e] = none || sum == 0.0f ? 0.0f : acc[e] * inv;
  reinterpret_cast<Vec<T, 4>*>(rows_at_mut<T>(p.out, b, kh * w.group + (rr - t * w.group), t) + lane * 4)->narrow(acc);
}

}  // namespace vattn
