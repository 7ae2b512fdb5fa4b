// paged_kernel.cuh -- attention of a few new tokens over the 8-bit paged cache
// (vattn_forward_paged).
//
// Memory bound: every visible key and value, one byte an element, is read once for
// all rows (new token, query head of the group) of its key head together.  A
// block takes up to 16 RW rows and a share of the keys, 64 at a time:
//   last warp   boxes of G rows of one page (G = 64, 32 or 16, what divides the page)
//               by TMA into a ring, with the page's scales beside them; the table's
//               entries and scales come 32 boxes at a time, ahead of the copies
//   the others  RW groups of warps with 16 rows each; the warps of a group share
//               the tile's keys by 16 (RW = 4: 32)
//
// The products are mma.sync m16n8k16 in f16, whose 16 rows fit the few there are.
// An e4m3 value is an f16 value, so keys and values enter exactly, converted in
// registers; so does q, a bf16 row times the power of two that takes its largest to
// 2^14 .. 2^15 (f16 as it is).  K: the four consecutive bytes that ldmatrix gives
// a lane are taken as elements 2 c, 2 c + 1, 2 c + 8, 2 c + 9 of the product's
// 16 (c = lane % 4), and q is laid out alike, so nothing moves between lanes.  V:
// ldmatrix.trans gives bytes of two keys and two dims; a byte permutation makes
// them pairs of keys, and an n-block's eight columns are every other dim of 16.
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

constexpr int kPagedKeys = 64;  // keys of a tile

struct PagedParams {
  WindowParams w;  // n_keys: rows that the table has room for; kv_len: the cache's
  RowsTensor q, out;
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  uint32_t* status;
  float* part_o;   // [sequence and key head][row block][split][16 RW][dim]
  float* part_ml;  // ... [16 RW][2]: maximum (log2 units) and sum
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
  int per, n;       // boxes of a share (whole tiles), of all

  __device__ __forceinline__ static PagedSpan make(const WindowParams& w, int log_box, int b, int splits) {
    PagedSpan s;
    const int box = 1 << log_box;
    s.len = min(max(w.kv_len[b], 0), w.n_keys);
    s.base = s.len - w.n_queries;
    s.first = max(0, s.base - w.window + 1);
    s.begin = s.first >> log_box;
    s.heads = min((min(w.sinks, s.len) + box - 1) >> log_box, s.begin);
    s.n = s.heads + ((s.len + box - 1) >> log_box) - s.begin;
    const int tile = kPagedKeys >> log_box;
    s.per = ((s.n + splits - 1) / splits + tile - 1) / tile * tile;
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

template <int DP, int RW>
struct PagedPlan {
  static constexpr int kMath = RW == 1 ? 4 : 8;  // math warps
  static constexpr int kThreads = 32 * (kMath + 1);
  static constexpr int kKw = kMath / RW;  // warps that share a tile's keys
  static constexpr int kWarpKeys = kPagedKeys / kKw;
  static constexpr int kTileBytes = kPagedKeys * DP;
  static constexpr int kStageBytes = 2 * kTileBytes;
  static constexpr int kStages = DP == 128 ? 4 : 6;
  static constexpr int kResultStride = DP + 4;  // floats of a row: O, maximum, sum
  static constexpr int kResultBytes = kMath * 16 * kResultStride * 4;
  static constexpr int kRingBytes = kStages * kStageBytes;
  static constexpr int kOffW = kRingBytes > kResultBytes ? kRingBytes : kResultBytes;  // weights of the loops' path
  static constexpr int kOffMeta = kOffW + kMath * 16 * 16 * 4;  // [stage][4] scales of a tile's boxes
  static constexpr int kOffBar = kOffMeta + kStages * 64;
  static constexpr int kSmemBytes = kOffBar + 16 * kStages + 32 + 1024;  // + alignment slack
};

template <typename T, int DP, int RW>
__global__ void __launch_bounds__(PagedPlan<DP, RW>::kThreads)
    vattn_paged_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ PagedParams p) {
  using P = PagedPlan<DP, RW>;
  constexpr int CH = DP / 16;  // 16-byte chunks of a shared row, 16-element steps of a product
  constexpr int RS = P::kResultStride;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int kpos[VATTN_MAX_NEW_TOKENS];
  const uint32_t raw_s = ptx::smem_addr(smem_raw);
  const uint32_t smem_s = (raw_s + 1023u) & ~1023u;
  uint8_t* const smem = smem_raw + (smem_s - raw_s);
  const uint32_t bar0 = smem_s + P::kOffBar;
  auto full = [bar0](int st) -> uint32_t { return bar0 + 8u * st; };
  auto empty = [bar0](int st) -> uint32_t { return bar0 + 8u * (P::kStages + st); };
  const Pipe pipe{bar0 + 16u * P::kStages};
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const WindowParams& w = p.w;
  const int D = w.dim;
  uint32_t split_u, rb_u, kh_u;
  const uint32_t bk = p.d_row_blocks.div(p.d_splits.div(blockIdx.x, &split_u), &rb_u);
  const int b = static_cast<int>(p.d_kv_heads.div(bk, &kh_u));
  const int split = static_cast<int>(split_u), rb = static_cast<int>(rb_u), kh = static_cast<int>(kh_u);
  const bool clustered = p.splits > 1 && p.splits <= kCachedCluster;

  if (tid == 0) {
    for (int i = 0; i < P::kStages; ++i) {
      ptx::mbar_init(full(i), 1);
      ptx::mbar_init(empty(i), P::kMath);
    }
    pipe.init(w, p.status);
    ptx::fence_mbar_init();
    ptx::prefetch_tensormap(&tm_k);
    ptx::prefetch_tensormap(&tm_v);
  }
  ptx::grid_dep_wait();
  const PagedSpan sp = PagedSpan::make(w, p.log_box, b, p.splits);
  const int v0 = split * sp.per, v1 = min(sp.n, v0 + sp.per);
  const int shares = sp.shares();
  if (!clustered && split >= shares) return;  // (in a cluster: with no keys, but at its barriers)
  if (tid < w.n_queries) kpos[tid] = sp.base + __popcll(cached_word(w, b, tid, sp.base)) - 1;
  __syncthreads();
  const int per_tile = kPagedKeys >> p.log_box;  // boxes
  const int tiles = (max(v1 - v0, 0) + per_tile - 1) / per_tile;

  if (warp == P::kMath) {
    // ------------------------------------------------------ boxes into the ring
    auto entry = [&](int i) -> int {  // page of box i, -1 if it is not there
      if (i >= v1) return -1;
      const int id = p.table[static_cast<long long>(b) * p.max_pages + p.d_page.div(static_cast<uint32_t>(sp.box(i) << p.log_box))];
      return id >= 0 && id < p.n_pages ? id : -1;
    };
    struct Scales {
      float k, log2_v, inv_v;
    };
    auto scales = [&](int id) {
      Scales s{-1.0f, 0.0f, 0.0f};  // k < 0: the keys are not there
      if (id < 0) return s;
      const long long at = static_cast<long long>(id) * w.kv_heads + kh;
      const float v = p.v_scale[at];
      s.k = p.k_scale[at];
      s.log2_v = log2f(v);
      s.inv_v = 1.0f / v;
      return s;
    };
    const uint64_t once = ptx::policy_evict_first();
    int id = entry(v0 + lane);
    Scales sc = scales(id);
    bool ok = true;
    int t = 0;
    for (int at = v0; ok && at < v1; at += 32) {  // 32 boxes: 8 tiles or more
      const int next = entry(at + 32 + lane);
      for (int i = 0; ok && i < 32 && at + i < v1; i += per_tile, ++t) {
        const int st = t % P::kStages;
        if (!(ok = pipe.wait_warp(empty(st), static_cast<uint32_t>((t / P::kStages) & 1) ^ 1u, kSitePagedLoad))) break;
        const int boxes = min(per_tile, v1 - (at + i));
        if (lane >= i && lane < i + boxes)
          ptx::st_shared_v4(smem_s + P::kOffMeta + st * 64 + (lane - i) * 16, sc.k, sc.log2_v, sc.inv_v, 0.0f);
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_expect_tx(full(st), static_cast<uint32_t>(boxes) * 2u * static_cast<uint32_t>(p.box * DP));
        __syncwarp();
        if (lane >= i && lane < i + boxes) {
          const int key0 = sp.box(at + lane) << p.log_box;
          const int row = key0 - static_cast<int>(p.d_page.div(static_cast<uint32_t>(key0))) * p.page;
          const uint32_t to = smem_s + st * P::kStageBytes + static_cast<uint32_t>((lane - i) * p.box * DP);
          // a page that is not there reads as zeros: behind the last
          const int pg = id >= 0 ? id : static_cast<int>(p.n_pages);
          ptx::tma_load_4d_hint(to, &tm_k, full(st), 0, row, kh, pg, once);
          ptx::tma_load_4d_hint(to + P::kTileBytes, &tm_v, full(st), 0, row, kh, pg, once);
        }
        __syncwarp();
      }
      id = next;
      sc = scales(id);
    }
    if (!ok && lane == 0)  // the copies in flight land before the block exits
      for (int d = max(0, t - P::kStages); d < t; ++d)
        pipe.drain(full(d % P::kStages), static_cast<uint32_t>((d / P::kStages) & 1), kSitePagedDrain);
    __syncwarp();
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  float o[CH][2][4];  // [16 dims][even, odd][C fragment]
#pragma unroll
  for (int n = 0; n < CH; ++n)
#pragma unroll
    for (int e = 0; e < 8; ++e) o[n][e >> 2][e & 3] = 0.0f;

  if (warp < P::kMath) {
    const int rw = warp % RW, kw = warp / RW, c4 = lane & 3;
    // ---- the warp's 16 rows: lane / 4 and lane / 4 + 8
    uint32_t qf[CH][4];
    int lo[2], sk[2];
    uint64_t word[2];
    float row_c[2];  // from a product's sum to log2 units, but for the key's scale
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int rr = rb * 16 * RW + rw * 16 + (lane >> 2) + 8 * e;
      uint32_t g;
      const int t = static_cast<int>(p.d_group.div(static_cast<uint32_t>(rr), &g));
      word[e] = rr < p.rows ? cached_word(w, b, t, sp.base) : 0;
      const T* qrow = word[e] != 0 ? rows_at<T>(p.q, b, kh * w.group + static_cast<int>(g), t) : nullptr;
      lo[e] = word[e] != 0 ? sp.base + __popcll(word[e]) - 1 - w.window : 0x7fffffff;
      sk[e] = word[e] != 0 ? w.sinks : 0;
      row_c[e] = p.scale_log2;
      float y[CH][4];
      float most = 0.0f;
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
        row_c[e] = p.scale_log2 * __int_as_float((127 - k) << 23);
#pragma unroll
        for (int ks = 0; ks < CH; ++ks)
#pragma unroll
          for (int f = 0; f < 4; ++f) y[ks][f] *= by;
      }
#pragma unroll
      for (int ks = 0; ks < CH; ++ks) {
        qf[ks][e] = pack2<__half>(y[ks][0], y[ks][1]);
        qf[ks][e + 2] = pack2<__half>(y[ks][2], y[ks][3]);
      }
    }

    for (int tile = 0; tile < tiles; ++tile) {
      const int st = tile % P::kStages;
      if (!pipe.wait_warp(full(st), static_cast<uint32_t>((tile / P::kStages) & 1), kSitePagedMath)) break;
      const uint32_t ks_s = smem_s + static_cast<uint32_t>(st) * P::kStageBytes;
      const uint32_t vs_s = ks_s + P::kTileBytes;
#pragma unroll 1
      for (int sub = 0; sub < P::kWarpKeys / 16; ++sub) {
        const int key0 = kw * P::kWarpKeys + sub * 16;      // the 16 keys in the tile
        const int x = key0 >> p.log_box, i = v0 + tile * per_tile + x;
        if (i >= v1) break;
        const float4 meta = ptx::ld_shared_v4(smem_s + P::kOffMeta + st * 64 + x * 16);
        if (meta.x < 0.0f) continue;
        const int j0 = (sp.box(i) << p.log_box) + (key0 & (p.box - 1)), j1 = j0 + 15;  // and in the sequence
        if (j0 >= sp.len || (j0 >= w.sinks && j1 < sp.first)) continue;
        // ---- S = Q K^T
        float s[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[n][e] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < CH; ks += 2) {
          // matrices (keys 0-7, dims 0-15 of 16 ks), (0-7, 16-31), (8-15, 0-15), (8-15, 16-31)
          const int r = key0 + (lane & 7) + ((lane >> 4) & 1) * 8, c = ks + ((lane >> 3) & 1);
          uint32_t kf[4];
          ldmatrix_x4(ks_s + static_cast<uint32_t>(r * DP + (paged_swizzled<CH>(r, c) << 4)), kf);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            mma_16816<__half>(s[0], qf[ks + y], e4m3_half2_lo(kf[y]), e4m3_half2_hi(kf[y]));
            mma_16816<__half>(s[1], qf[ks + y], e4m3_half2_lo(kf[2 + y]), e4m3_half2_hi(kf[2 + y]));
          }
        }
        // ---- masks: at the sequence's end, the first keys' end, the window's edge, among the new tokens
        auto sees = [&](int e, int j) {
          const int u = j - sp.base;
          const int at = u >= 0 && j < sp.len ? kpos[u] : j;
          return j < sp.len && (u < 0 || ((word[e] >> u) & 1)) && (at > lo[e] || at < sk[e]);
        };
        const bool masked = j1 >= sp.len || (w.n_queries > 1 && j1 >= sp.base) ||
                            (j1 >= w.sinks && (j0 < sp.first || (w.n_queries > 1 && j0 <= sp.base + w.n_queries - 1 - w.window)));
        if (masked) {
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!sees(e >> 1, j0 + n * 8 + c4 * 2 + (e & 1))) s[n][e] = -INFINITY;
        }
        // ---- online softmax, two rows a thread, four threads a row; a row is
        // rescaled once its maximum grew by more than 2^8 (exact after the final 1 / l)
        float alpha[2];
        bool grew = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float c = fminf(fmaxf(row_c[e] * meta.x, 0x1p-126f), 0x1p127f);  // not 0 or infinity, which -infinity or 0 make NaN
          float a = ptx::max3(s[0][2 * e], s[0][2 * e + 1], fmaxf(s[1][2 * e], s[1][2 * e + 1]));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 1));
          a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, 2));
          const float top = fmaf(a, c, meta.y);
          const bool more = top > m[e] + kLazyLog2;
          const float mn = more ? top : m[e];
          const float ref = mn == -INFINITY ? 0.0f : mn;
          alpha[e] = more ? ptx::ex2_approx(m[e] - ref) : 1.0f;
          m[e] = mn;
          grew |= more;
          const float shift = kWeightLog2<__half> - ref + meta.y;
          float sum = 0.0f;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int f = 0; f < 2; ++f) {
              const float y = ptx::ex2_approx(fmaf(s[n][2 * e + f], c, shift));
              sum += y;
              s[n][2 * e + f] = y;
            }
          l[e] = fmaf(l[e], alpha[e], sum * meta.z);  // of this thread's columns
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int n = 0; n < CH; ++n)
#pragma unroll
            for (int e = 0; e < 8; ++e) o[n][e >> 2][e & 3] *= alpha[(e >> 1) & 1];
        }
        // ---- O += P V
        bool loops = false;
        if (masked) {
          // rows that no query sees may hold anything: zeros; a NaN in another
          // that some do not see: loops over the visible pairs
          bool bad = false;
          for (int y = lane; y < 16 * CH; y += 32) {
            const int r = y / CH, c = y % CH, j = j0 + r;
            const uint32_t at = vs_s + static_cast<uint32_t>((key0 + r) * DP + (paged_swizzled<CH>(key0 + r, c) << 4));
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
          const uint32_t pf[4] = {pack2<__half>(s[0][0], s[0][1]), pack2<__half>(s[0][2], s[0][3]),
                                  pack2<__half>(s[1][0], s[1][1]), pack2<__half>(s[1][2], s[1][3])};
#pragma unroll
          for (int n = 0; n < CH; n += 2) {
            // matrices (keys 0-7, dims 0-15 of 16 n), (8-15, 0-15), (0-7, 16-31), (8-15, 16-31)
            const int r = key0 + (lane & 7) + ((lane >> 3) & 1) * 8, c = n + (lane >> 4);
            uint32_t vf[4];
            ldmatrix_x4_trans(vs_s + static_cast<uint32_t>(r * DP + (paged_swizzled<CH>(r, c) << 4)), vf);
#pragma unroll
            for (int y = 0; y < 4; ++y) vf[y] = __byte_perm(vf[y], 0u, 0x3120);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              mma_16816<__half>(o[n + y][0], pf, e4m3_half2_lo(vf[2 * y]), e4m3_half2_lo(vf[2 * y + 1]));
              mma_16816<__half>(o[n + y][1], pf, e4m3_half2_hi(vf[2 * y]), e4m3_half2_hi(vf[2 * y + 1]));
            }
          }
        } else {
          // weights by key in shared memory, -1 where a row does not see the key
          float* pw = reinterpret_cast<float*>(smem + P::kOffW) + warp * 16 * 16;
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int y = n * 8 + c4 * 2 + (e & 1);
              pw[((lane >> 2) + 8 * (e >> 1)) * 16 + y] = sees(e >> 1, j0 + y) ? s[n][e] : -1.0f;
            }
          __syncwarp();
#pragma unroll 1
          for (int y = 0; y < 16; ++y) {
            const float pa = pw[(lane >> 2) * 16 + y], pb = pw[((lane >> 2) + 8) * 16 + y];
            const int r = key0 + y;
#pragma unroll
            for (int n = 0; n < CH; ++n) {
              const uint32_t z = *reinterpret_cast<const uint32_t*>(
                  smem + (vs_s - smem_s) + r * DP + (paged_swizzled<CH>(r, n) << 4) + c4 * 4);
              const uint32_t z01 = e4m3_half2_lo(z), z23 = e4m3_half2_hi(z);
              const float2 v01 = __half22float2(*reinterpret_cast<const __half2*>(&z01));
              const float2 v23 = __half22float2(*reinterpret_cast<const __half2*>(&z23));
              if (!(pa < 0.0f)) {
                o[n][0][0] = fmaf(pa, v01.x, o[n][0][0]);
                o[n][1][0] = fmaf(pa, v01.y, o[n][1][0]);
                o[n][0][1] = fmaf(pa, v23.x, o[n][0][1]);
                o[n][1][1] = fmaf(pa, v23.y, o[n][1][1]);
              }
              if (!(pb < 0.0f)) {
                o[n][0][2] = fmaf(pb, v01.x, o[n][0][2]);
                o[n][1][2] = fmaf(pb, v01.y, o[n][1][2]);
                o[n][0][3] = fmaf(pb, v23.x, o[n][0][3]);
                o[n][1][3] = fmaf(pb, v23.y, o[n][1][3]);
              }
            }
          }
          __syncwarp();
        }
      }
      pipe_warp_arrive(empty(st));
    }
  }
  __syncthreads();  // the ring is free: the warps' results go there

  // ---- join the warps that shared the keys
  float* res = reinterpret_cast<float*>(smem);  // [warp][16][RS]
  if (warp < P::kMath) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      float* to = res + (warp * 16 + (lane >> 2) + 8 * e) * RS;
#pragma unroll
      for (int n = 0; n < CH; ++n)
        *reinterpret_cast<float4*>(to + n * 16 + (lane & 3) * 4) =
            make_float4(o[n][0][2 * e], o[n][1][2 * e], o[n][0][2 * e + 1], o[n][1][2 * e + 1]);
      if ((lane & 3) == 0) *reinterpret_cast<float2*>(to + DP) = make_float2(m[e], l[e]);
    }
  }
  __syncthreads();
  auto write = [&](int rr, int d, float sum, float (&acc)[8]) {
    uint32_t g;
    const int t = static_cast<int>(p.d_group.div(static_cast<uint32_t>(rr), &g));
    const bool none = sum == 0.0f || cached_word(w, b, t, sp.base) == 0;
    const float inv = 1.0f / sum;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] = none ? 0.0f : acc[e] * inv;
    reinterpret_cast<Vec<T, 8>*>(rows_at_mut<T>(p.out, b, kh * w.group + static_cast<int>(g), t) + d)->narrow(acc);
  };
  const bool alone = p.splits == 1 || (shares == 1 && !clustered);
  const int per_row = D / 8;
  for (int x = tid; x < 16 * RW * per_row; x += P::kThreads) {
    const int r = x / per_row, d = (x - r * per_row) * 8;
    const int rr = rb * 16 * RW + r;
    if (rr >= p.rows) continue;
    float* from = res + r * RS;  // warp r / 16, + RW for the next key share
    float mx = -INFINITY;
#pragma unroll
    for (int y = 0; y < P::kKw; ++y) mx = fmaxf(mx, from[y * RW * 16 * RS + DP]);
    const float ref = mx == -INFINITY ? 0.0f : mx;
    float sum = 0.0f, acc[8] = {};
#pragma unroll
    for (int y = 0; y < P::kKw; ++y) {
      const float* f = from + y * RW * 16 * RS;
      const float a = ptx::ex2_approx(f[DP] - ref);
      sum = fmaf(a, f[DP + 1], sum);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(a, f[d + e], acc[e]);
    }
    if (clustered) {  // in place of the first key share's
#pragma unroll
      for (int e = 0; e < 8; e += 4) *reinterpret_cast<float4*>(from + d + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
    } else if (alone) {
      write(rr, d, sum, acc);
    } else {
      const long long at = ((static_cast<long long>(bk) * p.row_blocks + rb) * p.splits + split) * 16 * RW + r;
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
  if (tid < 16 * RW) {
    float* row = res + tid * RS;
    float mx = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int y = 0; y < P::kKw; ++y) mx = fmaxf(mx, row[y * RW * 16 * RS + DP]);
    const float ref = mx == -INFINITY ? 0.0f : mx;
#pragma unroll
    for (int y = 0; y < P::kKw; ++y) {
      const float* f = row + y * RW * 16 * RS + DP;
      sum = fmaf(ptx::ex2_approx(f[0] - ref), f[1], sum);
    }
    *reinterpret_cast<float2*>(row + DP) = make_float2(mx, sum);
  }
  ptx::cluster_sync();
  for (int x = split * P::kThreads + tid; x < 16 * RW * per_row; x += p.splits * P::kThreads) {
    const int r = x / per_row, d = (x - r * per_row) * 8;
    const int rr = rb * 16 * RW + r;
    if (rr >= p.rows) continue;
    const uint32_t row = smem_s + static_cast<uint32_t>(r * RS * 4);
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
    write(rr, d, sum, acc);
  }
  ptx::cluster_sync();  // before the shared memory that others read goes
  ptx::grid_dep_launch();
}

// Merges the shares of a row, one block per row: the weight of every share
// first, then the four warps add a quarter of the shares each (4 dims a
// lane), in a fixed order.
template <typename T, int RW>
__global__ void __launch_bounds__(128) vattn_paged_join_kernel(const __grid_constant__ PagedParams p) {
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
  const PagedSpan sp = PagedSpan::make(w, p.log_box, b, p.splits);
  const int shares = sp.shares();
  if (shares == 1) return;  // written by its block
  const bool none = cached_word(w, b, t, sp.base) == 0;
  const long long at0 = (bk * p.row_blocks + rr / (16 * RW)) * p.splits * 16 * RW + rr % (16 * RW);
  const float2* ml = reinterpret_cast<const float2*>(p.part_ml) + at0;
  float mx = -INFINITY;
  for (int s = tid; s < shares; s += 128) mx = fmaxf(mx, ml[s * 16LL * RW].x);
  mx = warp_max(mx);
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
