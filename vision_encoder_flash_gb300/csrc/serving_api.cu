// serving_api.cu -- the C ABI declared in include/vattn_serving.h: argument
// checks, variant choice and launches of the calls on packed prompts and the
// paged cache on sm_103a (paged_launch.cuh: attention over that cache).
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <type_traits>

#include "../../include/vattn_serving.h"
#include "packed_list_kernel.cuh"
#include "paged_append_kernel.cuh"
#include "pages_host.h"
#include "rope_turns.h"
#include "window_fwd_kernel.cuh"
#include "window_host.h"

namespace {

using namespace vattn::host;

// ------------------------------------------------------------ the cache
vattn_status check_pages(const vattn_pages* c, const Pools& pools, int64_t batch, int64_t heads) {
  if (c->n_pages < 0 || c->n_pages >= INT32_MAX)
    return fail(VATTN_ERR_INVALID_ARG, "n_pages %lld outside [0, 2^31 - 1)", (long long)c->n_pages);
  if (c->page_size < 16 || c->page_size > 1024 || c->page_size % 16 != 0)
    return fail(VATTN_ERR_UNSUPPORTED, "page_size %lld: a multiple of 16 from 16 to 1024 is needed",
                (long long)c->page_size);
  if (c->max_pages < 0 || c->max_pages > kMaxKeys / c->page_size)
    return fail(VATTN_ERR_UNSUPPORTED, "max_pages * page_size must stay below 2^29");
  vattn_status st;
  if ((st = check_tensor(pools.k, 16)) != VATTN_OK || (st = check_tensor(pools.v, 16)) != VATTN_OK ||
      (st = check_apart(pools.k, pools.v)) != VATTN_OK)
    return st;
  const uint64_t bytes = static_cast<uint64_t>(c->n_pages) * static_cast<uint64_t>(heads) * 4u;
  const uintptr_t ks = reinterpret_cast<uintptr_t>(c->k_scale), vs = reinterpret_cast<uintptr_t>(c->v_scale);
  if (bytes > 0) {
    if (!c->k_scale || !c->v_scale) return fail(VATTN_ERR_INVALID_ARG, "null scales");
    if ((ks | vs) & 3u) return fail(VATTN_ERR_MISALIGNED, "scales must be 4-byte aligned");
    if (ks < vs + bytes && vs < ks + bytes) return fail(VATTN_ERR_INVALID_ARG, "k_scale overlaps v_scale");
    for (const Tensor* t : {&pools.k, &pools.v})
      if ((st = check_apart_bytes(c->k_scale, bytes, "k_scale", *t)) != VATTN_OK ||
          (st = check_apart_bytes(c->v_scale, bytes, "v_scale", *t)) != VATTN_OK)
        return st;
  }
  if (batch > 0 && !c->kv_len) return fail(VATTN_ERR_INVALID_ARG, "null kv_len");
  if (batch > 0 && c->max_pages > 0 && !c->table) return fail(VATTN_ERR_INVALID_ARG, "null table");
  if ((reinterpret_cast<uintptr_t>(c->kv_len) | reinterpret_cast<uintptr_t>(c->table)) & 3u)
    return fail(VATTN_ERR_MISALIGNED, "kv_len and table must be 4-byte aligned");
  return VATTN_OK;
}

// ------------------------------------------------------------ append
vattn_status check_append(const vattn_append_args* a) {
  if (a->batch < 0 || a->n_kv_heads < 0 || a->n_tokens < 0)
    return fail(VATTN_ERR_INVALID_ARG, "negative size (batch=%lld n_kv_heads=%lld n_tokens=%lld)",
                (long long)a->batch, (long long)a->n_kv_heads, (long long)a->n_tokens);
  if (a->head_dim < 1) return fail(VATTN_ERR_INVALID_ARG, "head_dim must be >= 1");
  if (a->head_dim > VATTN_MAX_HEAD_DIM || a->head_dim % 16 != 0)
    return fail(VATTN_ERR_UNSUPPORTED, "head_dim %lld: a multiple of 16 up to %d is needed (16-byte rows)",
                (long long)a->head_dim, VATTN_MAX_HEAD_DIM);
  if (a->rope_dims < 0 || a->rope_dims > a->head_dim)
    return fail(VATTN_ERR_INVALID_ARG, "rope_dims %lld outside [0, head_dim = %lld]", (long long)a->rope_dims,
                (long long)a->head_dim);
  if (!(a->base > 0.0) || !std::isfinite(a->base))
    return fail(VATTN_ERR_INVALID_ARG, "base must be a finite positive number");
  if (a->dtype != VATTN_F16 && a->dtype != VATTN_BF16)
    return fail(VATTN_ERR_UNSUPPORTED, "dtype must be VATTN_F16 or VATTN_BF16");
  if (a->batch > kMaxRows || a->n_kv_heads > kMaxRows || a->n_tokens > kMaxRows ||
      (!a->cu_seqlens && a->batch * a->n_tokens > (int64_t{1} << 36)))
    return fail(VATTN_ERR_UNSUPPORTED, "sizes must stay below 2^30 each, 2^36 tokens together");
  if ((reinterpret_cast<uintptr_t>(a->cu_seqlens) | reinterpret_cast<uintptr_t>(a->positions) |
       reinterpret_cast<uintptr_t>(a->factors)) & 3u)
    return fail(VATTN_ERR_MISALIGNED, "cu_seqlens, positions and factors must be 4-byte aligned");
  return VATTN_OK;
}

template <typename T, int V, int kForm>
vattn_status append_launch(const vattn::AppendParams& p, int64_t blocks, int threads, int device, cudaStream_t stream) {
  auto kernel = vattn::vattn_append_paged_kernel<T, V, kForm>;
  static std::atomic<uint8_t> done[kMaxDevices];
  const vattn_status st = allow_smem(kernel, vattn::append_smem<V, kForm>(vattn::kAppendThreads), done, device);
  if (st != VATTN_OK) return st;
  kernel<<<static_cast<unsigned>(blocks), threads, vattn::append_smem<V, kForm>(threads), stream>>>(p);
  return launched("cache append kernel launch");
}

// ------------------------------------------------------------ packed prompts
template <typename T, int NKB, int kMode>
vattn_status packed_go(const CUtensorMap (&tm)[4], const vattn::WindowFwdParams& p, unsigned grid, int device,
                       cudaStream_t stream) {
  using P = vattn::WindowFwdPlan<NKB>;
  auto kernel = vattn::vattn_window_fwd_kernel<T, NKB, kMode>;
  static std::atomic<uint8_t> done[kMaxDevices];
  const vattn_status st = allow_smem(kernel, P::kSmemBytes, done, device);
  if (st != VATTN_OK) return st;
  if (kMode == vattn::kPackedListed)
    return launch_behind("packed attention kernel launch", kernel, dim3(grid), dim3(P::kThreads), P::kSmemBytes, stream,
                         tm[0], tm[1], tm[2], tm[3], p);
  kernel<<<grid, P::kThreads, P::kSmemBytes, stream>>>(tm[0], tm[1], tm[2], tm[3], p);
  return launched("packed attention kernel launch");
}

template <typename T, int NKB>
vattn_status packed_launch(const CUtensorMap (&tm)[4], const vattn::WindowFwdParams& p, unsigned grid, int device,
                           cudaStream_t stream) {
  return p.list != nullptr ? packed_go<T, NKB, vattn::kPackedListed>(tm, p, grid, device, stream)
                           : packed_go<T, NKB, vattn::kPackedFound>(tm, p, grid, device, stream);
}

}  // namespace

extern "C" {

vattn_status vattn_append_paged(const vattn_rows* k, const vattn_rows* v, const vattn_pages* cache,
                                const vattn_append_args* a, void* stream_ptr) {
  clear_error();
  if (!a || !cache) return fail(VATTN_ERR_INVALID_ARG, "null args or cache");
  vattn_status st = check_append(a);
  if (st != VATTN_OK) return st;
  const Pools pools(cache, a->n_kv_heads, a->head_dim);
  if ((st = check_pages(cache, pools, a->batch, a->n_kv_heads)) != VATTN_OK) return st;
  const int64_t batch = a->cu_seqlens ? std::min<int64_t>(1, a->batch) : a->batch;
  const Tensor tk{"k", k, {batch, a->n_kv_heads, a->n_tokens}, a->head_dim, 2, false},
      tv{"v", v, {batch, a->n_kv_heads, a->n_tokens}, a->head_dim, 2, false};
  const uint64_t scale_bytes = static_cast<uint64_t>(cache->n_pages) * static_cast<uint64_t>(a->n_kv_heads) * 4u;
  for (const Tensor* t : {&tk, &tv}) {
    if ((st = check_tensor(*t, 2)) != VATTN_OK || (st = check_apart(pools.k, *t)) != VATTN_OK ||
        (st = check_apart(pools.v, *t)) != VATTN_OK ||
        (st = check_apart_bytes(cache->k_scale, scale_bytes, "k_scale", *t)) != VATTN_OK ||
        (st = check_apart_bytes(cache->v_scale, scale_bytes, "v_scale", *t)) != VATTN_OK)
      return st;
  }
  if (tk.empty() || cache->n_pages == 0 || cache->max_pages == 0) return VATTN_OK;

  vattn::AppendParams p{};
  p.x[0] = rows_tensor(k);
  p.x[1] = rows_tensor(v);
  p.pool[0] = static_cast<uint8_t*>(cache->k);
  p.pool[1] = static_cast<uint8_t*>(cache->v);
  for (int i = 0; i < 3; ++i) {
    p.ps[0][i] = cache->k_stride[i];
    p.ps[1][i] = cache->v_stride[i];
  }
  p.scale[0] = cache->k_scale;
  p.scale[1] = cache->v_scale;
  p.table = cache->table;
  p.kv_len = cache->kv_len;
  p.cu = a->cu_seqlens;
  p.positions = a->positions;
  p.factors = a->factors;
  p.n_pages = cache->n_pages;
  p.batch = static_cast<int>(a->batch);
  p.heads = static_cast<int>(a->n_kv_heads);
  p.n_tokens = static_cast<int>(a->n_tokens);
  p.page = static_cast<int>(cache->page_size);
  p.max_pages = static_cast<int>(cache->max_pages);
  p.D = static_cast<int>(a->head_dim);
  p.half = static_cast<int>(a->rope_dims / 2);
  rope_turns(a->base, static_cast<int>(a->rope_dims), p.turns, p.turns_rest);
  for (int i = 0; i < p.half; ++i) p.turn[i] = vattn::qk_turn(p.turns, p.turns_rest, nullptr, i);
  // 16-byte accesses where the rotated halves and the rest are cut evenly by them, else of 8
  auto cut_by = [&](int by) {
    bool yes = p.half % by == 0 && (p.D - 2 * p.half) % (2 * by) == 0;
    for (const Tensor* t : {&tk, &tv}) {
      yes = yes && t->base() % (2 * by) == 0;
      for (int i = 0; i < 3; ++i) yes = yes && (t->size[i] <= 1 || t->t->stride[i] % by == 0);
    }
    return yes;
  };
  const int cut = cut_by(8) ? 8 : (cut_by(4) ? 4 : 1), hold = cut == 1 ? 2 : 16 / cut;
  p.slots = p.D / (2 * cut);
  // pages that n rows in a row can touch: one for the first, and for the others as if the next began
  p.items = p.n_tokens <= 1 ? 1 : (p.n_tokens - 2) / p.page + 2;
  const int64_t items = a->cu_seqlens ? a->n_tokens / p.page + 2 * a->batch : a->batch * p.items;
  const int64_t units = items * p.heads * 2;
  if (units >= kMaxRows) return fail(VATTN_ERR_UNSUPPORTED, "too many pages and heads");
  int device = 0, sms = 0;
  if ((st = current_device(&device)) != VATTN_OK) return st;
  if ((st = sm_count(device, &sms)) != VATTN_OK) return st;
  p.units = static_cast<int>(units);
  p.d_heads = fast_div(p.heads);
  p.d_items = fast_div(p.items);
  p.d_page = fast_div(p.page);
  p.d_slots = fast_div(p.slots);
  const int slots = std::min(p.page, p.n_tokens) * p.slots;
  const int threads = std::min(vattn::kAppendThreads, (slots + 32 * hold - 1) / (32 * hold) * 32);
  const bool held = slots <= threads * hold, few = held && threads <= vattn::kAppendFewThreads;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  // As many blocks as are resident at a time (80 registers a thread in the form
  // for three of them, else 128), each with as many heads of consecutive pages: a block's first rows
  // wait for three loads in a row, and a second round of blocks for a few was 12 % slower.
  // (A packed sequence touches one page more than its rows fill, seldom two.)
  const int64_t touched = a->cu_seqlens ? std::min<int64_t>(items, a->n_tokens / p.page + a->batch) : items;
  const int64_t room = static_cast<int64_t>(sms) * std::max(1, 65536 / (few && cut > 1 ? 80 : 128) / threads);
  p.per_block = static_cast<int>((touched * p.heads * 2 + room - 1) / room);
  const int64_t grid = (units + p.per_block - 1) / p.per_block;
  auto go = [&](auto zero) {
    using T = decltype(zero);
    auto form = [&](auto width) {
      constexpr int V = decltype(width)::value;
      return few     ? append_launch<T, V, vattn::kAppendHeld256>(p, grid, threads, device, stream)
             : held ? append_launch<T, V, vattn::kAppendHeld>(p, grid, threads, device, stream)
                    : append_launch<T, V, vattn::kAppendMore>(p, grid, threads, device, stream);
    };
    if (cut == 8) return form(std::integral_constant<int, 8>());
    if (cut == 4) return form(std::integral_constant<int, 4>());
    return append_launch<T, 1, vattn::kAppendMore>(p, grid, threads, device, stream);
  };
  return a->dtype == VATTN_F16 ? go(__half()) : go(__nv_bfloat16());
}

vattn_status vattn_forward_paged(const vattn_rows* q, const vattn_pages* cache, const vattn_rows* out,
                                 const vattn_window_args* args, void* stream_ptr) {
  clear_error();
  if (!args || !cache) return fail(VATTN_ERR_INVALID_ARG, "null args or cache");
  if (args->kv_len || args->q_start)
    return fail(VATTN_ERR_INVALID_ARG, "kv_len is the cache's, and new tokens end the sequence: args' must be null");
  vattn_window_args with = *args;
  with.n_keys = 0;
  vattn_status st = check_window_args(&with);
  if (st != VATTN_OK) return st;
  if (with.n_queries > VATTN_MAX_NEW_TOKENS)
    return fail(VATTN_ERR_UNSUPPORTED, "%lld new tokens > %d", (long long)with.n_queries, VATTN_MAX_NEW_TOKENS);
  if (with.head_dim % 16 != 0)
    return fail(VATTN_ERR_UNSUPPORTED, "head_dim %lld: a multiple of 16 is needed (16-byte rows)", (long long)with.head_dim);
  const Pools pools(cache, with.n_kv_heads, with.head_dim);
  if ((st = check_pages(cache, pools, with.batch, with.n_kv_heads)) != VATTN_OK) return st;
  with.n_keys = cache->max_pages * cache->page_size;
  with.kv_len = cache->kv_len;
  const vattn_window_args* a = &with;
  const Tensor tq = window_tensor("q", q, a, true, false), to = window_tensor("out", out, a, true, true);
  if ((st = check_tensor(tq, 16)) != VATTN_OK || (st = check_tensor(to, 16)) != VATTN_OK ||
      (st = check_apart(to, tq)) != VATTN_OK || (st = check_apart(to, pools.k)) != VATTN_OK ||
      (st = check_apart(to, pools.v)) != VATTN_OK)
    return st;
  const uint64_t scale_bytes = static_cast<uint64_t>(cache->n_pages) * static_cast<uint64_t>(a->n_kv_heads) * 4u;
  if ((st = check_apart_bytes(cache->k_scale, scale_bytes, "k_scale", to)) != VATTN_OK ||
      (st = check_apart_bytes(cache->v_scale, scale_bytes, "v_scale", to)) != VATTN_OK)
    return st;
  if (tq.empty()) return VATTN_OK;
  if (a->n_q_heads / a->n_kv_heads > INT32_MAX / VATTN_MAX_NEW_TOKENS / 2)
    return fail(VATTN_ERR_UNSUPPORTED, "too many query heads for one key head");
  int device = 0, sms = 0;
  if ((st = current_device(&device)) != VATTN_OK) return st;
  if ((st = sm_count(device, &sms)) != VATTN_OK) return st;
  vattn::PagedParams p{};
  p.w = window_params(a);
  if ((st = status_word(device, &p.status)) != VATTN_OK) return st;
  p.q = rows_tensor(q);
  p.out = rows_tensor(out);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.table = cache->table;
  p.n_pages = cache->n_pages;
  p.max_pages = static_cast<int>(cache->max_pages);
  p.page = static_cast<int>(cache->page_size);
  p.rows = p.w.group * p.w.n_queries;
  p.scale_log2 = a->scale * vattn::kLog2E;
  p.d_page = fast_div(p.page);
  p.d_kv_heads = fast_div(p.w.kv_heads);
  p.d_group = fast_div(p.w.group);
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  return a->dtype == VATTN_F16 ? paged_dispatch<__half>(p, pools, sms, device, stream)
                               : paged_dispatch<__nv_bfloat16>(p, pools, sms, device, stream);
}

vattn_status vattn_forward_packed(const vattn_rows* q, const vattn_rows* k, const vattn_rows* v, const vattn_rows* out,
                                  float* lse, const int32_t* cu_seqlens, int64_t n_seqs, const vattn_window_args* a,
                                  void* stream_ptr) {
  clear_error();
  vattn_status st = check_window_args(a);
  if (st != VATTN_OK) return st;
  if (a->kv_len || a->q_start || a->tree)
    return fail(VATTN_ERR_INVALID_ARG, "kv_len, q_start and tree must be null: cu_seqlens says where sequences lie");
  if (a->batch != 1 || a->n_keys != a->n_queries)
    return fail(VATTN_ERR_INVALID_ARG, "packed prompts are one batch (is %lld) with as many keys (%lld) as queries (%lld)",
                (long long)a->batch, (long long)a->n_keys, (long long)a->n_queries);
  if (n_seqs < 0) return fail(VATTN_ERR_INVALID_ARG, "n_seqs must be >= 0");
  if (n_seqs >= (int64_t{1} << 24)) return fail(VATTN_ERR_UNSUPPORTED, "n_seqs must stay below 2^24");
  if (n_seqs > 0 && !cu_seqlens) return fail(VATTN_ERR_INVALID_ARG, "null cu_seqlens");
  if (reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) return fail(VATTN_ERR_MISALIGNED, "cu_seqlens must be 4-byte aligned");
  if ((st = forward_checks(q, k, v, out, lse, a)) != VATTN_OK) return st;
  const Tensor tq = window_tensor("q", q, a, true, false), tk = window_tensor("k", k, a, false, false),
               tv = window_tensor("v", v, a, false, false), to = window_tensor("out", out, a, true, true);
  for (const Tensor* t : {&tq, &tk, &tv})
    if ((st = check_map_rows(*t)) != VATTN_OK) return st;
  if (tq.empty() || n_seqs == 0) return VATTN_OK;

  int device = 0, sms = 0;
  if ((st = current_device(&device)) != VATTN_OK) return st;
  if ((st = sm_count(device, &sms)) != VATTN_OK) return st;
  vattn::WindowFwdParams p{};
  p.w = window_params(a);
  p.q = rows_tensor(q);
  p.k = rows_tensor(k);
  p.v = rows_tensor(v);
  p.out = rows_tensor(out);
  p.lse = lse;
  if ((st = status_word(device, &p.status)) != VATTN_OK) return st;
  // pairs: sequences of n rows have n / 128 row blocks and one more at most, their pairs half a unit more
  const int64_t some = std::min(n_seqs, a->n_queries);
  const int64_t cap = ((a->n_queries / vattn::kTile + some) * p.w.group + some) / 2 + 1;
  if (cap > kMaxKeys / p.w.kv_heads) return fail(VATTN_ERR_UNSUPPORTED, "too many tiles of 128 rows");
  p.kv_heads = fast_div(p.w.kv_heads);
  p.group = fast_div(p.w.group);
  p.scale_log2 = a->scale * vattn::kLog2E;
  CUtensorMap tm[4];
  if ((st = make_rows_map(&tm[0], &p.mq, tq, a->dtype, vattn::kTile)) != VATTN_OK ||
      (st = make_rows_map(&tm[1], &p.mk, tk, a->dtype, vattn::kTile)) != VATTN_OK ||
      (st = make_rows_map(&tm[2], &p.mv, tv, a->dtype, vattn::kTile)) != VATTN_OK ||
      (st = make_rows_map(&tm[3], &p.mo, to, a->dtype, 32, 32)) != VATTN_OK)
    return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  const int64_t items = cap * p.w.kv_heads;  // pairs; single units only where all fit the blocks at once
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(2 * items, sms));
  p.cu = cu_seqlens;
  p.n_seqs = static_cast<int>(n_seqs);
  p.sms = sms;
  Workspace ws;
  if (n_seqs <= vattn::kFindPrompts && items <= static_cast<int64_t>(vattn::kFindRounds) * grid) {
    p.seqs = fast_div(grid);
  } else {
    vattn::PackedListParams l{};
    l.cu = cu_seqlens;
    l.n_seqs = static_cast<int>(n_seqs);
    l.total = static_cast<int>(a->n_queries);
    l.group = p.w.group;
    l.kv_heads = p.w.kv_heads;
    l.sms = sms;
    l.buckets = (l.total + vattn::kTile - 1) / vattn::kTile;
    const size_t list_bytes = static_cast<size_t>(1 + cap) * sizeof(int4);
    const size_t count_bytes = l.buckets > vattn::kListBuckets ? static_cast<size_t>(l.buckets) * 4u : 0;
    if ((st = ws.take(list_bytes + count_bytes, device, stream)) != VATTN_OK) return st;
    l.list = reinterpret_cast<int4*>(ws.data());
    if (count_bytes > 0) l.counts = reinterpret_cast<int*>(ws.data() + list_bytes);
    p.list = l.list;
    vattn::vattn_packed_list_kernel<<<1, vattn::kListThreads, 0, stream>>>(l);
    if ((st = launched("packed list kernel launch")) != VATTN_OK) return st;
  }
  if (a->dtype == VATTN_F16)
    st = a->head_dim <= 64 ? packed_launch<__half, 1>(tm, p, grid, device, stream)
                           : packed_launch<__half, 2>(tm, p, grid, device, stream);
  else
    st = a->head_dim <= 64 ? packed_launch<__nv_bfloat16, 1>(tm, p, grid, device, stream)
                           : packed_launch<__nv_bfloat16, 2>(tm, p, grid, device, stream);
  if (st != VATTN_OK) return st;
  return ws.release();
}

}  // extern "C"
