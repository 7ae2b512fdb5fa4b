// decoder_api.cu -- the C ABI declared in include/vattn_decoder.h: argument
// checks, variant choice and launches of the decoder calls on sm_103a.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>

#include "../../include/vattn_decoder.h"
#include "cached_kernel.cuh"
#include "host_common.h"
#include "qk_norm_rope_kernel.cuh"
#include "rope_turns.h"
#include "window_bwd_kernel.cuh"
#include "window_fwd_kernel.cuh"

namespace {

using vattn::host::clear_error;
using vattn::host::cuda_fail;
using vattn::host::fail;
using vattn::host::Workspace;

constexpr int64_t kMaxRows = (int64_t{1} << 30) - 1;
constexpr int64_t kMaxKeys = (int64_t{1} << 29) - 1;  // positions and their differences fit in 32 bits

int elem_size(int32_t dtype) { return dtype == VATTN_F32 ? 4 : 2; }

// ------------------------------------------------------------ tensor checks
// A tensor of a call: its rows and the sizes of its dimensions.
struct Tensor {
  const char* name;
  const vattn_rows* t;
  int64_t size[3];  // batch, heads, rows
  int64_t dim;
  int esize;
  bool out;

  uintptr_t base() const { return reinterpret_cast<uintptr_t>(t->data); }
  bool empty() const { return size[0] == 0 || size[1] == 0 || size[2] == 0; }
  // bytes from the first element to the end of the last row (stride checks passed)
  uint64_t extent() const {
    uint64_t e = static_cast<uint64_t>(dim);
    for (int i = 0; i < 3; ++i) e += static_cast<uint64_t>(size[i] - 1) * static_cast<uint64_t>(t->stride[i]);
    return e * static_cast<uint64_t>(esize);
  }
};

// Every element of a tensor of these sizes and strides has its own address:
// from the innermost dimension outwards each stride passes all that is inside.
bool distinct(const int64_t (&size)[3], const int64_t (&stride)[3], int64_t dim) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return stride[a] < stride[b]; });
  int64_t inside = dim;
  for (int i : order) {
    if (size[i] <= 1) continue;
    if (stride[i] < inside) return false;
    inside += (size[i] - 1) * stride[i];
  }
  return true;
}

vattn_status check_tensor(const Tensor& x, int row_align_bytes) {
  if (x.empty()) return VATTN_OK;
  if (!x.t || !x.t->data) return fail(VATTN_ERR_INVALID_ARG, "null %s", x.name);
  const char* dims[3] = {"batch", "head", "row"};
  for (int i = 0; i < 3; ++i) {
    const int64_t s = x.t->stride[i];
    if (x.size[i] <= 1) continue;
    if (s < 0) return fail(VATTN_ERR_INVALID_ARG, "%s: negative %s stride", x.name, dims[i]);
    if (s > (int64_t{1} << 38) || (x.size[i] - 1) > (int64_t{1} << 58) / (s > 0 ? s : 1))
      return fail(VATTN_ERR_UNSUPPORTED, "%s: %s stride %lld too large", x.name, dims[i], (long long)s);
    if (s * x.esize % row_align_bytes != 0)
      return fail(VATTN_ERR_MISALIGNED, "%s: %s stride %lld is not a multiple of %d bytes", x.name,
                  dims[i], (long long)s, row_align_bytes);
  }
  const int align = row_align_bytes > x.esize ? row_align_bytes : x.esize;
  if (x.base() % static_cast<uintptr_t>(align) != 0)
    return fail(VATTN_ERR_MISALIGNED, "%s must be %d-byte aligned", x.name, align);
  if (x.out && !distinct(x.size, x.t->stride, x.dim))
    return fail(VATTN_ERR_INVALID_ARG, "%s: elements share addresses (a broadcast or overlapping view)", x.name);
  return VATTN_OK;
}

bool same_rows(const Tensor& a, const Tensor& b) {
  if (a.base() != b.base() || a.dim != b.dim || a.esize != b.esize) return false;
  for (int i = 0; i < 3; ++i)
    if (a.size[i] != b.size[i] || (a.size[i] > 1 && a.t->stride[i] != b.t->stride[i])) return false;
  return true;
}

// No element of a is an element of b: their byte ranges are apart, or they
// are parts of one packed buffer: equal strides, the one's first element some
// whole number of strides behind the other's, a box around both whose elements
// are distinct, and a dimension in which one's indexes end before the other's
// begin.
bool apart(const Tensor& a, const Tensor& b) {
  if (a.empty() || b.empty()) return true;
  if (a.base() + a.extent() <= b.base() || b.base() + b.extent() <= a.base()) return true;
  const Tensor& lo = a.base() <= b.base() ? a : b;
  const Tensor& hi = a.base() <= b.base() ? b : a;
  if (lo.esize != hi.esize || lo.dim != hi.dim) return false;
  const uint64_t bytes = hi.base() - lo.base();
  if (bytes % static_cast<uint64_t>(lo.esize) != 0) return false;
  int64_t delta = static_cast<int64_t>(bytes / static_cast<uint64_t>(lo.esize));
  int64_t size[3], stride[3] = {0, 0, 0}, off[3] = {0, 0, 0};
  int order[3] = {0, 1, 2};
  for (int i = 0; i < 3; ++i) {
    if (lo.size[i] > 1 && hi.size[i] > 1 && lo.t->stride[i] != hi.t->stride[i]) return false;
    if (lo.size[i] > 1 || hi.size[i] > 1) {
      stride[i] = lo.size[i] > 1 ? lo.t->stride[i] : hi.t->stride[i];
      if (stride[i] <= 0) return false;
    }
  }
  std::sort(order, order + 3, [&](int x, int y) { return stride[x] > stride[y]; });
  for (int i : order)
    if (stride[i] > 0) {
      off[i] = delta / stride[i];
      delta -= off[i] * stride[i];
    }
  if (delta > 0) {  // one head each: their distance is the buffer's head stride
    if (stride[1] > 0) return false;
    stride[1] = delta;
    off[1] = 1;
  }
  bool clear = false;
  for (int i = 0; i < 3; ++i) {
    size[i] = std::max(lo.size[i], off[i] + hi.size[i]);
    clear |= off[i] >= lo.size[i];
  }
  return clear && distinct(size, stride, lo.dim);
}

vattn_status check_apart(const Tensor& a, const Tensor& b) {
  if (apart(a, b)) return VATTN_OK;
  return fail(VATTN_ERR_INVALID_ARG, "%s overlaps %s", a.name, b.name);
}

// Plain memory [p, p + bytes) against a tensor's range.
vattn_status check_apart_bytes(const void* p, uint64_t bytes, const char* name, const Tensor& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(p);
  if (p == nullptr || bytes == 0 || b.empty()) return VATTN_OK;
  if (x + bytes <= b.base() || b.base() + b.extent() <= x) return VATTN_OK;
  return fail(VATTN_ERR_INVALID_ARG, "%s overlaps %s", name, b.name);
}

vattn_status current_device(int* device) {
  const cudaError_t e = cudaGetDevice(device);
  return e == cudaSuccess ? VATTN_OK : cuda_fail(e, "cudaGetDevice");
}

vattn_status launched(const char* what) {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? VATTN_OK : cuda_fail(e, what);
}

// Launches a kernel whose blocks may start while the kernel before it on the
// stream ends (they wait with griddepcontrol.wait before they read its work).
template <typename K, typename... A>
vattn_status launch_behind(const char* what, K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                           const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess ? VATTN_OK : cuda_fail(e, what);
}

// Opts a kernel in to its dynamic shared memory, once per device.
template <typename K>
vattn_status allow_smem(K kernel, int bytes, std::atomic<uint8_t>* done, int device) {
  if (done[device].load(std::memory_order_acquire)) return VATTN_OK;
  const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  done[device].store(1, std::memory_order_release);
  return VATTN_OK;
}

// ------------------------------------------------------------ norm + rotation
vattn_status check_qk(const vattn_qk_args* a) {
  if (!a) return fail(VATTN_ERR_INVALID_ARG, "null args");
  if (a->batch < 0 || a->n_q_heads < 0 || a->n_kv_heads < 0 || a->n_patches < 0)
    return fail(VATTN_ERR_INVALID_ARG, "negative size (batch=%lld n_q_heads=%lld n_kv_heads=%lld n_patches=%lld)",
                (long long)a->batch, (long long)a->n_q_heads, (long long)a->n_kv_heads, (long long)a->n_patches);
  if (a->head_dim < 1) return fail(VATTN_ERR_INVALID_ARG, "head_dim must be >= 1");
  if (a->head_dim > VATTN_MAX_HEAD_DIM)
    return fail(VATTN_ERR_UNSUPPORTED, "head_dim %lld > %d", (long long)a->head_dim, VATTN_MAX_HEAD_DIM);
  if (a->rope_dims < 0 || a->rope_dims > a->head_dim)
    return fail(VATTN_ERR_INVALID_ARG, "rope_dims %lld outside [0, head_dim = %lld]", (long long)a->rope_dims,
                (long long)a->head_dim);
  if (!(a->base > 0.0) || !std::isfinite(a->base))
    return fail(VATTN_ERR_INVALID_ARG, "base must be a finite positive number");
  if (!(a->eps >= 0.0f) || !std::isfinite(a->eps))
    return fail(VATTN_ERR_INVALID_ARG, "eps must be a finite number >= 0");
  if (a->dtype < VATTN_F32 || a->dtype > VATTN_BF16)
    return fail(VATTN_ERR_INVALID_ARG, "unknown dtype %d", (int)a->dtype);
  if (a->weight_dtype != VATTN_F32 && a->weight_dtype != a->dtype)
    return fail(VATTN_ERR_UNSUPPORTED, "weight_dtype must be VATTN_F32 or dtype");
  if (a->batch > kMaxRows || a->n_patches > kMaxRows || a->n_q_heads > kMaxRows || a->n_kv_heads > kMaxRows ||
      a->batch * a->n_patches > (int64_t{1} << 36))
    return fail(VATTN_ERR_UNSUPPORTED, "sizes must stay below 2^30 each, 2^36 tokens together");
  if (a->pos0 < 0) return fail(VATTN_ERR_INVALID_ARG, "pos0 must be >= 0");
  if (a->pos0 > INT32_MAX - a->n_patches)
    return fail(VATTN_ERR_UNSUPPORTED, "positions must fit in 32 bits");
  if ((reinterpret_cast<uintptr_t>(a->positions) | reinterpret_cast<uintptr_t>(a->factors)) & 3u)
    return fail(VATTN_ERR_MISALIGNED, "positions and factors must be 4-byte aligned");
  if ((reinterpret_cast<uintptr_t>(a->q_weight) | reinterpret_cast<uintptr_t>(a->k_weight)) %
      static_cast<uintptr_t>(elem_size(a->weight_dtype)))
    return fail(VATTN_ERR_MISALIGNED, "weights must be aligned to their element");
  return VATTN_OK;
}

Tensor qk_tensor(const char* name, const vattn_rows* t, const vattn_qk_args* a, bool is_q, bool out) {
  return Tensor{name, t, {a->batch, is_q ? a->n_q_heads : a->n_kv_heads, a->n_patches}, a->head_dim,
                elem_size(a->dtype), out};
}

// Vector width V of a call: the widest of 16 bytes, 8 bytes (16-bit types)
// and one element whose slots cut the row's two rotated halves and its rest
// evenly and whose accesses are aligned in every tensor.
int qk_vector(const Tensor* const* ts, int n, const vattn_qk_args* a) {
  const int64_t half = a->rope_dims / 2, rest = a->head_dim - 2 * half;
  const int es = elem_size(a->dtype);
  for (int v : {16 / es, 4}) {
    bool ok = half % v == 0 && rest % (2 * v) == 0;
    for (int i = 0; ok && i < n; ++i) {
      ok = ts[i]->base() % static_cast<uintptr_t>(v * es) == 0;
      for (int d = 0; ok && d < 3; ++d) ok = ts[i]->size[d] <= 1 || ts[i]->t->stride[d] % v == 0;
    }
    if (ok) return v;
  }
  return 1;
}

void qk_strides(long long (&to)[3], const vattn_rows* t) {
  for (int i = 0; i < 3; ++i) to[i] = t ? t->stride[i] : 0;
}

// Heads that a block takes for each of its tokens, 16 or fewer.  More heads
// share the angles, fewer leave shorter blocks: in units of one head's row, the
// angles cost about eight, and a call lasts as long as its blocks' share on one
// place of the resident ones, and its last block.  Halved while that gains 5 %.
// (16 heads against 8: 4 x 40 heads x 4096 x 128 bf16 52.4 us and 53.9, 16 + 16 x
// 4100 x 72 f32 17.5 and 15.2; 20 x 3000 x 128 bf16 7.3 us with 8, 9.4 with 4; 2 x
// 8 x 1025 x 80 f16, gradient, 10.2 with 2, 12.5 with 8.)
int qk_heads_per_block(const vattn::QkParams& p, double blocks_x, int resident) {
  int best = 16;
  double best_cost = 0.0;
  for (int per = 16; per >= 1; per /= 2) {
    double work = 0.0, longest = 0.0;
    for (int i = 0; i < 2; ++i) {
      const int heads = p.t[i].heads, slices = (heads + per - 1) / per;
      work += heads + 8.0 * slices;
      longest = std::max(longest, std::min(per, heads) + 8.0);
    }
    const double cost = work * blocks_x / resident + longest;
    if (per < 16 && cost > 0.95 * best_cost) continue;
    best = per;
    best_cost = cost;
  }
  return best;
}

// Sizes, angles and the split of rows over lanes and of heads over blocks.
// *odd: forward, a row takes as many lanes as it has slots where more rows fit a
// warp than with a power of two (3, 5, 6, 9, 10 slots; 32 heads x 3000 x 80 f16
// 13.7 us, else 17.2; 72 f32 14.7 and 15.1).  The gradient has two sums a row, to
// which the extra shuffles come (32 x 3000 x 80 f32 38.5 us, 34.8).
void qk_plan(vattn::QkParams* p, const vattn_qk_args* a, int v, int sms, int64_t* blocks_x, bool* odd) {
  p->positions = a->positions;
  p->factors = a->factors;
  p->tokens = a->batch * a->n_patches;
  p->pos0 = a->pos0;
  p->n = static_cast<int>(a->n_patches);
  p->d_n = vattn::FastDiv::make(static_cast<uint32_t>(a->n_patches));
  p->D = static_cast<int>(a->head_dim);
  p->half = static_cast<int>(a->rope_dims / 2);
  p->w_f32 = a->weight_dtype == VATTN_F32;
  p->eps = a->eps;
  vattn::host::rope_turns(a->base, static_cast<int>(a->rope_dims), p->turns, p->turns_rest);
  const int rest = p->D - 2 * p->half;
  p->slots = p->half / v + (rest / 2 + v - 1) / v + (v == 1 ? rest & 1 : 0);
  p->log_lanes = 0;
  while ((1 << p->log_lanes) < p->slots && p->log_lanes < 5) ++p->log_lanes;
  const bool backward = p->t[0].g != nullptr || p->t[1].g != nullptr;
  *odd = !backward && v > 1 && 32 / p->slots > 32 >> p->log_lanes;
  const int groups = *odd ? vattn::kQkThreads / 32 * (32 / p->slots) : vattn::kQkThreads >> p->log_lanes;
  *blocks_x = (p->tokens + groups - 1) / groups;
  const int resident = vattn::qk_resident(v, backward) * sms;
  const int per = qk_heads_per_block(*p, static_cast<double>(*blocks_x), resident);
  for (int i = 0; i < 2; ++i) {
    int hp = per;
    while ((p->t[i].heads + hp - 1) / hp > 16384) hp *= 2;  // grid limit in y
    p->t[i].heads_per_slice = hp;
    p->t[i].slices = (p->t[i].heads + hp - 1) / hp;
  }
  // up to eight rounds of what is resident at a time (a block in flight for
  // each that ends), behind that the blocks walk over several tokens: with
  // gradients, each leaves one row of weight gradient
  const int64_t most = 8LL * resident / (p->t[0].slices + p->t[1].slices);
  *blocks_x = std::min(*blocks_x, std::max<int64_t>(1, most));
}

template <typename T, int V, int SL, bool kBackward, bool kOdd>
vattn_status qk_go(const vattn::QkParams& p, dim3 grid, int device, cudaStream_t stream) {
  constexpr int kSmem = vattn::QkRing<T, V, SL, kBackward ? 2 : 1>::kSmemBytes;
  void (*kernel)(vattn::QkParams);
  if constexpr (kBackward) kernel = vattn::vattn_qk_norm_rope_backward_kernel<T, V, SL>;
  else kernel = vattn::vattn_qk_norm_rope_kernel<T, V, SL, kOdd>;
  static std::atomic<uint8_t> done[vattn::host::kMaxDevices];
  const vattn_status st = allow_smem(kernel, kSmem, done, device);
  if (st != VATTN_OK) return st;
  kernel<<<grid, vattn::kQkThreads, kSmem, stream>>>(p);
  return launched("norm and rotation kernel launch");
}

template <typename T, bool kBackward>
vattn_status qk_launch(const vattn::QkParams& p, int v, bool odd, dim3 grid, int device, cudaStream_t stream) {
  if constexpr (sizeof(T) == 2) {
    if (v == 8 && odd) return qk_go<T, 8, 1, kBackward, !kBackward>(p, grid, device, stream);
    if (v == 8) return qk_go<T, 8, 1, kBackward, false>(p, grid, device, stream);
  }
  if (v == 4 && odd) return qk_go<T, 4, 1, kBackward, !kBackward>(p, grid, device, stream);
  if (v == 4) return qk_go<T, 4, 1, kBackward, false>(p, grid, device, stream);
  return qk_go<T, 1, 2, kBackward, false>(p, grid, device, stream);
}

template <bool kBackward>
vattn_status qk_dispatch(const vattn::QkParams& p, int32_t dtype, int v, bool odd, dim3 grid, int device,
                         cudaStream_t stream) {
  switch (dtype) {
    case VATTN_F32: return qk_launch<float, kBackward>(p, v, odd, grid, device, stream);
    case VATTN_F16: return qk_launch<__half, kBackward>(p, v, odd, grid, device, stream);
    default: return qk_launch<__nv_bfloat16, kBackward>(p, v, odd, grid, device, stream);
  }
}

// ------------------------------------------------------------ attention
vattn_status check_window_args(const vattn_window_args* a) {
  if (!a) return fail(VATTN_ERR_INVALID_ARG, "null args");
  if (a->batch < 0 || a->n_q_heads < 0 || a->n_kv_heads < 0 || a->n_queries < 0 || a->n_keys < 0)
    return fail(VATTN_ERR_INVALID_ARG,
                "negative size (batch=%lld n_q_heads=%lld n_kv_heads=%lld n_queries=%lld n_keys=%lld)",
                (long long)a->batch, (long long)a->n_q_heads, (long long)a->n_kv_heads,
                (long long)a->n_queries, (long long)a->n_keys);
  if (a->head_dim < 1) return fail(VATTN_ERR_INVALID_ARG, "head_dim must be >= 1");
  if (a->head_dim > VATTN_MAX_HEAD_DIM || a->head_dim % 8 != 0)
    return fail(VATTN_ERR_UNSUPPORTED, "head_dim %lld: a multiple of 8 up to %d is needed (16-byte rows)",
                (long long)a->head_dim, VATTN_MAX_HEAD_DIM);
  if (a->dtype != VATTN_F16 && a->dtype != VATTN_BF16)
    return fail(VATTN_ERR_UNSUPPORTED, "dtype must be VATTN_F16 or VATTN_BF16");
  if (a->n_kv_heads == 0 ? a->n_q_heads != 0 : a->n_q_heads % a->n_kv_heads != 0)
    return fail(VATTN_ERR_INVALID_ARG, "n_q_heads %lld is not a multiple of n_kv_heads %lld",
                (long long)a->n_q_heads, (long long)a->n_kv_heads);
  if (a->n_queries > kMaxKeys || a->n_keys > kMaxKeys)
    return fail(VATTN_ERR_UNSUPPORTED, "n_queries and n_keys must stay below 2^29");
  if (a->n_q_heads > kMaxRows || a->n_kv_heads > kMaxRows || a->batch > kMaxRows ||
      a->batch * std::max(a->n_q_heads, a->n_kv_heads) > kMaxRows)
    return fail(VATTN_ERR_UNSUPPORTED, "batch * n_q_heads and batch * n_kv_heads must stay below 2^30");
  if (a->window < 0) return fail(VATTN_ERR_INVALID_ARG, "window must be >= 0");
  if (a->n_sinks < 0) return fail(VATTN_ERR_INVALID_ARG, "n_sinks must be >= 0");
  if (!(a->scale > 0.0f) || !std::isfinite(a->scale))
    return fail(VATTN_ERR_INVALID_ARG, "scale must be a finite positive number");
  if ((reinterpret_cast<uintptr_t>(a->kv_len) | reinterpret_cast<uintptr_t>(a->q_start)) & 3u)
    return fail(VATTN_ERR_MISALIGNED, "kv_len and q_start must be 4-byte aligned");
  if (reinterpret_cast<uintptr_t>(a->tree) & 7u)
    return fail(VATTN_ERR_MISALIGNED, "tree must be 8-byte aligned");
  return VATTN_OK;
}

Tensor window_tensor(const char* name, const vattn_rows* t, const vattn_window_args* a, bool is_q, bool out) {
  return Tensor{name, t, {a->batch, is_q ? a->n_q_heads : a->n_kv_heads, is_q ? a->n_queries : a->n_keys},
                a->head_dim, 2, out};
}

vattn::WindowParams window_params(const vattn_window_args* a) {
  vattn::WindowParams w{};
  w.kv_len = a->kv_len;
  w.q_start = a->q_start;
  w.tree = a->tree;
  w.batch = static_cast<int>(a->batch);
  w.heads = static_cast<int>(a->n_q_heads);
  w.kv_heads = static_cast<int>(a->n_kv_heads);
  w.group = a->n_kv_heads > 0 ? static_cast<int>(a->n_q_heads / a->n_kv_heads) : 0;
  w.n_queries = static_cast<int>(a->n_queries);
  w.n_keys = static_cast<int>(a->n_keys);
  w.dim = static_cast<int>(a->head_dim);
  const int64_t none = kMaxKeys + 1;
  w.window = static_cast<int>(a->window == 0 || a->window > none ? none : a->window);
  w.sinks = static_cast<int>(a->n_sinks > none ? none : a->n_sinks);
  w.scale = a->scale;
  const uint64_t key_tiles = static_cast<uint64_t>(a->n_keys) / vattn::kTile + 1;
  const uint64_t row_tiles = static_cast<uint64_t>(w.group) * (static_cast<uint64_t>(a->n_queries) / vattn::kTile + 1);
  w.wait_ns = vattn::kPipeTimeoutNs + vattn::kPipeTileNs * (key_tiles + row_tiles);
  return w;
}

vattn::RowsTensor rows_tensor(const vattn_rows* t) {
  vattn::RowsTensor r{};
  if (t) {
    r.p = t->data;
    for (int i = 0; i < 3; ++i) r.s[i] = t->stride[i];
  }
  return r;
}

// Tensors that are read through a tensor map have their rows apart: a map's
// row stride is not below the row's own length.
vattn_status check_map_rows(const Tensor& x) {
  if (x.empty() || x.size[2] <= 1 || x.t->stride[2] >= x.dim) return VATTN_OK;
  return fail(VATTN_ERR_UNSUPPORTED, "%s: row stride %lld below head_dim (rows broadcast or overlapping)", x.name,
              (long long)x.t->stride[2]);
}

vattn_status forward_checks(const vattn_rows* q, const vattn_rows* k, const vattn_rows* v,
                            const vattn_rows* out, const float* lse, const vattn_window_args* a) {
  const Tensor tq = window_tensor("q", q, a, true, false), tk = window_tensor("k", k, a, false, false),
               tv = window_tensor("v", v, a, false, false), to = window_tensor("out", out, a, true, true);
  for (const Tensor* t : {&tq, &tk, &tv, &to}) {
    const vattn_status st = check_tensor(*t, 16);
    if (st != VATTN_OK) return st;
  }
  for (const Tensor* t : {&tq, &tk, &tv}) {
    const vattn_status st = check_apart(to, *t);
    if (st != VATTN_OK) return st;
  }
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return fail(VATTN_ERR_MISALIGNED, "lse must be 4-byte aligned");
  const uint64_t bytes = static_cast<uint64_t>(a->batch) * a->n_q_heads * a->n_queries * 4u;
  for (const Tensor* t : {&tq, &tk, &tv, &to}) {
    const vattn_status st = check_apart_bytes(lse, bytes, "lse", *t);
    if (st != VATTN_OK) return st;
  }
  return VATTN_OK;
}

// Tensor map {dim, rows, heads, batch} of 16-bit rows with boxes of
// `box_cols` columns (64: 128-byte swizzle, 32: 64-byte) x `box_rows` rows;
// what is outside reads 0 and is not written.  A
// head or batch dimension of stride 0 (or size 1) becomes a single one, and
// *mul zeroes its coordinate.
vattn_status make_rows_map(CUtensorMap* tm, vattn::MapMul* mul, const Tensor& x, int32_t dtype, int box_rows,
                           int box_cols = 64) {
  vattn::host::EncodeTiledFn enc = nullptr;
  const vattn_status st = vattn::host::tensor_map_encoder(&enc);
  if (st != VATTN_OK) return st;
  const bool one_h = x.size[1] <= 1 || x.t->stride[1] == 0, one_b = x.size[0] <= 1 || x.t->stride[0] == 0;
  mul->h = one_h ? 0 : 1;
  mul->b = one_b ? 0 : 1;
  const cuuint64_t row = static_cast<cuuint64_t>(x.dim) * 2u;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(x.dim), static_cast<cuuint64_t>(x.size[2]),
                              static_cast<cuuint64_t>(one_h ? 1 : x.size[1]),
                              static_cast<cuuint64_t>(one_b ? 1 : x.size[0])};
  const cuuint64_t strides[3] = {x.size[2] <= 1 ? row : static_cast<cuuint64_t>(x.t->stride[2]) * 2u,
                                 one_h ? row : static_cast<cuuint64_t>(x.t->stride[1]) * 2u,
                                 one_b ? row : static_cast<cuuint64_t>(x.t->stride[0]) * 2u};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1u, 1u};
  const cuuint32_t steps[4] = {1u, 1u, 1u, 1u};
  const CUresult r = enc(tm, dtype == VATTN_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                         4, x.t->data, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         box_cols == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS)
    return fail(VATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed with CUresult %d", static_cast<int>(r));
  return VATTN_OK;
}

template <typename T, int NKB>
vattn_status window_fwd_launch(const CUtensorMap (&tm)[4], const vattn::WindowFwdParams& p, int sms, int device,
                               cudaStream_t stream) {
  using P = vattn::WindowFwdPlan<NKB>;
  auto kernel = vattn::vattn_window_fwd_kernel<T, NKB>;
  static std::atomic<uint8_t> done[vattn::host::kMaxDevices];
  const vattn_status st = allow_smem(kernel, P::kSmemBytes, done, device);
  if (st != VATTN_OK) return st;
  const unsigned grid = static_cast<unsigned>(std::min(p.items, sms));
  kernel<<<grid, P::kThreads, P::kSmemBytes, stream>>>(tm[0], tm[1], tm[2], tm[3], p);
  return launched("window attention kernel launch");
}

// The tensor-core forward pass (checks passed, at least one query row).
vattn_status forward_window(const vattn_rows* q, const vattn_rows* k, const vattn_rows* v, const vattn_rows* out,
                            float* lse, const vattn_window_args* a, cudaStream_t stream) {
  int device = 0, sms = 0;
  vattn_status st;
  if ((st = current_device(&device)) != VATTN_OK) return st;
  if ((st = vattn::host::sm_count(device, &sms)) != VATTN_OK) return st;
  vattn::WindowFwdParams p{};
  p.w = window_params(a);
  p.q = rows_tensor(q);
  p.k = rows_tensor(k);
  p.v = rows_tensor(v);
  p.out = rows_tensor(out);
  p.lse = lse;
  if ((st = vattn::host::status_word(device, &p.status)) != VATTN_OK) return st;
  const int64_t units = (a->n_queries + vattn::kTile - 1) / vattn::kTile * p.w.group;
  const int64_t seqs = a->batch * a->n_kv_heads;
  if ((units + 1) / 2 > kMaxKeys / seqs) return fail(VATTN_ERR_UNSUPPORTED, "too many tiles of 128 rows");
  p.units = static_cast<int>(units);
  p.pairs = static_cast<int>((units + 1) / 2);
  p.items = static_cast<int>(p.pairs * seqs);
  // Where the items are no more than half the blocks, every unit is an item of
  // its own (2 x 5(1) x 1111 x 96: 20.5 us, in pairs 22.2; a unit alone takes
  // nine tenths of a pair's time, so a last round is better left in pairs: 2 x
  // 16(4) x 4096 x 64 window 1024 52.6 us, with its last 56 pairs split 55.2).
  p.whole = 2 * p.items <= sms ? 0 : p.items;
  p.items += p.items - p.whole;
  p.seqs = vattn::FastDiv::make(static_cast<uint32_t>(seqs));
  p.kv_heads = vattn::FastDiv::make(static_cast<uint32_t>(p.w.kv_heads));
  p.group = vattn::FastDiv::make(static_cast<uint32_t>(p.w.group));
  p.scale_log2 = a->scale * vattn::kLog2E;
  CUtensorMap tm[4];
  if ((st = make_rows_map(&tm[0], &p.mq, window_tensor("q", q, a, true, false), a->dtype, vattn::kTile)) != VATTN_OK ||
      (st = make_rows_map(&tm[3], &p.mo, window_tensor("out", out, a, true, true), a->dtype, 32, 32)) != VATTN_OK)
    return st;
  if (a->n_keys == 0) {  // no key tile is ever loaded: any valid map does
    tm[1] = tm[2] = tm[0];
  } else if ((st = make_rows_map(&tm[1], &p.mk, window_tensor("k", k, a, false, false), a->dtype, vattn::kTile)) != VATTN_OK ||
             (st = make_rows_map(&tm[2], &p.mv, window_tensor("v", v, a, false, false), a->dtype, vattn::kTile)) != VATTN_OK) {
    return st;
  }
  if (a->dtype == VATTN_F16)
    return a->head_dim <= 64 ? window_fwd_launch<__half, 1>(tm, p, sms, device, stream)
                             : window_fwd_launch<__half, 2>(tm, p, sms, device, stream);
  return a->head_dim <= 64 ? window_fwd_launch<__nv_bfloat16, 1>(tm, p, sms, device, stream)
                           : window_fwd_launch<__nv_bfloat16, 2>(tm, p, sms, device, stream);
}

// The three gradients (checks passed; queries or keys may be none).
template <typename T, int NKB>
vattn_status backward_window(const Tensor& tg, const Tensor& tq, const Tensor& tk, const Tensor& tv,
                             vattn::WindowGradParams p, int32_t dtype, int sms, int device, cudaStream_t stream) {
  using vattn::kGradCols;
  using vattn::kTile;
  vattn_status st;
  const long long seqs = static_cast<long long>(p.w.batch) * p.w.kv_heads;
  // (no query heads: no query rows either, and dk and dv are zeros)
  const int row_tiles = p.w.heads > 0 ? (p.w.n_queries + kTile - 1) / kTile : 0;
  p.stat_tiles = 2 * row_tiles;
  p.key_tiles = (p.w.n_keys + kTile - 1) / kTile;
  // Items (query tiles of all heads of the group) of an ordinary key tile,
  // and of one of the first keys, which every later query sees.  A key tile
  // is cut so that no block has more than a third of a multiprocessor's share
  // of the call (the walk over query tiles is about as long as that over key
  // tiles; without a window a tile sees half the rows on average), but not
  // under 8 items unless there are fewer blocks than multiprocessors.  (2 x
  // 5(1) x 1111 x 96: 36 us, with 4 items 41; 1 x 8(1) x 200 x 64: 15 us, with 8
  // items 21; 2 x 16(4) x 4096 x 64, window 1024: a half 154 us, a third 142, a fifth 159.)
  const long long all_items = static_cast<long long>(p.w.group) * row_tiles;
  const long long items = std::min<long long>(
      all_items, static_cast<long long>(p.w.group) * ((static_cast<long long>(p.w.window) + kTile - 2) / kTile + 1));
  p.sink_tiles = items < all_items ? std::min(p.key_tiles, (p.w.sinks - 1) / kTile + (p.w.sinks > 0)) : 0;
  const long long bhs = static_cast<long long>(p.w.batch) * p.w.heads;
  const long long key_tiles = std::max<long long>(1, seqs * p.key_tiles), query_tiles = bhs * row_tiles;
  const double total = static_cast<double>(key_tiles) * static_cast<double>(items) * (items < all_items ? 2.0 : 1.0);
  long long most = std::max(8LL, static_cast<long long>(total / (3.0 * sms)));
  auto cut = [&most](long long n) { return static_cast<int>(std::max(1LL, std::min(256LL, (n + most - 1) / most))); };
  while (most > 2 && key_tiles * cut(items) + query_tiles < sms) most /= 2;
  p.chunks = cut(items);
  // The first keys' tiles together into eight pieces a multiprocessor at most:
  // 160 MB of partial sums, where every key as a first key would take gigabytes.
  const long long budget = 8LL * sms / std::max(1LL, seqs * p.sink_tiles);
  p.sink_chunks = p.sink_tiles > 0 ? static_cast<int>(std::max(1LL, std::min<long long>(cut(all_items), budget))) : 1;
  const long long sink_blocks = seqs * p.sink_tiles * p.sink_chunks;
  const long long rest_blocks = seqs * (p.key_tiles - p.sink_tiles) * p.chunks;
  if (sink_blocks + rest_blocks + query_tiles > kMaxRows || bhs * p.stat_tiles > kMaxRows)
    return fail(VATTN_ERR_UNSUPPORTED, "too many tiles of 128 rows");
  p.sink_blocks = static_cast<int>(sink_blocks);
  p.key_blocks = static_cast<int>(sink_blocks + rest_blocks);
  p.blocks = static_cast<int>(sink_blocks + rest_blocks + query_tiles);
  auto div = [](long long d) { return vattn::FastDiv::make(static_cast<uint32_t>(std::max(1LL, d))); };
  p.d_sink_chunks = div(p.sink_chunks);
  p.d_chunks = div(p.chunks);
  p.d_seqs = div(seqs);
  p.d_kv_heads = div(p.w.kv_heads);
  p.d_bhs = div(bhs);
  p.d_heads = div(p.w.heads);
  p.d_stat_tiles = div(p.stat_tiles);
  const long long slots = (p.sink_chunks > 1 ? sink_blocks : 0) + (p.chunks > 1 ? rest_blocks : 0);
  const size_t stat_bytes = static_cast<size_t>(p.w.batch) * p.w.heads * p.stat_tiles * vattn::kGradStat * 4;
  const size_t part_bytes = static_cast<size_t>(slots) * 2 * kTile * p.w.dim * 4;
  Workspace ws;
  // f16: the largest values of every 64 rows too, of V by blocks of their own
  const long long v_halves = dtype == VATTN_F16 ? 2 * seqs * p.key_tiles : 0;
  if (bhs * p.stat_tiles + v_halves > kMaxRows) return fail(VATTN_ERR_UNSUPPORTED, "too many tiles of 128 rows");
  const size_t peak_bytes = dtype == VATTN_F16 ? (static_cast<size_t>(bhs) * p.stat_tiles * 8 + v_halves * 4 + 255) / 256 * 256 : 0;
  if ((st = ws.take(256 + stat_bytes + peak_bytes + part_bytes, device, stream)) != VATTN_OK) return st;
  p.next = reinterpret_cast<uint32_t*>(ws.data());
  p.stat = reinterpret_cast<float*>(ws.data() + 256);
  p.peak = reinterpret_cast<float2*>(ws.data() + 256 + stat_bytes);
  p.v_peak = reinterpret_cast<float*>(p.peak + bhs * p.stat_tiles);
  p.part = reinterpret_cast<float*>(ws.data() + 256 + stat_bytes + peak_bytes);
  {
    // (one block for the counter alone where there are neither queries nor V's)
    const unsigned grid = static_cast<unsigned>(std::max(1LL, bhs * p.stat_tiles + v_halves));
    if (p.w.dim <= 64) vattn::vattn_window_stat_kernel<T, 8><<<grid, 256, 0, stream>>>(p);
    else vattn::vattn_window_stat_kernel<T, 16><<<grid, 256, 0, stream>>>(p);
    if ((st = launched("gradient statistics kernel launch")) != VATTN_OK) return st;
  }
  // each tensor as an X tile (128 rows) and as a Y tile (64 rows); one that
  // is empty is never loaded, and another's map stands in for it
  const Tensor* t[4] = {&tq, &tg, &tk, &tv};
  CUtensorMap x[4], y[4];
  vattn::MapMul mul[4] = {};
  for (int i = 0; i < 4; ++i) {
    const Tensor& u = !t[i]->empty() ? *t[i] : (i < 2 ? tk : tq);
    if ((st = make_rows_map(&x[i], &mul[i], u, dtype, kTile)) != VATTN_OK ||
        (st = make_rows_map(&y[i], &mul[i], u, dtype, kGradCols)) != VATTN_OK)
      return st;
  }
  p.mq = mul[0];
  p.mg = mul[1];
  p.mk = mul[2];
  p.mv = mul[3];
  using P = vattn::GradPlan<NKB>;
  auto kernel = vattn::vattn_window_bwd_kernel<T, NKB>;
  static std::atomic<uint8_t> done[vattn::host::kMaxDevices];
  if ((st = allow_smem(kernel, P::kSmemBytes, done, device)) != VATTN_OK) return st;
  if ((st = launch_behind("gradient kernel launch", kernel, dim3(static_cast<unsigned>(std::min(p.blocks, sms))),
                          dim3(P::kThreads), P::kSmemBytes, stream, x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3],
                          p)) != VATTN_OK)
    return st;
  if (slots > 0) {
    const long long joined = seqs * ((p.sink_chunks > 1 ? p.sink_tiles : 0) + (p.chunks > 1 ? p.key_tiles - p.sink_tiles : 0));
    const dim3 grid(static_cast<unsigned>(joined), static_cast<unsigned>((2 * kTile * (p.w.dim / 8) + 255) / 256));
    if ((st = launch_behind("gradient join kernel launch", vattn::vattn_window_join_kernel<T>, grid, dim3(256), 0,
                            stream, p)) != VATTN_OK)
      return st;
  }
  return ws.release();
}

template <typename T, int DP, int RW>
vattn_status cached_launch(vattn::CachedParams p, int sms, int device, cudaStream_t stream) {
  using P = vattn::CachedPlan<DP, RW>;
  auto kernel = vattn::vattn_cached_kernel<T, DP, RW>;
  static std::atomic<uint8_t> done[vattn::host::kMaxDevices];
  vattn_status st = allow_smem(kernel, P::kSmemBytes, done, device);
  if (st != VATTN_OK) return st;
  const long long seqs = static_cast<long long>(p.w.batch) * p.w.kv_heads;
  p.row_blocks = (p.rows + 16 * RW - 1) / (16 * RW);
  if (p.row_blocks > 65535 || seqs * p.rows > INT32_MAX)
    return fail(VATTN_ERR_UNSUPPORTED, "too many query rows");
  // Shares of the keys: as many blocks as are resident at a time (32 sequences
  // x 8 key heads x 16385 keys of 128, lengths from 5.4 k: with two a head 0.71 of
  // the time with one, 0.95 of that with five, now 201 us; a tree of 31 over 4096
  // keys: one round 0.78 of two, now 19.6 us), of 256 keys at least, or of 128 where that makes no more
  // than 32 shares (500 keys: 8.0 us against 10.6; 30000 keys: 12 us with 118
  // shares, 16 with 235).
  const long long most_keys = std::min<long long>(p.w.n_keys, static_cast<long long>(p.w.sinks) + p.w.window + p.w.n_queries);
  const long long blocks = seqs * p.row_blocks, room = static_cast<long long>(P::kResident) * sms;
  const long long fill = room / blocks >= 4 ? room / blocks : (room + blocks - 1) / blocks;
  const long long fine = std::max(std::min(32LL, (most_keys + 127) / 128), (most_keys + 255) / 256);
  p.splits = static_cast<int>(std::max(1LL, std::min({fill, fine, static_cast<long long>(vattn::kCachedMaxSplits)})));
  Workspace ws;
  const bool clustered = p.splits > 1 && p.splits <= vattn::kCachedCluster;
  if (p.splits > 1 && !clustered) {
    const size_t rows = static_cast<size_t>(blocks) * p.splits * 16 * RW;
    if ((st = ws.take(rows * (p.w.dim + 2) * 4, device, stream)) != VATTN_OK) return st;
    p.part_o = reinterpret_cast<float*>(ws.data());
    p.part_ml = p.part_o + rows * p.w.dim;
  }
  const dim3 grid(static_cast<unsigned>(p.splits), static_cast<unsigned>(p.row_blocks),
                  static_cast<unsigned>(std::min<long long>(seqs, 65535)));
  if (clustered) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(P::kThreads);
    cfg.dynamicSmemBytes = P::kSmemBytes;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = grid.x;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    return e == cudaSuccess ? VATTN_OK : cuda_fail(e, "cached attention kernel launch");
  }
  kernel<<<grid, P::kThreads, P::kSmemBytes, stream>>>(p);
  if ((st = launched("cached attention kernel launch")) != VATTN_OK) return st;
  if (p.splits == 1) return VATTN_OK;
  if ((st = launch_behind("cached attention join kernel launch", vattn::vattn_cached_join_kernel<T, RW>,
                          dim3(static_cast<unsigned>(seqs * p.rows)), dim3(128), 0, stream, p)) != VATTN_OK)
    return st;
  return ws.release();
}

template <typename T>
vattn_status cached_dispatch(const vattn::CachedParams& p, int sms, int device, cudaStream_t stream) {
  const int rw = p.rows <= 16 ? 1 : (p.rows <= 32 ? 2 : 4);
  if (p.w.dim <= 32)
    return rw == 1   ? cached_launch<T, 32, 1>(p, sms, device, stream)
           : rw == 2 ? cached_launch<T, 32, 2>(p, sms, device, stream)
                     : cached_launch<T, 32, 4>(p, sms, device, stream);
  if (p.w.dim <= 64)
    return rw == 1   ? cached_launch<T, 64, 1>(p, sms, device, stream)
           : rw == 2 ? cached_launch<T, 64, 2>(p, sms, device, stream)
                     : cached_launch<T, 64, 4>(p, sms, device, stream);
  return rw == 1   ? cached_launch<T, 128, 1>(p, sms, device, stream)
         : rw == 2 ? cached_launch<T, 128, 2>(p, sms, device, stream)
                   : cached_launch<T, 128, 4>(p, sms, device, stream);
}

}  // namespace

extern "C" {

vattn_status vattn_qk_norm_rope(const vattn_rows* q, const vattn_rows* k, const vattn_rows* q_out,
                                const vattn_rows* k_out, const vattn_qk_args* a, void* stream_ptr) {
  clear_error();
  vattn_status st = check_qk(a);
  if (st != VATTN_OK) return st;
  const Tensor tq = qk_tensor("q", q, a, true, false), tk = qk_tensor("k", k, a, false, false),
               oq = qk_tensor("q_out", q_out, a, true, true), ok = qk_tensor("k_out", k_out, a, false, true);
  const Tensor* all[4] = {&tq, &tk, &oq, &ok};
  for (const Tensor* t : all)
    if ((st = check_tensor(*t, elem_size(a->dtype))) != VATTN_OK) return st;
  if (!oq.empty() && !same_rows(oq, tq) && (st = check_apart(oq, tq)) != VATTN_OK) return st;
  if (!ok.empty() && !same_rows(ok, tk) && (st = check_apart(ok, tk)) != VATTN_OK) return st;
  if ((st = check_apart(oq, tk)) != VATTN_OK || (st = check_apart(ok, tq)) != VATTN_OK ||
      (st = check_apart(oq, ok)) != VATTN_OK)
    return st;
  if (tq.empty() && tk.empty()) return VATTN_OK;

  int device = 0, sms = 0;
  if ((st = current_device(&device)) != VATTN_OK) return st;
  if ((st = vattn::host::sm_count(device, &sms)) != VATTN_OK) return st;
  const Tensor* used[4];
  int n_used = 0;
  for (const Tensor* t : all)
    if (!t->empty()) used[n_used++] = t;
  const int v = qk_vector(used, n_used, a);
  vattn::QkParams p{};
  const vattn_rows* in[2] = {q, k};
  const vattn_rows* out[2] = {q_out, k_out};
  const void* w[2] = {a->q_weight, a->k_weight};
  for (int i = 0; i < 2; ++i) {
    vattn::QkTensor& t = p.t[i];
    t.heads = static_cast<int>(i == 0 ? a->n_q_heads : a->n_kv_heads);
    if (t.heads == 0) continue;
    t.x = in[i]->data;
    t.y = out[i]->data;
    t.w = w[i];
    qk_strides(t.xs, in[i]);
    qk_strides(t.ys, out[i]);
  }
  int64_t bx = 0;
  bool odd = false;
  qk_plan(&p, a, v, sms, &bx, &odd);
  const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>(p.t[0].slices + p.t[1].slices));
  return qk_dispatch<false>(p, a->dtype, v, odd, grid, device, static_cast<cudaStream_t>(stream_ptr));
}

vattn_status vattn_qk_norm_rope_backward(const vattn_rows* dq_out, const vattn_rows* dk_out,
                                         const vattn_rows* q, const vattn_rows* k,
                                         const vattn_rows* dq, const vattn_rows* dk,
                                         float* dq_weight, float* dk_weight, const vattn_qk_args* a,
                                         void* stream_ptr) {
  clear_error();
  vattn_status st = check_qk(a);
  if (st != VATTN_OK) return st;
  const Tensor gq = qk_tensor("dq_out", dq_out, a, true, false), gk = qk_tensor("dk_out", dk_out, a, false, false),
               tq = qk_tensor("q", q, a, true, false), tk = qk_tensor("k", k, a, false, false),
               oq = qk_tensor("dq", dq, a, true, true), ok = qk_tensor("dk", dk, a, false, true);
  const Tensor* all[6] = {&gq, &gk, &tq, &tk, &oq, &ok};
  for (const Tensor* t : all)
    if ((st = check_tensor(*t, elem_size(a->dtype))) != VATTN_OK) return st;
  for (const Tensor* t : {&gq, &tq})
    if (!oq.empty() && !same_rows(oq, *t) && (st = check_apart(oq, *t)) != VATTN_OK) return st;
  for (const Tensor* t : {&gk, &tk})
    if (!ok.empty() && !same_rows(ok, *t) && (st = check_apart(ok, *t)) != VATTN_OK) return st;
  for (const Tensor* t : {&gk, &tk})
    if ((st = check_apart(oq, *t)) != VATTN_OK) return st;
  for (const Tensor* t : {&gq, &tq, &oq})
    if ((st = check_apart(ok, *t)) != VATTN_OK) return st;
  if ((reinterpret_cast<uintptr_t>(dq_weight) | reinterpret_cast<uintptr_t>(dk_weight)) & 3u)
    return fail(VATTN_ERR_MISALIGNED, "dq_weight and dk_weight must be 4-byte aligned");
  float* dw[2] = {a->q_weight ? dq_weight : nullptr, a->k_weight ? dk_weight : nullptr};
  const uint64_t w_bytes = static_cast<uint64_t>(a->head_dim) * 4u;
  for (int i = 0; i < 2; ++i)
    for (const Tensor* t : all)
      if ((st = check_apart_bytes(dw[i], w_bytes, i == 0 ? "dq_weight" : "dk_weight", *t)) != VATTN_OK) return st;
  if (dw[0] && dw[1] &&
      reinterpret_cast<uintptr_t>(dw[0]) < reinterpret_cast<uintptr_t>(dw[1]) + w_bytes &&
      reinterpret_cast<uintptr_t>(dw[1]) < reinterpret_cast<uintptr_t>(dw[0]) + w_bytes)
    return fail(VATTN_ERR_INVALID_ARG, "dq_weight overlaps dk_weight");

  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (tq.empty() && tk.empty()) {  // sums over no rows
    for (float* d : dw)
      if (d) {
        const cudaError_t e = cudaMemsetAsync(d, 0, w_bytes, stream);
        if (e != cudaSuccess) return cuda_fail(e, "clearing a weight gradient");
      }
    return VATTN_OK;
  }
  int device = 0, sms = 0;
  if ((st = current_device(&device)) != VATTN_OK) return st;
  if ((st = vattn::host::sm_count(device, &sms)) != VATTN_OK) return st;
  const Tensor* used[6];
  int n_used = 0;
  for (const Tensor* t : all)
    if (!t->empty()) used[n_used++] = t;
  const int v = qk_vector(used, n_used, a);
  vattn::QkParams p{};
  const vattn_rows* in[2] = {q, k};
  const vattn_rows* grad[2] = {dq_out, dk_out};
  const vattn_rows* out[2] = {dq, dk};
  const void* w[2] = {a->q_weight, a->k_weight};
  for (int i = 0; i < 2; ++i) {
    vattn::QkTensor& t = p.t[i];
    t.heads = static_cast<int>(i == 0 ? a->n_q_heads : a->n_kv_heads);
    if (t.heads == 0) continue;
    t.x = in[i]->data;
    t.g = grad[i]->data;
    t.y = out[i]->data;
    t.w = w[i];
    qk_strides(t.xs, in[i]);
    qk_strides(t.gs, grad[i]);
    qk_strides(t.ys, out[i]);
  }
  int64_t bx = 0;
  bool odd = false;
  qk_plan(&p, a, v, sms, &bx, &odd);
  const int slices = p.t[0].slices + p.t[1].slices;
  const dim3 grid(static_cast<unsigned>(bx), static_cast<unsigned>(slices));
  Workspace ws;
  if (dw[0] || dw[1]) {
    if ((st = ws.take(static_cast<size_t>(bx) * slices * p.D * 4, device, stream)) != VATTN_OK) return st;
    p.part = reinterpret_cast<float*>(ws.data());
  }
  if ((st = qk_dispatch<true>(p, a->dtype, v, odd, grid, device, stream)) != VATTN_OK) return st;
  if (!p.part) return VATTN_OK;
  vattn::QkWeightSum s{};
  s.part = p.part;
  s.D = p.D;
  for (int i = 0; i < 2; ++i) s.dw[i] = dw[i];
  s.row1[0] = s.row0[1] = bx * p.t[0].slices;
  s.row1[1] = bx * slices;
  if ((st = launch_behind("weight gradient kernel launch", vattn::vattn_qk_weight_sum_kernel,
                          dim3(static_cast<unsigned>((p.D + 31) / 32), 2), dim3(32, 32), 0, stream, s)) != VATTN_OK)
    return st;
  return ws.release();
}

vattn_status vattn_forward_window(const vattn_rows* q, const vattn_rows* k, const vattn_rows* v,
                                  const vattn_rows* out, float* lse, const vattn_window_args* a,
                                  void* stream_ptr) {
  clear_error();
  vattn_status st = check_window_args(a);
  if (st != VATTN_OK) return st;
  if (a->tree) return fail(VATTN_ERR_INVALID_ARG, "tree is for vattn_forward_cached");
  if ((st = forward_checks(q, k, v, out, lse, a)) != VATTN_OK) return st;
  for (const Tensor& t : {window_tensor("q", q, a, true, false), window_tensor("k", k, a, false, false),
                          window_tensor("v", v, a, false, false)})
    if ((st = check_map_rows(t)) != VATTN_OK) return st;
  if (a->batch * a->n_q_heads == 0 || a->n_queries == 0) return VATTN_OK;
  return forward_window(q, k, v, out, lse, a, static_cast<cudaStream_t>(stream_ptr));
}

vattn_status vattn_backward_window(const vattn_rows* dout, const vattn_rows* q, const vattn_rows* k,
                                   const vattn_rows* v, const vattn_rows* out, const float* lse,
                                   const vattn_rows* dq, const vattn_rows* dk, const vattn_rows* dv,
                                   const vattn_window_args* a, void* stream_ptr) {
  clear_error();
  vattn_status st = check_window_args(a);
  if (st != VATTN_OK) return st;
  if (a->tree) return fail(VATTN_ERR_INVALID_ARG, "tree is for vattn_forward_cached");
  const Tensor tg = window_tensor("dout", dout, a, true, false), tq = window_tensor("q", q, a, true, false),
               tk = window_tensor("k", k, a, false, false), tv = window_tensor("v", v, a, false, false),
               to = window_tensor("out", out, a, true, false), oq = window_tensor("dq", dq, a, true, true),
               ok = window_tensor("dk", dk, a, false, true), ov = window_tensor("dv", dv, a, false, true);
  const Tensor* ins[5] = {&tg, &tq, &tk, &tv, &to};
  const Tensor* outs[3] = {&oq, &ok, &ov};
  for (const Tensor* t : ins)
    if ((st = check_tensor(*t, 16)) != VATTN_OK || (st = check_map_rows(*t)) != VATTN_OK) return st;
  for (const Tensor* t : outs)
    if ((st = check_tensor(*t, 16)) != VATTN_OK) return st;
  for (const Tensor* t : outs)
    for (const Tensor* u : ins)
      if ((st = check_apart(*t, *u)) != VATTN_OK) return st;
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < i; ++j)
      if ((st = check_apart(*outs[i], *outs[j])) != VATTN_OK) return st;
  if (!tq.empty() && !lse) return fail(VATTN_ERR_INVALID_ARG, "null lse");
  if (reinterpret_cast<uintptr_t>(lse) & 3u) return fail(VATTN_ERR_MISALIGNED, "lse must be 4-byte aligned");
  const uint64_t bytes = static_cast<uint64_t>(a->batch) * a->n_q_heads * a->n_queries * 4u;
  for (const Tensor* t : outs)
    if ((st = check_apart_bytes(lse, bytes, "lse", *t)) != VATTN_OK) return st;
  if (tq.empty() && tk.empty()) return VATTN_OK;
  int device = 0, sms = 0;
  if ((st = current_device(&device)) != VATTN_OK) return st;
  if ((st = vattn::host::sm_count(device, &sms)) != VATTN_OK) return st;
  vattn::WindowGradParams p{};
  p.w = window_params(a);
  p.q = rows_tensor(q);
  p.k = rows_tensor(k);
  p.v = rows_tensor(v);
  p.out = rows_tensor(out);
  p.dout = rows_tensor(dout);
  p.dq = rows_tensor(dq);
  p.dk = rows_tensor(dk);
  p.dv = rows_tensor(dv);
  p.lse = lse;
  p.scale_log2 = a->scale * vattn::kLog2E;
  if ((st = vattn::host::status_word(device, &p.status)) != VATTN_OK) return st;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  if (a->dtype == VATTN_F16)
    return a->head_dim <= 64 ? backward_window<__half, 1>(tg, tq, tk, tv, p, a->dtype, sms, device, stream)
                             : backward_window<__half, 2>(tg, tq, tk, tv, p, a->dtype, sms, device, stream);
  return a->head_dim <= 64 ? backward_window<__nv_bfloat16, 1>(tg, tq, tk, tv, p, a->dtype, sms, device, stream)
                           : backward_window<__nv_bfloat16, 2>(tg, tq, tk, tv, p, a->dtype, sms, device, stream);
}

vattn_status vattn_forward_cached(const vattn_rows* q, const vattn_rows* k, const vattn_rows* v,
                                  const vattn_rows* out, const vattn_window_args* a, void* stream_ptr) {
  clear_error();
  vattn_status st = check_window_args(a);
  if (st != VATTN_OK) return st;
  if (a->q_start) return fail(VATTN_ERR_INVALID_ARG, "q_start must be null: new tokens end the sequence");
  if (a->n_queries > VATTN_MAX_NEW_TOKENS)
    return fail(VATTN_ERR_UNSUPPORTED, "%lld new tokens > %d: use vattn_forward_window", (long long)a->n_queries,
                VATTN_MAX_NEW_TOKENS);
  if (a->batch > 0 && !a->kv_len) return fail(VATTN_ERR_INVALID_ARG, "null kv_len");
  if ((st = forward_checks(q, k, v, out, nullptr, a)) != VATTN_OK) return st;
  if (a->batch * a->n_q_heads == 0 || a->n_queries == 0) return VATTN_OK;
  if (a->n_q_heads / a->n_kv_heads > INT32_MAX / VATTN_MAX_NEW_TOKENS / 2)
    return fail(VATTN_ERR_UNSUPPORTED, "too many query heads for one key head");
  int device = 0, sms = 0;
  if ((st = current_device(&device)) != VATTN_OK) return st;
  if ((st = vattn::host::sm_count(device, &sms)) != VATTN_OK) return st;
  vattn::CachedParams p{};
  p.w = window_params(a);
  p.q = rows_tensor(q);
  p.k = rows_tensor(k);
  p.v = rows_tensor(v);
  p.out = rows_tensor(out);
  p.rows = p.w.group * p.w.n_queries;
  p.scale_log2 = a->scale * vattn::kLog2E;
  cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
  return a->dtype == VATTN_F16 ? cached_dispatch<__half>(p, sms, device, stream)
                               : cached_dispatch<__nv_bfloat16>(p, sms, device, stream);
}

}  // extern "C"
