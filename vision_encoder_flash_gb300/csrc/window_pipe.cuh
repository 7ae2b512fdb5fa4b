// window_pipe.cuh -- what the tensor-core kernels of the decoder calls share:
// bounded waits, key ranges of query tiles, visibility masks.
#pragma once

#include <cuda.h>
#include <cstdint>

#include "ptx.cuh"
#include "window_common.cuh"

namespace vattn {

constexpr int kTile = 128;                  // query rows and keys of a tile
constexpr int kBlockBytes = kTile * 128;    // 128 rows x 64 elements, 128-byte swizzle
constexpr float kLog2E = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLazyLog2 = 8.0f;           // O is rescaled once a row's maximum grew by 2^8
// Weights of a row, its sum and its O are held times 2^this: f16 has no digits
// below 2^-24, and rows of 2^20 keys have weights of 2^-20 that add up.
template <typename T>
constexpr float kWeightLog2 = Elem<T>::kBf16 ? 0.0f : 15.0f - kLazyLog2;
// Longest wait: some are for a whole walk (a loader's for the end of an item, the
// counter's for the last X tile's roles), hence 2 s and 10 us for each tile of the
// longest walk that a call can have, ten times what one takes.
constexpr uint64_t kPipeTimeoutNs = 2000000000ull, kPipeTileNs = 10000ull;

// Wait sites in the low byte of the status word (attn_kernel.cuh has 1..18).
enum PipeSite : uint32_t {
  kSiteWinKv = 32, kSiteWinQ = 33, kSiteWinMma = 34, kSiteWinSoft = 35, kSiteWinOut = 36,
  kSiteWinDrain = 37, kSiteWinClean = 38,
  kSiteGradLoad = 40, kSiteGradMma = 41, kSiteGradSoft = 42, kSiteGradOut = 43, kSiteGradDrain = 44,
  kSiteGradNext = 45,
};

// Bounded waits on mbarriers: one that runs out records its site in the
// status word and raises the block's abort flag, which ends the others.  What
// that takes is in shared memory at `at`, kPipeBytes aligned to 8 (abort flag, limit,
// address of the status word): registers are what these kernels are short of.
constexpr uint32_t kPipeBytes = 24;
struct Pipe {
  uint32_t at;

  __device__ __forceinline__ void init(const WindowParams& w, uint32_t* status) const {  // by one thread
    ptx::st_shared_volatile(at, 0);
    ptx::st_shared_volatile_u64(at + 8, w.wait_ns);
    ptx::st_shared_volatile_u64(at + 16, reinterpret_cast<uint64_t>(status));
  }
  __device__ __forceinline__ bool aborted() const { return ptx::ld_shared_volatile(at) != 0; }
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, uint32_t site,
                                       bool heed_abort = true) const {
    if (ptx::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = ptx::global_timer_ns();
    for (uint32_t it = 1;; ++it) {
      if (ptx::mbar_try_wait(bar, parity)) return true;
      if ((it & 31u) == 0) {
        if (heed_abort && aborted()) return false;
        if (ptx::global_timer_ns() - t0 > ptx::ld_shared_volatile_u64(at + 8)) {
          ptx::st_shared_volatile(at, 1);
          atomicOr(reinterpret_cast<uint32_t*>(ptx::ld_shared_volatile_u64(at + 16)), 0x100u | site);
          return false;
        }
      }
    }
  }
  // All lanes of the warp wait and leave together.
  __device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint32_t site) const {
    return __all_sync(0xffffffffu, wait(bar, parity, site));
  }
  // Before the block exits: also after an abort.
  __device__ __forceinline__ void drain(uint32_t bar, uint32_t parity, uint32_t site) const {
    (void)wait(bar, parity, site, false);
  }
};

// One arrival per warp, after all its lanes' earlier accesses.
__device__ __forceinline__ void pipe_warp_arrive(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) ptx::mbar_arrive(bar);
}

// Bits c <= hi of word w (columns 32 w .. 32 w + 31).
__device__ __forceinline__ uint32_t bits_upto(int hi, int w) {
  const int h = hi - 32 * w;
  return h >= 31 ? 0xffffffffu : (h < 0 ? 0u : (2u << h) - 1u);
}

// A tensor map seen as [batch, heads, rows, dim]: a dimension of stride 0
// (or size 1) is a single one in the map, its coordinate multiplied away.
struct MapMul {
  int h, b;
};

}  // namespace vattn
