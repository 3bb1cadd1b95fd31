// What the kernels of the attention to an encoder's states share: bounded
// waits, rings, and the softmax warps' accesses to tensor memory.
#pragma once

#include "epilogue.cuh"

namespace wsattn {
namespace cross {

using namespace ptx;

constexpr int kRows = kCrossRows;
constexpr uint32_t kBoxBytes = kRows * 128;  // 64 columns of 128 rows
constexpr long long kWaitLimitCycles = 1LL << 31;  // about one second
constexpr uint32_t kTmemCols = 512;
constexpr float kLn2 = 0.69314718055994531f;

struct Sync {
  uint32_t bars;
  volatile int* abort_flag;
  int* status;
};
__device__ __forceinline__ uint32_t bar(const Sync& s, int i) {
  return s.bars + 8u * static_cast<uint32_t>(i);
}
static __device__ __noinline__ bool wait_slow(const Sync& s, uint32_t b, uint32_t parity, int code) {
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(b, parity)) return true;
    if (*s.abort_flag) return false;
    if (clock64() - t0 > kWaitLimitCycles) {
      atomicOr(s.status, code);
      *s.abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(const Sync& s, uint32_t b, uint32_t parity, int code) {
  if (mbar_try_wait(b, parity)) return true;
  return wait_slow(s, b, parity, code);
}
// Every lane waits, then the warp agrees and reconverges.
__device__ __forceinline__ bool wait_warp(const Sync& s, uint32_t b, uint32_t parity, int code) {
  return __all_sync(0xffffffffu, wait(s, b, parity, code));
}
// One arrival for a warp, after every lane's writes.
__device__ __forceinline__ void warp_arrive(uint32_t b) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(b);
}

// Position in a ring of N stages: slot, and the parity of its current use.
template <int N>
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) {
      slot = 0;
      phase ^= 1u;
    }
  }
};
// A producer's ring: remembers what it loaded, to wait for it before leaving
// after an expired wait (the copies land whatever the consumers do).
template <int N>
struct LoadRing : Ring<N> {
  uint32_t issued = 0, last = 0;
  __device__ __forceinline__ void loaded() {
    last = (last & ~(1u << this->slot)) | this->phase << this->slot;
    issued |= 1u << this->slot;
    this->next();
  }
  __device__ __noinline__ void drain(uint32_t full0) const {
    for (int i = 0; i < N; ++i) {
      if (!(issued >> i & 1u)) continue;
      const long long t0 = clock64();
      while (!mbar_try_wait(full0 + 8u * i, last >> i & 1u))
        if (clock64() - t0 > kWaitLimitCycles) break;
    }
  }
};

__device__ __forceinline__ int keys_of(const CrossParams& p, int b) {
  return p.lengths ? max(0, min(__ldg(p.lengths + b), p.m)) : p.m;
}

// 16-bit element type of the kernels' tensors.
template <bool BF16>
struct Elem {
  using type = __nv_bfloat16;
};
template <>
struct Elem<false> {
  using type = __half;
};

// Row r's 16-byte unit u of a 128-byte-swizzled tile of 64-column boxes.
__device__ __forceinline__ uint32_t swizzled(uint32_t tile, int r, int u) {
  return tile + static_cast<uint32_t>(u / 8) * kBoxBytes + static_cast<uint32_t>(r) * 128u +
         (static_cast<uint32_t>((u ^ r) & 7) << 4);
}

}  // namespace cross
}  // namespace wsattn
