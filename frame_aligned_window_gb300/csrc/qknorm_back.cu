// Gradients of the per-head norms with the rotation (qknorm.cuh has the
// formulas and what the passes share).
#include "qknorm.cuh"

namespace wsattn {
namespace {

using namespace ptx;
using namespace qk;

// Backward.  Persistent: the work items (rows of one CTA, one head group) of
// q and k form one list, the group the slow index, of which each CTA takes a
// contiguous share of equal weight; then the same for v's copies.  A CTA's share of the gain
// gradients stays in registers until its part changes, and one partial row
// per CTA and part goes to global memory: the sums have a fixed order.
//
// A head row takes about 300 instructions here and 128 registers a thread
// hold little beside its sums, gains and angles, so loads in registers would
// leave too few bytes in flight: the rows come through a ring of cp.async
// stages in shared memory, one head row a stage and lane group, that runs
// ahead across the items (each lane reads what it loaded: no barrier).
template <typename T>
constexpr int kBackStages = sizeof(T) == 4 ? 3 : 5;
template <typename T>
constexpr int kBackStageBytes = 32 * 32 * static_cast<int>(sizeof(T));  // a warp's x and dy rows

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where a warp is in its list of items: the item, and the head within it.
struct BackCursor {
  int64_t rb;     // row block
  int64_t left;   // items from here on, this one included
  int g, pi;      // head group, part
  int h, heads;   // head within the group, heads of the group
  int64_t b, n;   // this lane group's token
  bool active;
};

template <int LG>
__device__ __forceinline__ void open_item(const QkParams& p, const Lane& ln, BackCursor& c) {
  while (c.pi == 0 && c.g >= p.part[1].group0) c.pi = 1;
  const QkPart& part = p.part[c.pi];
  c.h = 0;
  c.heads = min(part.io.heads - (c.g - part.group0) * part.group_heads, part.group_heads);
  const int64_t row = (c.rb * (kQkThreads / 32) + threadIdx.x / 32) * (32 >> LG) +
                      ((threadIdx.x & 31) >> LG);
  c.active = row < p.rows && ln.on &&
             WSATTN_BOUNDS(p.status, c.rb < p.row_blocks && c.heads >= 1 &&
                                         (c.g - part.group0) * part.group_heads + c.heads <=
                                             part.io.heads &&
                                         16 * ln.c + 16 <= 2 * ln.half);
  c.b = c.n = 0;
  if (c.active) split_row(p, row, c.b, c.n);
}
__device__ __forceinline__ void next_item(const QkParams& p, BackCursor& c) {
  --c.left;
  if (++c.rb == p.row_blocks) {
    c.rb = 0;
    ++c.g;
  }
}

template <typename T, bool VEC, int LG>
__global__ void __launch_bounds__(kQkThreads, kQkBackCtasPerSm)
    qk_backward_kernel(const __grid_constant__ QkParams p) {
  extern __shared__ __align__(16) uint8_t ring_raw[];
  constexpr int kStages = kBackStages<T>, kBytes = kBackStageBytes<T>;
  constexpr int kPieces = sizeof(T) / 2;  // 16-byte pieces of 8 elements
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
  const Lane ln = make_lane<T, LG>(p.rot);
  const float inv_d = 0.5f / static_cast<float>(p.rot.pairs);
  const bool inter = p.rot.interleaved != 0;
  const int D = 2 * p.rot.pairs;
  // stage: 16-byte pieces [dy 0, dy 1, x 0, x 1][lane] (twice as many in fp32)
  const uint32_t ring = smem_u32(ring_raw) + static_cast<uint32_t>(warp * kStages * kBytes + 16 * lane);
  float acc[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) acc[i] = 0.f;

  // adds the CTA's gain gradient of part pi and writes its partial row
  __shared__ float red[kQkThreads / 32][2 * kRotMaxPairs];
  auto flush = [&](int pi) {
    if (!p.dw_part) return;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
#pragma unroll
      for (int o = 1 << LG; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
      if (lane < (1 << LG) && ln.on) red[warp][lane_element<T>(ln, i)] = acc[i];
      acc[i] = 0.f;
    }
    __syncthreads();
    float* out = p.dw_part + (static_cast<int64_t>(pi) * gridDim.x + blockIdx.x) * D;
    for (int d = threadIdx.x; d < D; d += kQkThreads) {
      float t = 0.f;
      for (int v = 0; v < kQkThreads / 32; ++v) t += red[v][d];
      out[d] = t;
    }
    __syncthreads();
  };
  // This CTA's share of q's and k's items.  An item weighs its heads and about
  // one and a half more for its angles; the shares are equal in weight.
  const int64_t nq = p.part[0].groups * p.row_blocks;
  const int64_t wq = 2 * p.part[0].group_heads + 3, wk = 2 * p.part[1].group_heads + 3;
  const int64_t weight = nq * wq + p.part[1].groups * p.row_blocks * wk;
  auto item_at = [&](int64_t x) {
    return x <= nq * wq ? (x + wq - 1) / wq : nq + (x - nq * wq + wk - 1) / wk;
  };

  griddep_wait();
  griddep_launch_dependents();
  int64_t i = item_at(weight * blockIdx.x / gridDim.x);
  int64_t i1 = item_at(weight * (blockIdx.x + 1) / gridDim.x);
  int g = static_cast<int>(i / p.row_blocks);
  int64_t rb = i - g * p.row_blocks;
  int done_part = 0;
  if (i < i1) {
    BackCursor cur;
    cur.g = g;
    cur.rb = rb;
    cur.left = i1 - i;
    cur.pi = 0;
    BackCursor ahead = cur;
    const T* gy = nullptr;  // the next head row to load (the ring) or to use (plain loads)
    const T* xs = nullptr;
    auto open_ahead = [&] {
      open_item<LG>(p, ln, ahead);
      const QkPart& part = p.part[ahead.pi];
      const int64_t h0 = static_cast<int64_t>(ahead.g - part.group0) * part.group_heads;
      gy = static_cast<const T*>(part.io.in) + ahead.b * part.io.ib + ahead.n * part.io.in_ +
           h0 * part.io.ih + ln.off;
      xs = static_cast<const T*>(part.x) + ahead.b * part.xb + ahead.n * part.xn + h0 * part.xh +
           ln.off;
    };
    auto step_ahead = [&] {
      const QkPart& part = p.part[ahead.pi];
      gy += part.io.ih;
      xs += part.xh;
      if (++ahead.h == ahead.heads) {
        next_item(p, ahead);
        if (ahead.left > 0) open_ahead();
      }
    };
    uint32_t load_slot = 0;
    auto issue = [&] {
      if (ahead.left > 0) {
        if (ahead.active) {
          const uint32_t d = ring + load_slot * kBytes;
#pragma unroll
          for (int q = 0; q < kPieces; ++q) {
            const int e = q * ln.step;  // fp32: the lane's second four elements
            cp_async16(d + (0 + q) * 512, gy + e);
            cp_async16(d + (kPieces + q) * 512, gy + ln.half + e);
            cp_async16(d + (2 * kPieces + q) * 512, xs + e);
            cp_async16(d + (3 * kPieces + q) * 512, xs + ln.half + e);
          }
        }
        step_ahead();
      }
      cp_async_commit();
      if (++load_slot == kStages) load_slot = 0;
    };
    open_ahead();
    if (VEC)
      for (int k = 0; k < kStages - 1; ++k) issue();
    uint32_t slot = 0;
    float w[16];
    int w_part = -1;
    for (; cur.left > 0; next_item(p, cur)) {
      open_item<LG>(p, ln, cur);
      const QkPart& part = p.part[cur.pi];
      if (w_part != cur.pi) {
        for (; done_part < cur.pi; ++done_part) flush(done_part);
        load_gain<T>(p, part, ln, w);
        w_part = cur.pi;
      }
      const int64_t dstep = part.io.oh;
      T* dx = static_cast<T*>(part.io.out) + cur.b * part.io.ob + cur.n * part.io.on +
              static_cast<int64_t>(cur.g - part.group0) * part.group_heads * dstep + ln.off;
      // idle lanes hold zeros and join the row sums: no turn there
      float cs[8] = {}, sn[8] = {};
      if (cur.active)
        lane_angles<T>(p.rot, ln, p.pos + cur.b * p.pos_b + cur.n * p.rot.axes, -1.f, cs, sn);
      for (; cur.h < cur.heads; ++cur.h) {
        float gr[16], x[16];
        if (VEC) {
          issue();
          cp_async_wait<kStages - 1>();
          const uint32_t d = ring + slot * kBytes;
          if (++slot == kStages) slot = 0;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            Half8<T> a, c;
            a.a = ld_shared_v4(d + q * kPieces * 512);
            c.a = ld_shared_v4(d + (2 + q) * kPieces * 512);
            if constexpr (sizeof(T) == 4) {
              a.b = ld_shared_v4(d + (q * kPieces + 1) * 512);
              c.b = ld_shared_v4(d + ((2 + q) * kPieces + 1) * 512);
            }
            unpack8(a, gr + 8 * q);
            unpack8(c, x + 8 * q);
          }
        } else if (cur.active) {
          unpack8(load8<false>(gy, ln.step), gr);
          unpack8(load8<false>(gy + ln.half, ln.step), gr + 8);
          unpack8(load8<false>(xs, ln.step), x);
          unpack8(load8<false>(xs + ln.half, ln.step), x + 8);
        }
        if (!VEC) step_ahead();
        if (!cur.active) {
#pragma unroll
          for (int e = 0; e < 16; ++e) gr[e] = x[e] = 0.f;
        }
        turn16(gr, cs, sn, inter);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          ss = fmaf(x[e], x[e], ss);
          dot = fmaf(gr[e] * w[e], x[e], dot);
        }
        const float r = rsqrtf(fmaf(row_sum<LG>(ss), inv_d, p.eps));
        const float m = row_sum<LG>(dot) * inv_d * r * r;
        if (cur.active) {
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            acc[e] = fmaf(gr[e], x[e] * r, acc[e]);
            gr[e] = r * fmaf(-x[e], m, gr[e] * w[e]);
          }
          store8<VEC>(dx, ln.step, gr);
          store8<VEC>(dx + ln.half, ln.step, gr + 8);
        }
        dx += dstep;
      }
    }
  }
  // partial rows of the parts this CTA did not reach are zero
  for (; done_part < 2; ++done_part) flush(done_part);
  if (p.parts < 3) return;

  const QkPart& part = p.part[2];
  const int64_t copies = part.groups * p.row_blocks;
  i = copies * blockIdx.x / gridDim.x;
  i1 = copies * (blockIdx.x + 1) / gridDim.x;
  g = static_cast<int>(i / p.row_blocks);
  rb = i - g * p.row_blocks;
  for (; i < i1; ++i) {
    const int h0 = g * part.group_heads;
    const int heads = min(part.io.heads - h0, part.group_heads);
    const int64_t row = (rb * (kQkThreads / 32) + warp) * (32 >> LG) + (lane >> LG);
    if (row < p.rows && ln.on) {
      int64_t b, n;
      split_row(p, row, b, n);
      copy_heads<T, VEC>(static_cast<const T*>(part.io.in) + b * part.io.ib + n * part.io.in_ +
                             h0 * part.io.ih + ln.off,
                         part.io.ih,
                         static_cast<T*>(part.io.out) + b * part.io.ob + n * part.io.on +
                             h0 * part.io.oh + ln.off,
                         part.io.oh, heads, ln);
    }
    if (++rb == p.row_blocks) {
      rb = 0;
      ++g;
    }
  }
}

// Gain gradients from the partial rows: CTA (x, y) takes 32 columns of part
// y; thread (c, g) adds rows g, g + 32, ... and the 32 sums are added in order.
__global__ void __launch_bounds__(1024) qk_reduce_gain(const float* __restrict__ parts, int blocks,
                                                       int D, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  griddep_wait();
  const int c = 32 * blockIdx.x + threadIdx.x;
  const float* src = parts + static_cast<int64_t>(blockIdx.y) * blocks * D;
  float t = 0.f;
  if (c < D)
    for (int i = threadIdx.y; i < blocks; i += 32) t += src[static_cast<int64_t>(i) * D + c];
  red[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0 && c < D) {
    float s = 0.f;
    for (int i = 0; i < 32; ++i) s += red[i][threadIdx.x];
    float* out = blockIdx.y ? dwk : dwq;
    if (out) out[c] = s;
  }
}

template <typename T, bool VEC, int LG>
cudaError_t backward_lg(const QkParams& p, unsigned grid, cudaStream_t s) {
  static bool attr_set[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  constexpr int kSmem = VEC ? kQkThreads / 32 * kBackStages<T> * kBackStageBytes<T> : 0;
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(qk_backward_kernel<T, VEC, LG>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  return launch_dependent(qk_backward_kernel<T, VEC, LG>, dim3(grid), dim3(kQkThreads), kSmem, s, p);
}

template <typename T>
cudaError_t backward_t(const QkParams& p, bool vec, unsigned grid, cudaStream_t s) {
  if (vec) WSATTN_BY_LANES(backward_lg, T, true)
  WSATTN_BY_LANES(backward_lg, T, false)
}

}  // namespace

cudaError_t launch_qk_backward(const QkParams& p, int dtype, bool vec, int blocks, float* dwq,
                               float* dwk, cudaStream_t s) {
  cudaError_t e;
  if (dtype == WSATTN_BF16)
    e = backward_t<__nv_bfloat16>(p, vec, static_cast<unsigned>(blocks), s);
  else if (dtype == WSATTN_FP16)
    e = backward_t<__half>(p, vec, static_cast<unsigned>(blocks), s);
  else
    e = backward_t<float>(p, vec, static_cast<unsigned>(blocks), s);
  if (e != cudaSuccess || !p.dw_part) return e;
  const int D = 2 * p.rot.pairs;
  return launch_dependent(qk_reduce_gain, dim3((D + 31) / 32, 2), dim3(32, 32), 0, s,
                          static_cast<const float*>(p.dw_part), blocks, D, dwq, dwk);
}

}  // namespace wsattn
