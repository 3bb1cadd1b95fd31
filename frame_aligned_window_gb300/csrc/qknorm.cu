// Rotary positions and per-head norms, forward (qknorm.cuh has the formulas
// and what the passes share).
#include "qknorm.cuh"

namespace wsattn {
namespace {

using namespace ptx;
using namespace qk;

// One warp: the heads of one group, each lane group for one token.
template <typename T, bool VEC, int LG, bool NORM>
__global__ void __launch_bounds__(kQkThreads) qk_forward_kernel(const __grid_constant__ QkParams p) {
  // heads whose loads are in flight together (with the norm's registers, four of
  // 16 bits are 2 % faster at 40 heads, two 5 to 30 % at 12 and fewer)
  constexpr int U = sizeof(T) == 4 || NORM ? 2 : 4;
  const Lane ln = make_lane<T, LG>(p.rot);
  const int g = static_cast<int>(blockIdx.x % p.groups);
  const int64_t rb = blockIdx.x / p.groups;
  constexpr int kPerWarp = 32 >> LG;
  const int64_t row =
      (rb * (kQkThreads / 32) + threadIdx.x / 32) * kPerWarp + ((threadIdx.x & 31) >> LG);
  int pi = 0;
  while (pi + 1 < p.parts && g >= p.part[pi + 1].group0) ++pi;
  const QkPart& part = p.part[pi];
  const int h0 = (g - part.group0) * part.group_heads;
  const int heads = min(part.io.heads - h0, part.group_heads);
  const bool active = row < p.rows && ln.on &&
                      WSATTN_BOUNDS(p.status, g < p.groups && h0 >= 0 && heads >= 1 &&
                                                  h0 + heads <= part.io.heads &&
                                                  16 * ln.c + 16 <= 2 * ln.half);
  int64_t b = 0, n = 0;
  if (active) split_row(p, row, b, n);
  const int64_t sstep = part.io.ih, dstep = part.io.oh;
  const T* src = static_cast<const T*>(part.io.in) + b * part.io.ib + n * part.io.in_ + h0 * sstep +
                 ln.off;
  T* dst =
      static_cast<T*>(part.io.out) + b * part.io.ob + n * part.io.on + h0 * dstep + ln.off;
  griddep_wait();
  griddep_launch_dependents();
  if (!part.turn) {
    if (active) copy_heads<T, VEC>(src, sstep, dst, dstep, heads, ln);
    return;
  }
  // the first loads go out before the angles are formed
  Half8<T> r0[U], r1[U];
  auto load = [&](int left) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (active && u < left) {
        r0[u] = load8<VEC>(src + u * sstep, ln.step);
        r1[u] = load8<VEC>(src + u * sstep + ln.half, ln.step);
      } else {
        r0[u] = Half8<T>{};
        r1[u] = Half8<T>{};
      }
  };
  load(heads);
  float cs[8], sn[8], w[16];
  if (active)
    lane_angles<T>(p.rot, ln, p.pos + b * p.pos_b + n * p.rot.axes, static_cast<float>(part.turn), cs,
                sn);
  if (NORM) load_gain<T>(p, part, ln, w);
  const float inv_d = 0.5f / static_cast<float>(p.rot.pairs);
  const bool inter = p.rot.interleaved != 0;

  auto head = [&](int u) {
    float x[16];
    unpack8(r0[u], x);
    unpack8(r1[u], x + 8);
    if (NORM) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss = fmaf(x[i], x[i], ss);
      const float r = rsqrtf(fmaf(row_sum<LG>(ss), inv_d, p.eps));
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= r * w[i];
    }
    turn16(x, cs, sn, inter);
    if (active) {
      store8<VEC>(dst + u * dstep, ln.step, x);
      store8<VEC>(dst + u * dstep + ln.half, ln.step, x + 8);
    }
  };
  for (int h = 0; h < heads; h += U) {
    if (h > 0) load(heads - h);
    if (heads - h >= U) {  // all of them, interleaved by the compiler
#pragma unroll
      for (int u = 0; u < U; ++u) head(u);
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (u < heads - h) head(u);
    }
    src += U * sstep;
    dst += U * dstep;
  }
}

template <typename T, bool VEC, int LG>
cudaError_t forward_lg(const QkParams& p, unsigned grid, cudaStream_t s) {
  return p.part[0].norm
             ? launch_dependent(qk_forward_kernel<T, VEC, LG, true>, dim3(grid), dim3(kQkThreads),
                                0, s, p)
             : launch_dependent(qk_forward_kernel<T, VEC, LG, false>, dim3(grid), dim3(kQkThreads),
                                0, s, p);
}
template <typename T>
cudaError_t forward_t(const QkParams& p, bool vec, cudaStream_t s) {
  const int64_t blocks = p.row_blocks * p.groups;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (vec) WSATTN_BY_LANES(forward_lg, T, true)
  WSATTN_BY_LANES(forward_lg, T, false)
}

}  // namespace

cudaError_t launch_qk_forward(const QkParams& p, int dtype, bool vec, cudaStream_t s) {
  if (dtype == WSATTN_BF16) return forward_t<__nv_bfloat16>(p, vec, s);
  if (dtype == WSATTN_FP16) return forward_t<__half>(p, vec, s);
  return forward_t<float>(p, vec, s);
}

}  // namespace wsattn
