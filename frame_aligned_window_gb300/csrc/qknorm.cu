// Rotary positions on several axes, alone or in one pass with the per-head
// RMS norm of queries and keys, and their gradients.
//
//   forward   y = R_a (g * x r),          r = 1 / sqrt(mean_d x_d^2 + eps)
//   backward  h = R_-a dy,  u = g * h,  xh = x r
//             dx = r (u - xh mean_d(u xh)),   dg = sum over rows of h * xh
//
// R_a turns pair p of a head by a_p = pos[axis(p)] * freq(p).  The norm and
// the gain act on a whole head row and the turn on pairs of it, so one read
// of x and one write of y is all the traffic there has to be: the passes are
// bound by HBM (the angles come from the positions, 4 bytes per token and
// axis, not from a table of D values per token).
//
// Work split: 2^l lanes (the least power of two that covers D / 16) hold one
// head row, 16 elements a lane in 16-byte pieces, the same ones of each half
// of the head: element e of the first half and e + D/2 then sit in one thread,
// which serves both pair layouts without an exchange.  A lane group keeps one
// token and walks its heads: sine and cosine are formed once for all heads
// of q (or k), the loads of several heads are in flight together, and the
// lane groups of a warp hold neighbouring tokens, so that the packed
// [B, H, N, D] side is written in runs of whole lines.  A launch with few
// tokens splits the heads into groups until every SM has warps.
//
// Angles: pos * (freq / 2 pi) is an fp32 product with its exact error term
// and a second float of the rate; the whole revolutions are dropped before
// the sum is rounded, so the fraction of a turn is good to 2^-25 at any
// position (an fp32 angle at position 70000 would be off by 2^-9).
#include "ops.h"
#include "ptx.cuh"

namespace wsattn {
namespace {

using namespace ptx;

template <typename T>
struct Half8;  // 8 elements as raw words
template <>
struct Half8<float> {
  uint4 a, b;
};
template <>
struct Half8<__nv_bfloat16> {
  uint4 a;
};
template <>
struct Half8<__half> {
  uint4 a;
};

__device__ __forceinline__ void words2(uint32_t w, float& lo, float& hi, __nv_bfloat16) {
  lo = __uint_as_float(w << 16);
  hi = __uint_as_float(w & 0xFFFF0000u);
}
__device__ __forceinline__ void words2(uint32_t w, float& lo, float& hi, __half) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w));
  lo = f.x;
  hi = f.y;
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi, __half) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t elem_bits(float v) { return __float_as_uint(v); }
__device__ __forceinline__ uint32_t elem_bits(__nv_bfloat16 v) { return __bfloat16_as_ushort(v); }
__device__ __forceinline__ uint32_t elem_bits(__half v) { return __half_as_ushort(v); }

// Raw 8-element load; VEC: 16-byte loads, else element by element (rows that
// start on any element).
template <bool VEC>
__device__ __forceinline__ Half8<float> load8(const float* p, int step) {
  const float* q = p + step;
  Half8<float> r;
  if (VEC) {
    r.a = *reinterpret_cast<const uint4*>(p);
    r.b = *reinterpret_cast<const uint4*>(q);
  } else {
    r.a = make_uint4(elem_bits(p[0]), elem_bits(p[1]), elem_bits(p[2]), elem_bits(p[3]));
    r.b = make_uint4(elem_bits(q[0]), elem_bits(q[1]), elem_bits(q[2]), elem_bits(q[3]));
  }
  return r;
}
template <bool VEC, typename T>
__device__ __forceinline__ Half8<T> load8(const T* p, int) {
  Half8<T> r;
  if (VEC) {
    r.a = *reinterpret_cast<const uint4*>(p);
  } else {
    r.a = make_uint4(elem_bits(p[0]) | elem_bits(p[1]) << 16, elem_bits(p[2]) | elem_bits(p[3]) << 16,
                     elem_bits(p[4]) | elem_bits(p[5]) << 16, elem_bits(p[6]) | elem_bits(p[7]) << 16);
  }
  return r;
}

__device__ __forceinline__ void unpack8(const Half8<float>& r, float* f) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
}
template <typename T>
__device__ __forceinline__ void unpack8(const Half8<T>& r, float* f) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) words2(w[i], f[2 * i], f[2 * i + 1], T());
}

template <bool VEC>
__device__ __forceinline__ void store8(float* p, int step, const float* f) {
  float* q = p + step;
  if (VEC) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(q) = make_float4(f[4], f[5], f[6], f[7]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = f[4 + i];
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void store8(T* p, int, const float* f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2(f[2 * i], f[2 * i + 1], T());
  if (VEC) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    uint16_t* u = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[2 * i] = static_cast<uint16_t>(w[i]);
      u[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
    }
  }
}

// The lane's place in its head row: eight elements of each half of the head,
// in 16 bits elements [8c, 8c + 8), in fp32 [4c, 4c + 4) of the half's first
// half and of its second (either way neighbouring lanes touch neighbouring
// 16 bytes).
struct Lane {
  int c;
  bool on;   // the lane holds a piece (D / 16 need not be a power of two)
  int half;  // D / 2
  int off;   // its first element
  int step;  // fp32: from its first four elements to its second
};

template <typename T, int LG>
__device__ __forceinline__ Lane make_lane(const RotTable& t) {
  Lane ln;
  ln.c = threadIdx.x & ((1 << LG) - 1);
  ln.half = t.pairs;
  ln.on = 16 * ln.c < 2 * t.pairs;
  ln.off = (sizeof(T) == 4 ? 4 : 8) * ln.c;
  ln.step = t.pairs / 2;
  return ln;
}
// Element (of the head) that the lane's i-th value is.
template <typename T>
__device__ __forceinline__ int lane_element(const Lane& ln, int i) {
  const int in_half = sizeof(T) == 4 ? (i & 4 ? ln.step : 0) + (i & 3) : i & 7;
  return (i < 8 ? 0 : ln.half) + ln.off + in_half;
}

// Row (of B * N) -> batch element and token.
__device__ __forceinline__ void split_row(const QkParams& p, int64_t row, int64_t& b, int64_t& n) {
  if (p.rows <= INT32_MAX) {
    const uint32_t q = static_cast<uint32_t>(row) / static_cast<uint32_t>(p.tokens);
    b = q;
    n = static_cast<uint32_t>(row) - q * static_cast<uint32_t>(p.tokens);
  } else {
    b = row / p.tokens;
    n = row - b * p.tokens;
  }
}

// The rates of a lane's eight pairs, in the order in which turn16 takes them.
// They are read from the kernel's parameters through generic addresses:
// indexed reads of constant memory would go lane by lane.
struct Rates {
  float hi[8], lo[8];
  uint32_t axis[8];
};
// N consecutive pairs from p0 on
template <int N>
__device__ __forceinline__ void read_rates(const RotTable* g, int p0, float* hi, float* lo,
                                           uint32_t* axis) {
  if constexpr (N == 4) {
    const float4 h = *reinterpret_cast<const float4*>(g->hi + p0);
    const float4 l = *reinterpret_cast<const float4*>(g->lo + p0);
    const uint32_t a = *reinterpret_cast<const uint32_t*>(g->axis + p0);
    hi[0] = h.x, hi[1] = h.y, hi[2] = h.z, hi[3] = h.w;
    lo[0] = l.x, lo[1] = l.y, lo[2] = l.z, lo[3] = l.w;
#pragma unroll
    for (int i = 0; i < 4; ++i) axis[i] = a >> (8 * i) & 255u;
  } else {
    const float2 h = *reinterpret_cast<const float2*>(g->hi + p0);
    const float2 l = *reinterpret_cast<const float2*>(g->lo + p0);
    const uint32_t a = *reinterpret_cast<const uint16_t*>(g->axis + p0);
    hi[0] = h.x, hi[1] = h.y;
    lo[0] = l.x, lo[1] = l.y;
    axis[0] = a & 255u, axis[1] = a >> 8;
  }
}
template <typename T>
__device__ __forceinline__ Rates lane_rates(const RotTable& t, const Lane& ln) {
  const RotTable* g = &t;
  asm volatile("" : "+l"(g));  // an address like any other from here on
  Rates r;
  if (!t.interleaved) {  // pair e: elements e and e + D / 2
    const int second = sizeof(T) == 4 ? ln.off + ln.step : ln.off + 4;
    read_rates<4>(g, ln.off, r.hi, r.lo, r.axis);
    read_rates<4>(g, second, r.hi + 4, r.lo + 4, r.axis + 4);
  } else if constexpr (sizeof(T) == 4) {  // pair e / 2: elements e and e + 1
#pragma unroll
    for (int k = 0; k < 4; ++k)
      read_rates<2>(g, (ln.off + k * ln.step) / 2, r.hi + 2 * k, r.lo + 2 * k, r.axis + 2 * k);
  } else {
    read_rates<4>(g, ln.off / 2, r.hi, r.lo, r.axis);
    read_rates<4>(g, (ln.half + ln.off) / 2, r.hi + 4, r.lo + 4, r.axis + 4);
  }
  return r;
}

template <typename T>
__device__ __forceinline__ void lane_angles(const RotTable& t, const Lane& ln, const float* pos,
                                            float sign, float (&cs)[8], float (&sn)[8]) {
  float x[kRotMaxAxes];
#pragma unroll
  for (int a = 0; a < kRotMaxAxes; ++a) x[a] = a < t.axes ? pos[a] : 0.f;
  const Rates r = lane_rates<T>(t, ln);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float w = r.hi[i], wl = r.lo[i];
    const uint32_t a = r.axis[i];
    const float v = a < 2 ? (a == 0 ? x[0] : x[1]) : (a == 2 ? x[2] : x[3]);
    const float hi = v * w;
    const float err = fmaf(v, w, -hi);
    const float frac = (hi - rintf(hi)) + fmaf(v, wl, err);
    float s, c;
    sincospif(2.f * frac, &s, &c);
    cs[i] = c;
    sn[i] = sign * s;
  }
}

// Turns the lane's 16 elements (x: 8 of each half) in place.
__device__ __forceinline__ void turn16(float (&x)[16], const float (&cs)[8], const float (&sn)[8],
                                       bool interleaved) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = fmaf(a, cs[i], -b * sn[i]);
      x[2 * i + 1] = fmaf(a, sn[i], b * cs[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float a = x[i], b = x[8 + i];
      x[i] = fmaf(a, cs[i], -b * sn[i]);
      x[8 + i] = fmaf(a, sn[i], b * cs[i]);
    }
  }
}

// Sum over the 2^LG lanes of a head row (every lane gets it).
template <int LG>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 1 << LG >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The lane's gains, from E values laid out as its T elements are.
template <typename E, typename T>
__device__ __forceinline__ void gain16(const void* weight, const Lane& ln, float (&w)[16]) {
  const E* g = static_cast<const E*>(weight) + ln.off;
  // fp32 gains of 16-bit heads: eight in a row
  const int step = sizeof(T) == 4 ? ln.step : 4;
  if ((reinterpret_cast<uintptr_t>(weight) & 15u) == 0) {
    unpack8(load8<true>(g, step), w);
    unpack8(load8<true>(g + ln.half, step), w + 8);
  } else {
    unpack8(load8<false>(g, step), w);
    unpack8(load8<false>(g + ln.half, step), w + 8);
  }
}
template <typename T>
__device__ __forceinline__ void load_gain(const QkParams& p, const QkPart& part, const Lane& ln,
                                          float (&w)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) w[i] = 1.f;
  if (!part.weight || !ln.on) return;
  if (p.weight_f32) gain16<float, T>(part.weight, ln, w);
  else gain16<T, T>(part.weight, ln, w);
}

template <bool VEC>
__device__ __forceinline__ void store_raw8(float* p, int step, const Half8<float>& r) {
  float f[8];
  unpack8(r, f);
  store8<VEC>(p, step, f);
}
template <bool VEC, typename T>
__device__ __forceinline__ void store_raw8(T* p, int, const Half8<T>& r) {
  if (VEC) {
    *reinterpret_cast<uint4*>(p) = r.a;
  } else {
    const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
    uint16_t* u = reinterpret_cast<uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      u[2 * i] = static_cast<uint16_t>(w[i]);
      u[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
    }
  }
}

// Copies a lane's share of `heads` head rows (v: neither norm nor turn).
template <typename T, bool VEC>
__device__ __forceinline__ void copy_heads(const T* src, int64_t sstep, T* dst, int64_t dstep,
                                           int heads, const Lane& ln) {
  constexpr int U = sizeof(T) == 4 ? 2 : 4;
  for (int h = 0; h < heads; h += U) {
    Half8<T> r0[U], r1[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u < heads) {
        r0[u] = load8<VEC>(src + u * sstep, ln.step);
        r1[u] = load8<VEC>(src + u * sstep + ln.half, ln.step);
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (h + u < heads) {
        store_raw8<VEC>(dst + u * dstep, ln.step, r0[u]);
        store_raw8<VEC>(dst + u * dstep + ln.half, ln.step, r1[u]);
      }
    src += U * sstep;
    dst += U * dstep;
  }
}

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
cudaError_t forward_lg(const QkParams& p, unsigned grid, cudaStream_t s) {
  return p.part[0].norm
             ? launch_dependent(qk_forward_kernel<T, VEC, LG, true>, dim3(grid), dim3(kQkThreads),
                                0, s, p)
             : launch_dependent(qk_forward_kernel<T, VEC, LG, false>, dim3(grid), dim3(kQkThreads),
                                0, s, p);
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

// Calls F<T, VEC, LG> for the lanes of a head row.
#define WSATTN_BY_LANES(F, T, VEC)                  \
  switch (p.lanes_log2) {                           \
    case 0: return F<T, VEC, 0>(p, grid, s);        \
    case 1: return F<T, VEC, 1>(p, grid, s);        \
    case 2: return F<T, VEC, 2>(p, grid, s);        \
    case 3: return F<T, VEC, 3>(p, grid, s);        \
    default: return F<T, VEC, 4>(p, grid, s);       \
  }

template <typename T>
cudaError_t forward_t(const QkParams& p, bool vec, cudaStream_t s) {
  const int64_t blocks = p.row_blocks * p.groups;
  if (blocks > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  if (vec) WSATTN_BY_LANES(forward_lg, T, true)
  WSATTN_BY_LANES(forward_lg, T, false)
}

template <typename T>
cudaError_t backward_t(const QkParams& p, bool vec, unsigned grid, cudaStream_t s) {
  if (vec) WSATTN_BY_LANES(backward_lg, T, true)
  WSATTN_BY_LANES(backward_lg, T, false)
}

}  // namespace

cudaError_t launch_qk_forward(const QkParams& p, int dtype, bool vec, cudaStream_t s) {
  if (dtype == WSATTN_BF16) return forward_t<__nv_bfloat16>(p, vec, s);
  if (dtype == WSATTN_FP16) return forward_t<__half>(p, vec, s);
  return forward_t<float>(p, vec, s);
}

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
