// Linear products on pairs of CTAs: out = residual + act(P Q^T + bias).
//
// Bound by the tensor cores from a few hundred rows up (2 R C K operations
// on (R K + C K + R C) values).  A cluster of two CTAs computes 256 x 256
// (or 256 x 128) outputs with tcgen05.mma.cta_group::2: each CTA stages its
// own 128 rows of P and its own half of Q's rows, so a value that enters
// shared memory meets 256 others, twice what one CTA's 128 x 256 tile gets
// from its shared memory and L2.  The grid is persistent (one pair per two
// SMs); two accumulators of 256 columns fill tensor memory, and the MMAs of
// one tile run while the previous one's epilogue drains.
//   warp 0      TMA: 64-wide contraction slices, ring of 5 (6 at 128 columns)
//   warp 1      MMA issue (CTA 0 of the pair)
//   warp 2      tensor memory
//   warp 3      the bias gradient's partial sums, where there is one
//   warps 4-11  epilogue: thread = row (TMEM lane), two warps per lane
//               quarter, each on half of the tile's columns
// P and Q may lie either way round (the contraction contiguous, or the
// operand's own dimension): only the TMA boxes and the descriptors differ,
// which gives the forward product and both gradients from one kernel.
//
// Tiles are dealt in groups of 8 row tiles, the row the fast index: the 76
// pairs at work together then read about 8 slices of P and 10 of Q, which
// L2 serves to the others.
//
// When the last round of tiles would leave most pairs idle, its tiles are
// split along the contraction instead (`split` parts each, one a pair): the
// partial tiles go to the workspace in fp32, and a small kernel adds them in
// order and applies the epilogue.
//
// One launch may hold two products (both gradients of a linear layer): the
// tiles of the one with the longer contraction go round the pairs first and
// the other's fill in behind them in the order in which pairs fall free, so
// that neither product ends in a wave of its own that is mostly empty.
//
// Epilogue: residual rows are read and outputs are written in whole lines
// through a 128-byte-swizzled staging buffer (TMA store; per-row stores when
// out's rows are not 16-byte aligned, and for the chunk of the last columns when
// they do not fill 16 bytes, which TMA would); sums and activation in fp32, one
// rounding at the end.  With a short contraction it bounds the kernel, so tiles
// without residual, activation and pre-activation take a loop of their own that
// moves 32 columns at a time and does nothing else: 43904 x 192 -> 5120 takes
// 84 us (80 % of a copy's rate) instead of the general loop's 140.  The column
// tile that ends inside 16 bytes goes through the general loop (93 us for 5117
// columns in rows of 5120; with the question in both loops every width takes
// 88).
#include "epilogue.cuh"
#include "ptx.cuh"

namespace wsattn {
namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kEpiWarp0 = 4;
constexpr int kEpiWarps = 8;
constexpr uint32_t kABytes = 128 * kGemmK * 2;  // one CTA's rows of P
constexpr uint32_t kBuf = 32 * 128;             // a warp's 32 rows x 128 bytes
constexpr int kRowGroup = 8;

constexpr int n_stages(int bn) { return bn == 256 ? 5 : 6; }
constexpr uint32_t stage_bytes(int bn) { return kABytes + bn / 2 * kGemmK * 2; }

enum : int { FULL0 = 0, EMPTY0 = 8, ACCFULL0 = 16, ACCEMPTY0 = 18, NBARS = 20 };

__device__ __forceinline__ uint32_t bar(const GemmShared& s, int i) {
  return s.bars + 8u * static_cast<uint32_t>(i);
}

__device__ __noinline__ bool wait_slow(const GemmShared& s, uint32_t b, uint32_t parity, int code,
                                       int values) {
  const long long t0 = clock64();
  while (true) {
    if (mbar_try_wait(b, parity)) return true;
    if (*s.abort_flag) return false;
    if (clock64() - t0 > accumulator_limit(values)) {
      atomicOr(s.status, code);
      *s.abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(const GemmShared& s, uint32_t b, uint32_t parity, int code,
                                     int values = 0) {
  if (mbar_try_wait(b, parity)) return true;
  return wait_slow(s, b, parity, code, values);
}

// A pair's it-th tile: which product, its row and column tile, the steps of
// the contraction, and (part >= 0) which partial tile they make.
struct TileRef {
  int which, tr, tc, k0, k1, part;
};

__device__ __forceinline__ void tile_at(const GemmParams& p, int t, int& tr, int& tc) {
  const int per = kRowGroup * p.tiles_c;
  const int g = t / per, rest = t - g * per;
  const int rows = min(kRowGroup, p.tiles_r - g * kRowGroup);
  tc = rest / rows;
  tr = g * kRowGroup + rest - tc * rows;
}

template <bool TWO>
__device__ __forceinline__ bool nth_tile(const PairParams& pp, int pair, int pairs, int it,
                                         TileRef& r) {
  r.part = -1;
  r.k0 = 0;
  if (!TWO) {
    const GemmParams& p = pp.g[0];
    int t = pair + it * pairs;
    r.which = 0;
    r.k1 = (p.K + kGemmK - 1) / kGemmK;
    if (t >= p.whole_tiles) {
      if (p.split < 2) return false;
      const int u = t - p.whole_tiles, rest = pp.tiles_a - p.whole_tiles;
      if (u >= rest * p.split) return false;
      const int part = u / rest;
      t = p.whole_tiles + u - part * rest;
      r.part = (t - p.whole_tiles) * p.split + part;
      r.k0 = static_cast<int>(static_cast<int64_t>(r.k1) * part / p.split);
      r.k1 = static_cast<int>(static_cast<int64_t>(r.k1) * (part + 1) / p.split);
    }
    tile_at(p, t, r.tr, r.tc);
    return true;
  }
  const int full = pp.tiles_a / pairs, rest = pp.tiles_a - full * pairs;
  const int own = full + (pair < rest ? 1 : 0);
  if (it < own) {
    r.which = 0;
    r.k1 = (pp.g[0].K + kGemmK - 1) / kGemmK;
    tile_at(pp.g[0], pair + it * pairs, r.tr, r.tc);
    return true;
  }
  int t = it - own;
  if (rest == 0) {
    t = t * pairs + pair;
  } else {
    const int others = pairs - rest, head = pp.head_rounds;
    if (pair < rest) t = head * others + t * pairs + pair;
    else if (t < head) t = t * others + pair - rest;
    else t = head * others + (t - head) * pairs + pair;
  }
  if (t >= pp.tiles_b) return false;
  r.which = 1;
  r.k1 = (pp.g[1].K + kGemmK - 1) / kGemmK;
  tile_at(pp.g[1], t, r.tr, r.tc);
  return true;
}

template <int BN, bool TWO>
__device__ void producer(const PairParams& pp, const GemmShared& s, int pair, int pairs,
                         uint32_t rank) {
  constexpr int kStages = n_stages(BN);
  constexpr uint32_t kStage = stage_bytes(BN);
  uint32_t slot = 0, phase = 0, last_phase = 0, issued = 0;
  bool ok = true;
  TileRef ref;
  for (int it = 0; ok && nth_tile<TWO>(pp, pair, pairs, it, ref); ++it) {
    const GemmParams& p = pp.g[TWO ? ref.which : 0];
    const int tr = ref.tr, tc = ref.tc;
    const int kt1 = ref.k1;
    const bool p_mn = p.p_mn != 0, q_mn = p.q_mn != 0;
    const CUtensorMap* const tm_p = &p.tm_p;
    const CUtensorMap* const tm_q = &p.tm_q;
    const int row0 = tr * kPairRows + 128 * static_cast<int>(rank);
    const int col0 = tc * BN + BN / 2 * static_cast<int>(rank);
    if (!WSATTN_BOUNDS(p.status, tr >= 0 && tr < p.tiles_r && tc >= 0 && tc < p.tiles_c))
      break;
    for (int kt = ref.k0; kt < kt1; ++kt) {
      if (!wait(s, bar(s, EMPTY0 + slot), phase ^ 1u, kStatusTimeoutProducer)) {
        ok = false;
        break;
      }
      const uint32_t a = s.stages + slot * kStage, b = a + kABytes;
      // the pair's loads are all counted by CTA 0's barrier
      const uint32_t full = map_to_rank(bar(s, FULL0 + slot), 0);
      if (rank == 0) mbar_arrive_expect_tx(bar(s, FULL0 + slot), 2 * kStage);
      const int k0 = kt * kGemmK;
      if (!p_mn) {
        tma_load_2d_pair(a, tm_p, full, k0, row0);
      } else {
        tma_load_2d_pair(a, tm_p, full, row0, k0);
        tma_load_2d_pair(a + kABytes / 2, tm_p, full, row0 + 64, k0);
      }
      if (!q_mn) {
        tma_load_2d_pair(b, tm_q, full, k0, col0);
      } else {
#pragma unroll
        for (int j = 0; j < BN / 128; ++j)
          tma_load_2d_pair(b + 8192u * j, tm_q, full, col0 + 64 * j, k0);
      }
      last_phase = (last_phase & ~(1u << slot)) | (phase << slot);
      issued |= 1u << slot;
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
  }
  if (ok) return;
  // after an expired wait: copies in flight land whatever the consumers do;
  // CTA 0 waits (bounded) for each slot's last one, and CTA 1 for CTA 0 at
  // the cluster barrier behind this
  if (rank == 0)
    for (int i = 0; i < kStages; ++i) {
      if (!(issued >> i & 1u)) continue;
      const long long t0 = clock64();
      while (!mbar_try_wait(bar(s, FULL0 + i), last_phase >> i & 1u))
        if (clock64() - t0 > kGemmWaitLimit) break;
    }
}

template <int BN, bool TWO>
__device__ void mma_issuer(const PairParams& pp, const GemmShared& s, int pair, int pairs,
                           uint32_t tbase, bool bf16) {
  constexpr int kStages = n_stages(BN);
  constexpr uint32_t kStage = stage_bytes(BN);
  uint32_t slot = 0, phase = 0;
  TileRef ref;
  for (uint32_t it = 0; nth_tile<TWO>(pp, pair, pairs, static_cast<int>(it), ref); ++it) {
    const GemmParams& p = pp.g[TWO ? ref.which : 0];
    const uint32_t idesc = idesc_16_f32(kPairRows, BN, bf16, p.p_mn != 0, p.q_mn != 0);
    // contraction contiguous: 16 values are 32 bytes further on in a row;
    // own dimension contiguous: 16 rows of 128 bytes, 8 KB per 64 columns
    const uint32_t a_lbo = p.p_mn ? 8192u : 16u, b_lbo = p.q_mn ? 8192u : 16u;
    const uint64_t a_step = p.p_mn ? 128 : 2, b_step = p.q_mn ? 128 : 2;
    const int kt0 = ref.k0, kt1 = ref.k1;
    const uint32_t ab = it & 1u, use = it >> 1;
    if (!wait(s, bar(s, ACCEMPTY0 + ab), (use & 1u) ^ 1u, kStatusTimeoutMma)) return;
    tc_fence_after();
    const uint32_t d = tbase + ab * BN;
    for (int kt = kt0; kt < kt1; ++kt) {
      if (!wait(s, bar(s, FULL0 + slot), phase, kStatusTimeoutMma)) return;
      tc_fence_after();
      const uint32_t a = s.stages + slot * kStage;
      const uint64_t ad = sdesc_sw128(a, a_lbo, 1024), bd = sdesc_sw128(a + kABytes, b_lbo, 1024);
#pragma unroll
      for (int kk = 0; kk < kGemmK / 16; ++kk)
        mma_ss_pair(d, ad + kk * a_step, bd + kk * b_step, idesc, kt > kt0 || kk > 0 ? 1u : 0u);
      tc_commit_pair(bar(s, EMPTY0 + slot));
      if (++slot == kStages) {
        slot = 0;
        phase ^= 1u;
      }
    }
    tc_commit_pair(bar(s, ACCFULL0 + ab));
  }
}

// 16-byte unit u of row r in a swizzled staging buffer
__device__ __forceinline__ uint32_t unit_at(uint32_t buf, int r, int u) {
  return buf + 128u * static_cast<uint32_t>(r) + 16u * static_cast<uint32_t>(u ^ (r & 7));
}
template <typename E>
__device__ __forceinline__ uint32_t elem_at(uint32_t buf, int r, int e) {
  const int byte = e * static_cast<int>(sizeof(E));
  return unit_at(buf, r, byte >> 4) + static_cast<uint32_t>(byte & 15);
}
__device__ __forceinline__ void st_elem(uint32_t a, uint16_t v) {
  asm volatile("st.shared.u16 [%0], %1;" ::"r"(a), "h"(v) : "memory");
}
__device__ __forceinline__ void st_elem(uint32_t a, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void ld_elem(uint32_t a, uint16_t& v) {
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
}
__device__ __forceinline__ void ld_elem(uint32_t a, uint32_t& v) {
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
}
template <typename E>
struct Raw {
  using type = uint16_t;
};
template <>
struct Raw<float> {
  using type = uint32_t;
};

// Staging buffer -> global rows, lanes along the columns (rows of any
// alignment).
template <typename E>
__device__ void store_rows(uint32_t buf, void* out, int64_t ld, int64_t row0, int64_t R, int col0,
                           int C, int lane) {
  using W = typename Raw<E>::type;
  constexpr int kCols = 128 / sizeof(E);
  W* o = static_cast<W*>(out);
  for (int r = 0; r < 32 && row0 + r < R; ++r)
#pragma unroll
    for (int e = 0; e < kCols; e += 32)
      if (col0 + e + lane < C) {
        W v;
        ld_elem(elem_at<E>(buf, r, e + lane), v);
        o[(row0 + r) * ld + col0 + e + lane] = v;
      }
}

// Residual rows -> staging buffer: in 16-byte words, all in flight together,
// where the rows are on 16 bytes.
template <typename O>
__device__ __forceinline__ void fetch_rows(const GemmParams& p, int64_t row0, int col0, int lane,
                                           uint4 (&v)[8]) {
  using W = typename Raw<O>::type;
  const int col = col0 + (lane & 7) * (16 / static_cast<int>(sizeof(O)));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t row = row0 + 4 * i + lane / 8;
    v[i] = row < p.R && col < p.C ? *reinterpret_cast<const uint4*>(static_cast<const W*>(p.res) +
                                                                    row * p.ldr + col)
                                  : make_uint4(0, 0, 0, 0);
  }
}
__device__ __forceinline__ void put_rows(uint32_t buf, int lane, const uint4 (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    st_shared_v4(unit_at(buf, 4 * i + lane / 8, lane & 7), v[i].x, v[i].y, v[i].z, v[i].w);
}
template <typename O>
__device__ void load_rows(const GemmParams& p, uint32_t buf, int64_t row0, int col0, int lane) {
  using W = typename Raw<O>::type;
  constexpr int kCols = 128 / sizeof(O);
  const W* res = static_cast<const W*>(p.res);
  for (int r = 0; r < 32; ++r)
#pragma unroll
    for (int e = 0; e < kCols; e += 32) {
      const bool on = row0 + r < p.R && col0 + e + lane < p.C;
      st_elem(elem_at<O>(buf, r, e + lane),
              on ? res[(row0 + r) * p.ldr + col0 + e + lane] : static_cast<W>(0));
    }
}

template <typename T, int ACT>
__device__ __forceinline__ void act16(float (&y)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = act_value<ACT>(y[i]);
}

// Adds eight 16-bit values.
template <typename T>
__device__ __forceinline__ void add8(float* y, const uint4& b) {
  const uint32_t w[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_pair(w[i], T());
    y[2 * i] += f.x;
    y[2 * i + 1] += f.y;
  }
}
// The bias of 16 columns of any alignment (0 past the last one).
template <typename T>
__device__ __forceinline__ void load_bias16(const GemmParams& p, int col, float (&b)[16]) {
  const T* bp = static_cast<const T*>(p.bias) + col;
#pragma unroll
  for (int i = 0; i < 16; ++i) b[i] = col + i < p.C ? to_f32(bp[i]) : 0.f;
}

// A chunk of the output that is the product, with a bias or without: its 128
// bytes a row go to staging in one sweep.  An eighth of the instructions of
// the general way below, which a short contraction would wait for.
template <typename T, typename O>
__device__ __forceinline__ void plain_half(const GemmParams& p, uint32_t taddr, uint32_t buf,
                                           int col0, int first, int lane) {
  constexpr int kBlocks = 4 / sizeof(O);  // of 16 columns
  uint32_t r[kBlocks][16];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) tmem_ld16(taddr + 16 * i, r[i]);
  // a whole chunk's bias is on its way while the accumulator is
  const bool whole = p.bias && p.bias_vec && col0 + 16 * kBlocks <= p.C;
  uint4 raw[2 * kBlocks];
  if (whole) {
    const uint4* bp = reinterpret_cast<const uint4*>(static_cast<const T*>(p.bias) + col0);
#pragma unroll
    for (int i = 0; i < 2 * kBlocks; ++i) raw[i] = __ldg(bp + i);
  }
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) tmem_wait_ld16(r[i]);
  if (whole) {
#pragma unroll
    for (int i = 0; i < 2 * kBlocks; ++i) {
      const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      uint32_t* d = r[i / 2] + 8 * (i % 2);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = unpack_pair(w[e], T());
        d[2 * e] = __float_as_uint(__uint_as_float(d[2 * e]) + f.x);
        d[2 * e + 1] = __float_as_uint(__uint_as_float(d[2 * e + 1]) + f.y);
      }
    }
  } else if (p.bias) {
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      float b[16];
      load_bias16<T>(p, col0 + 16 * i, b);
#pragma unroll
      for (int e = 0; e < 16; ++e) r[i][e] = __float_as_uint(__uint_as_float(r[i][e]) + b[e]);
    }
  }
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    if constexpr (sizeof(O) == 4) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        st_shared_v4(unit_at(buf, lane, first + 4 * i + u), r[i][4 * u], r[i][4 * u + 1], r[i][4 * u + 2],
                     r[i][4 * u + 3]);
    } else {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = pack_pair(__uint_as_float(r[i][8 * u + 2 * e]),
                           __uint_as_float(r[i][8 * u + 2 * e + 1]), T());
        st_shared_v4(unit_at(buf, lane, first + 2 * i + u), w[0], w[1], w[2], w[3]);
      }
    }
  }
}
template <typename T, typename O>
__device__ __forceinline__ void plain_chunk(const GemmParams& p, uint32_t taddr, uint32_t buf,
                                            int col0, int lane) {
  constexpr int kCols = 64 / sizeof(O);
#pragma unroll 1
  for (int i = 0; i < 2; ++i)
    plain_half<T, O>(p, taddr + kCols * i, buf, col0 + kCols * i, 4 * i, lane);
}

template <typename T, typename O, int BN, bool TWO>
__device__ void epilogue(const PairParams& pp, const GemmShared& s, uint32_t staging, int pair,
                         int pairs, uint32_t rank, uint32_t tbase) {
  constexpr int kCols = 128 / sizeof(O);  // columns of a staging chunk
  const int warp = threadIdx.x / 32 - kEpiWarp0, lane = threadIdx.x & 31;
  const int wq = warp & 3, half = warp >> 2;
  const uint32_t tlane = tbase + (static_cast<uint32_t>(32 * wq) << 16);
  const uint32_t buf0 = staging + 2 * kBuf * static_cast<uint32_t>(warp);
  const uint32_t acc_free[2] = {map_to_rank(bar(s, ACCEMPTY0), 0),
                                map_to_rank(bar(s, ACCEMPTY0 + 1), 0)};
  uint32_t ob = 0;
  bool aborted = false;
  TileRef ref;
  for (uint32_t it = 0; !aborted && nth_tile<TWO>(pp, pair, pairs, static_cast<int>(it), ref); ++it) {
    const GemmParams& p = pp.g[TWO ? ref.which : 0];
    const int tr = ref.tr, tc = ref.tc;
    // pre-activations of 16 bits beside outputs of 16 bits go through staging
    const bool stage_pre = p.pre != nullptr && sizeof(O) == 2;
    const uint32_t ab = it & 1u, use = it >> 1;
    const int64_t row0 = static_cast<int64_t>(tr) * kPairRows + 128 * rank + 32 * wq;
    const bool tile_ok =
        WSATTN_BOUNDS(p.status, tr >= 0 && tr < p.tiles_r && tc >= 0 && tc < p.tiles_c);
    if (!TWO && ref.part >= 0) {  // fp32 partial tile [256][256] to global memory
      const bool ok = wait(s, bar(s, ACCFULL0 + ab), use & 1u, kStatusTimeoutSoftmax, p.K);
      if (!__all_sync(0xffffffffu, ok)) {
        aborted = true;
        break;
      }
      tc_fence_after();
      float* dst = p.partial + static_cast<int64_t>(ref.part) * kPairRows * BN +
                   static_cast<int64_t>(128 * rank + 32 * wq + lane) * BN + half * (BN / 2);
#pragma unroll 1
      for (int g = 0; tile_ok && g < BN / 32; ++g) {
        uint32_t r[16];
        tmem_ld16(tlane + ab * BN + half * (BN / 2) + 16 * g, r);
        tmem_wait_ld16(r);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(dst + 16 * g + 4 * i) =
              make_uint4(r[4 * i], r[4 * i + 1], r[4 * i + 2], r[4 * i + 3]);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(acc_free[ab]);
      continue;
    }
    if (!p.pre && !p.res && p.act == WSATTN_ACT_NONE && tc != p.edge_tile) {
      bool ok = true;
#pragma unroll 1
      for (int j = 0; ok && j < BN / 2 / kCols; ++j) {
        const int tcol = half * (BN / 2) + j * kCols;
        const int col0 = tc * BN + tcol;
        const bool on = tile_ok && row0 < p.R && col0 < p.C;
        const uint32_t buf = buf0 + ob * kBuf;
        if (on && lane == 0) bulk_wait_read_1();  // the buffer's previous store has read it
        if (j == 0) {
          ok = __all_sync(0xffffffffu,
                          wait(s, bar(s, ACCFULL0 + ab), use & 1u, kStatusTimeoutSoftmax, p.K));
          if (!ok) break;
          tc_fence_after();
        }
        __syncwarp();
        if (on) plain_chunk<T, O>(p, tlane + ab * BN + tcol, buf, col0, lane);
        if (j == BN / 2 / kCols - 1) {  // this warp has read its columns of the accumulator
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_relaxed(acc_free[ab]);
        }
        if (!on) continue;
        fence_proxy_async_smem();
        __syncwarp();
        if (!p.out_vec) store_rows<O>(buf, p.out, p.ldo, row0, p.R, col0, p.C, lane);
        else if (lane == 0) tma_store_2d(&p.tm_out, buf, col0, static_cast<int>(row0));
        if (lane == 0) bulk_commit_group();
        __syncwarp();
        ob ^= 1u;
      }
      aborted = !ok;
      continue;
    }
    bool waited = false;
#pragma unroll 1
    for (int j = 0; j < BN / 2 / kCols; ++j) {
      const int tcol = half * (BN / 2) + j * kCols;
      const int col0 = tc * BN + tcol;
      const bool on = tile_ok && row0 < p.R && col0 < p.C;
      if (stage_pre) ob = 1;
      const uint32_t buf = buf0 + ob * kBuf;
      if (on) {
        // the buffer's previous store has read it (with pre-activations,
        // both buffers')
        if (lane == 0) {
          if (stage_pre) bulk_wait_read_all();
          else bulk_wait_read_1();
        }
        __syncwarp();
        if (p.res_vec) {
          uint4 res[8];
          fetch_rows<O>(p, row0, col0, lane, res);
          put_rows(buf, lane, res);
        } else if (p.res) {
          load_rows<O>(p, buf, row0, col0, lane);
        }
      }
      if (!waited) {
        const bool ok = wait(s, bar(s, ACCFULL0 + ab), use & 1u, kStatusTimeoutSoftmax, p.K);
        if (!__all_sync(0xffffffffu, ok)) {
          aborted = true;
          break;
        }
        tc_fence_after();
        waited = true;
      }
      __syncwarp();
      // 16 columns at a time: the next ones' accumulators and bias are on
      // their way while these are worked on
      const bool bias_fast = p.bias_vec && col0 + kCols <= p.C;
      uint32_t r[16];
      uint4 b0, b1;
      auto start = [&](int g) {
        tmem_ld16(tlane + ab * BN + tcol + 16 * g, r);
        if (bias_fast) {
          const uint4* bp =
              reinterpret_cast<const uint4*>(static_cast<const T*>(p.bias) + col0 + 16 * g);
          b0 = __ldg(bp);
          b1 = __ldg(bp + 1);
        }
      };
      if (on) {
        start(0);
        tmem_wait_ld16(r);
      }
#pragma unroll 1
      for (int g = 0; on && g < kCols / 16; ++g) {
        const int col = col0 + 16 * g;
        float y[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(r[i]);
        if (bias_fast) {
          add8<T>(y, b0);
          add8<T>(y + 8, b1);
        } else if (p.bias) {
          float bv[16];
          load_bias16<T>(p, col, bv);
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] += bv[i];
        }
        // (the last ones once more: no branch between the load and its wait below
        // may leave the registers in two states)
        start(g + 1 < kCols / 16 ? g + 1 : g);
        if (p.pre) {
          uint32_t w[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) w[i] = pack_pair(y[2 * i], y[2 * i + 1], T());
          if (stage_pre) {
            st_shared_v4(unit_at(buf0, lane, 2 * g), w[0], w[1], w[2], w[3]);
            st_shared_v4(unit_at(buf0, lane, 2 * g + 1), w[4], w[5], w[6], w[7]);
          } else if (row0 + lane < p.R) {
            uint16_t* o = static_cast<uint16_t*>(p.pre) + (row0 + lane) * p.ldp + col;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (col + i < p.C) o[i] = static_cast<uint16_t>(w[i / 2] >> (16 * (i & 1)));
          }
        }
        switch (p.act) {
          case WSATTN_ACT_GELU: act16<T, WSATTN_ACT_GELU>(y); break;
          case WSATTN_ACT_GELU_TANH: act16<T, WSATTN_ACT_GELU_TANH>(y); break;
          case WSATTN_ACT_SILU: act16<T, WSATTN_ACT_SILU>(y); break;
          default: break;
        }
        if constexpr (sizeof(O) == 4) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint32_t a = unit_at(buf, lane, 4 * g + u);
            float4 v = make_float4(y[4 * u], y[4 * u + 1], y[4 * u + 2], y[4 * u + 3]);
            if (p.res) {
              const uint4 q = ld_shared_v4(a);
              v.x += __uint_as_float(q.x);
              v.y += __uint_as_float(q.y);
              v.z += __uint_as_float(q.z);
              v.w += __uint_as_float(q.w);
            }
            st_shared_v4(a, __float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                         __float_as_uint(v.w));
          }
        } else {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t a = unit_at(buf, lane, 2 * g + u);
            if (p.res) {
              const uint4 q = ld_shared_v4(a);
              const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float2 f = unpack_pair(w[i], T());
                y[8 * u + 2 * i] += f.x;
                y[8 * u + 2 * i + 1] += f.y;
              }
            }
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_pair(y[8 * u + 2 * i], y[8 * u + 2 * i + 1], T());
            st_shared_v4(a, w[0], w[1], w[2], w[3]);
          }
        }
        tmem_wait_ld16(r);
      }
      if (j == BN / 2 / kCols - 1) {  // this warp has read its columns of the accumulator
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_relaxed(acc_free[ab]);
      }
      if (!on) continue;
      fence_proxy_async_smem();
      __syncwarp();
      if (stage_pre) {
        if (col0 < p.pre_tma) {
          if (lane == 0) tma_store_2d(&p.tm_pre, buf0, col0, static_cast<int>(row0));
        } else {
          store_rows<T>(buf0, p.pre, p.ldp, row0, p.R, col0, p.C, lane);
        }
      }
      if (col0 < p.out_tma) {
        if (lane == 0) tma_store_2d(&p.tm_out, buf, col0, static_cast<int>(row0));
      } else {
        store_rows<O>(buf, p.out, p.ldo, row0, p.R, col0, p.C, lane);
      }
      if (lane == 0) bulk_commit_group();
      __syncwarp();
      ob ^= 1u;
    }
  }
  if (lane == 0) bulk_wait_all();  // the stores have left shared memory before the CTA does
}

template <typename T, typename O, int BN, bool TWO>
__global__ void __launch_bounds__(kThreads, 1) gemm_pair_kernel(const __grid_constant__ PairParams p) {
  extern __shared__ uint8_t smem_raw[];
  constexpr int kStages = n_stages(BN);
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  GemmShared s;
  s.stages = base;
  const uint32_t staging = base + kStages * stage_bytes(BN);
  s.bars = staging + 2 * kEpiWarps * kBuf;
  uint8_t* gb = smem_raw + (s.bars - raw);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(gb + 8 * NBARS);
  s.abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  s.status = p.g[0].status;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = static_cast<int>(blockIdx.x >> 1), pairs = static_cast<int>(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(s, FULL0 + i), 1);
      mbar_init(bar(s, EMPTY0 + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(s, ACCFULL0 + i), 1);
      mbar_init(bar(s, ACCEMPTY0 + i), 2 * kEpiWarps);  // the epilogue warps of both CTAs
    }
    *s.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tensormap(&p.g[0].tm_p);
    prefetch_tensormap(&p.g[0].tm_q);
    if (p.g[0].out_tma) prefetch_tensormap(&p.g[0].tm_out);
  }
  if (warp == 2) {
    tmem_alloc_pair(smem_u32(tslot), 2 * BN);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are ready before either signals them
  tc_fence_after();
  const uint32_t tbase = *tslot;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    if (lane == 0) producer<BN, TWO>(p, s, pair, pairs, rank);
  } else if (warp == 1) {
    if (lane == 0 && rank == 0)
      mma_issuer<BN, TWO>(p, s, pair, pairs, tbase, !IsHalf<T>::value);
  } else if (warp == 3) {
    side_sums(p.g[0], static_cast<int>(blockIdx.x) * 32 + lane, static_cast<int>(gridDim.x) * 32);
  } else if (warp >= kEpiWarp0) {
    epilogue<T, O, BN, TWO>(p, s, staging, pair, pairs, rank, tbase);
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other may signal or feed it
  tc_fence_after();
  if (warp == 2) tmem_dealloc_pair(tbase, 2 * BN);
}

template <typename T, typename O, int BN, bool TWO>
cudaError_t launch(PairParams* p, int sms, cudaStream_t s) {
  static bool attr_set[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  const size_t smem = pair_smem_bytes(BN);
  if (!attr_set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(gemm_pair_kernel<T, O, BN, TWO>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int64_t ta = static_cast<int64_t>(p->g[0].tiles_r) * p->g[0].tiles_c;
  const int64_t tb = static_cast<int64_t>(p->g[1].tiles_r) * p->g[1].tiles_c;
  // the index of the last tile, plus one round, has to fit an int
  if (ta + tb > INT32_MAX - 4 * sms) return cudaErrorInvalidValue;
  p->tiles_a = static_cast<int>(ta);
  p->tiles_b = static_cast<int>(tb);
  const int ka = (p->g[0].K + kGemmK - 1) / kGemmK, kb = (p->g[1].K + kGemmK - 1) / kGemmK;
  p->head_rounds = tb > 0 ? (ka + kb - 1) / kb : 0;
  const GemmParams& g = p->g[0];
  // tiles and parts of tiles to deal out
  const int64_t units = tb > 0 || g.split < 2 ? ta + tb
                                              : g.whole_tiles + (ta - g.whole_tiles) * g.split;
  const int pairs = static_cast<int>(units < sms / 2 ? units : sms / 2);
  return launch_cluster(gemm_pair_kernel<T, O, BN, TWO>, dim3(2 * pairs), dim3(kThreads), 2, smem,
                        s, *p);
}

// Sums of a split tile's partial tiles, with the epilogue.  A thread takes
// four columns of a row; the parts are added in their order.
template <typename T, typename O>
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ GemmParams p) {
  constexpr int kTile = kPairRows * 256;
  griddep_wait();
  griddep_launch_dependents();
  const int tile = static_cast<int>(blockIdx.x / (kTile / 1024));
  const int e = static_cast<int>(blockIdx.x % (kTile / 1024)) * 1024 + 4 * static_cast<int>(threadIdx.x);
  int tr, tc;
  tile_at(p, p.whole_tiles + tile, tr, tc);
  const int64_t row = static_cast<int64_t>(tr) * kPairRows + e / 256;
  const int col = tc * 256 + e % 256;
  if (row >= p.R || col >= p.C) return;
  const float* src = p.partial + static_cast<int64_t>(tile) * p.split * kTile + e;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = 0; i < p.split; ++i) {
    const float4 q = *reinterpret_cast<const float4*>(src + static_cast<int64_t>(i) * kTile);
    v.x += q.x;
    v.y += q.y;
    v.z += q.z;
    v.w += q.w;
  }
  const float y4[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int c = col + i;
    if (c >= p.C) break;
    float y = y4[i];
    if (p.bias) y += to_f32(static_cast<const T*>(p.bias)[c]);
    if (p.pre) static_cast<T*>(p.pre)[row * p.ldp + c] = from_f32<T>(y);
    y = act_any(p.act, y);
    if (p.res) y += to_f32(static_cast<const O*>(p.res)[row * p.ldr + c]);
    static_cast<O*>(p.out)[row * p.ldo + c] = from_f32<O>(y);
  }
}

template <typename T, typename O>
cudaError_t launch_bn(PairParams* p, int pair_cols, int sms, cudaStream_t s) {
  if constexpr (sizeof(O) == 2) {  // two products: the gradients, 256 columns
    if (p->g[1].tiles_r > 0) return launch<T, O, 256, true>(p, sms, s);
  }
  if (pair_cols == 128) return launch<T, O, 128, false>(p, sms, s);
  const cudaError_t e = launch<T, O, 256, false>(p, sms, s);
  const GemmParams& g = p->g[0];
  if (e != cudaSuccess || g.split < 2) return e;
  const int rest = p->tiles_a - g.whole_tiles;
  return launch_dependent(finish_kernel<T, O>, dim3(rest * (kPairRows * 256 / 1024)), dim3(256), 0,
                          s, g);
}

}  // namespace

size_t pair_smem_bytes(int bn) {
  return 1024 + n_stages(bn) * stage_bytes(bn) + 2 * kEpiWarps * kBuf + 8 * NBARS + 16;
}

cudaError_t launch_gemm_pair(PairParams* p, int dtype, bool out_f32, int pair_cols, int sms,
                             cudaStream_t s) {
  if (dtype == WSATTN_BF16)
    return out_f32 ? launch_bn<__nv_bfloat16, float>(p, pair_cols, sms, s)
                   : launch_bn<__nv_bfloat16, __nv_bfloat16>(p, pair_cols, sms, s);
  return out_f32 ? launch_bn<__half, float>(p, pair_cols, sms, s)
                 : launch_bn<__half, __half>(p, pair_cols, sms, s);
}

}  // namespace wsattn
