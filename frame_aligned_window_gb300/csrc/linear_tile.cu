// Linear products on single CTAs: out = residual + act(P Q^T + bias) for few
// rows, and for shapes too small to fill the machine with 256 x 256 tiles.
//
// With a few rows the product reads Q (the weights) once and does little
// with it: bound by HBM.  The operands trade places here: 128 columns of the
// output (rows of Q) are the MMA's M, the BN = 16 .. 128 rows of P its N, so
// the padding of a single row costs 15 rows of tensor-core time instead of
// 127, and the weights stream through a TMA ring of 16 KB slices.  When the
// tiles alone do not fill the SMs, a cluster of `split` CTAs shares the
// contraction of one tile: each leaves its fp32 partial tile in its own
// shared memory, and the CTAs add them through distributed shared memory,
// each for its own rows and in the order of the ranks, so that the sums do
// not depend on timing and no partial result goes to global memory.
//   warp 0     TMA
//   warp 1     MMA issue, tensor memory
//   warps 2-5  epilogue: the accumulator goes to shared memory (over the idle
//              ring), from where a warp takes whole rows of 128 columns
#include "epilogue.cuh"
#include "ptx.cuh"

namespace wsattn {
namespace {

using namespace ptx;

constexpr int kThreads = 192;
constexpr uint32_t kQBytes = kTileCols * kGemmK * 2;
constexpr int kMaxStages = 12;

enum : int { FULL0 = 0, EMPTY0 = kMaxStages, ACCFULL = 2 * kMaxStages, NBARS = 2 * kMaxStages + 1 };

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

__device__ void producer(const GemmParams& p, const GemmShared& s, int row0, int col0, int k0,
                         int k1) {
  const uint32_t p_bytes = static_cast<uint32_t>(p.bn) * kGemmK * 2;
  const uint32_t stage = kQBytes + p_bytes;
  uint32_t slot = 0, phase = 0, last_phase = 0, issued = 0;
  for (int kt = k0; kt < k1; ++kt) {
    if (!wait(s, bar(s, EMPTY0 + slot), phase ^ 1u, kStatusTimeoutProducer)) {
      // copies in flight land whatever the consumer does: wait (bounded)
      for (int i = 0; i < p.stages; ++i) {
        if (!(issued >> i & 1u)) continue;
        const long long t0 = clock64();
        while (!mbar_try_wait(bar(s, FULL0 + i), last_phase >> i & 1u))
          if (clock64() - t0 > kGemmWaitLimit) break;
      }
      return;
    }
    const uint32_t q = s.stages + slot * stage, pp = q + kQBytes, full = bar(s, FULL0 + slot);
    mbar_arrive_expect_tx(full, stage);
    const int k = kt * kGemmK;
    if (!p.q_mn) {
      tma_load_2d(q, &p.tm_q, full, k, col0);
    } else {
      tma_load_2d(q, &p.tm_q, full, col0, k);
      tma_load_2d(q + 8192, &p.tm_q, full, col0 + 64, k);
    }
    if (!p.p_mn) {
      tma_load_2d(pp, &p.tm_p, full, k, row0);
    } else {
      for (int j = 0; j < p.bn / 64; ++j)
        tma_load_2d(pp + 8192u * j, &p.tm_p, full, row0 + 64 * j, k);
    }
    last_phase = (last_phase & ~(1u << slot)) | (phase << slot);
    issued |= 1u << slot;
    if (++slot == static_cast<uint32_t>(p.stages)) {
      slot = 0;
      phase ^= 1u;
    }
  }
}

__device__ void mma_issuer(const GemmParams& p, const GemmShared& s, int steps, uint32_t tbase,
                           bool bf16) {
  const uint32_t stage = kQBytes + static_cast<uint32_t>(p.bn) * kGemmK * 2;
  const uint32_t idesc = idesc_16_f32(kTileCols, p.bn, bf16, p.q_mn != 0, p.p_mn != 0);
  const uint32_t a_lbo = p.q_mn ? 8192u : 16u, b_lbo = p.p_mn ? 8192u : 16u;
  const uint64_t a_step = p.q_mn ? 128 : 2, b_step = p.p_mn ? 128 : 2;
  uint32_t slot = 0, phase = 0;
  for (int kt = 0; kt < steps; ++kt) {
    if (!wait(s, bar(s, FULL0 + slot), phase, kStatusTimeoutMma)) return;
    tc_fence_after();
    const uint32_t a = s.stages + slot * stage;
    const uint64_t ad = sdesc_sw128(a, a_lbo, 1024), bd = sdesc_sw128(a + kQBytes, b_lbo, 1024);
#pragma unroll
    for (int kk = 0; kk < kGemmK / 16; ++kk)
      mma_ss(tbase, ad + kk * a_step, bd + kk * b_step, idesc, (kt | kk) != 0 ? 1u : 0u);
    tc_commit(bar(s, EMPTY0 + slot));
    if (++slot == static_cast<uint32_t>(p.stages)) {
      slot = 0;
      phase ^= 1u;
    }
  }
  tc_commit(bar(s, ACCFULL));
}

// Four consecutive columns of a row, from or to global memory: one access
// where the row allows it and all four are inside, else one by one.
template <typename E>
__device__ __forceinline__ void load4(const void* base, int64_t ld, int64_t row, int col, int C,
                                      bool vec, float (&v)[4]) {
  const E* p = static_cast<const E*>(base) + row * ld + col;
  if (vec && col + 4 <= C) {
    if constexpr (sizeof(E) == 4) {
      const float4 q = *reinterpret_cast<const float4*>(p);
      v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
    } else {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      const float2 lo = unpack_pair(q.x, E()), hi = unpack_pair(q.y, E());
      v[0] = lo.x, v[1] = lo.y, v[2] = hi.x, v[3] = hi.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = col + i < C ? to_f32(p[i]) : 0.f;
  }
}
template <typename E>
__device__ __forceinline__ void store4(void* base, int64_t ld, int64_t row, int col, int C, bool vec,
                                       const float (&v)[4]) {
  E* p = static_cast<E*>(base) + row * ld + col;
  if (vec && col + 4 <= C) {
    if constexpr (sizeof(E) == 4)
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    else
      *reinterpret_cast<uint2*>(p) =
          make_uint2(pack_pair(v[0], v[1], E()), pack_pair(v[2], v[3], E()));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (col + i < C) p[i] = from_f32<E>(v[i]);
  }
}

// Rows [j0, j1) of the tile from the partial tiles of `split` CTAs, summed in
// the order of their ranks.  A warp takes U of its rows at a time (every
// fourth row of the tile is its own), a lane four columns: the residuals, and
// the loads from Q CTAs, are in flight together.
template <typename T, typename O, int U, int Q>
__device__ void finish_rows(const GemmParams& p, uint32_t part, int split, int64_t row0, int j0,
                            int j1, int col, int warp) {
  const int lane = threadIdx.x & 31;
  float bias[4] = {0.f, 0.f, 0.f, 0.f};
  if (p.bias) load4<T>(p.bias, 0, 0, col, p.C, false, bias);
  const uint32_t mine = part + 16u * static_cast<uint32_t>(lane);
  for (int j = j0 + warp; j < j1; j += 4 * U) {
    float res[U][4], v[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (p.res && j + 4 * u < j1)
        load4<O>(p.res, p.ldr, row0 + j + 4 * u, col, p.C, p.res_vec != 0, res[u]);
#pragma unroll
    for (int u = 0; u < U; ++u) v[u][0] = v[u][1] = v[u][2] = v[u][3] = 0.f;
    for (int q = 0; q < split; q += Q) {
      float4 t[Q][U];
#pragma unroll
      for (int k = 0; k < Q; ++k) {
        const uint32_t from =
            map_to_rank(mine, static_cast<uint32_t>(q + k < split ? q + k : split - 1));
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const uint32_t a = static_cast<uint32_t>(min(j + 4 * u, j1 - 1)) * kTileCols * 4u;
          t[k][u] = ld_cluster_v4(from + a);
        }
      }
#pragma unroll
      for (int k = 0; k < Q; ++k)
        if (q + k < split)
#pragma unroll
          for (int u = 0; u < U; ++u) {
            v[u][0] += t[k][u].x;
            v[u][1] += t[k][u].y;
            v[u][2] += t[k][u].z;
            v[u][3] += t[k][u].w;
          }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (j + 4 * u >= j1) break;
      const int64_t row = row0 + j + 4 * u;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[u][i] += bias[i];
      if (p.pre) store4<T>(p.pre, p.ldp, row, col, p.C, p.pre_vec != 0, v[u]);
      if (p.act != WSATTN_ACT_NONE) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] = act_any(p.act, v[u][i]);
      }
      if (p.res) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[u][i] += res[u][i];
      }
      store4<O>(p.out, p.ldo, row, col, p.C, p.out_vec != 0, v[u]);
    }
  }
}

template <typename T, typename O>
__global__ void __launch_bounds__(kThreads) gemm_tile_kernel(const __grid_constant__ GemmParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const uint32_t stage = kQBytes + static_cast<uint32_t>(p.bn) * kGemmK * 2;
  GemmShared s;
  s.stages = base;
  s.bars = base + static_cast<uint32_t>(p.stages) * stage;
  uint8_t* gb = smem_raw + (s.bars - raw);
  uint32_t* tslot = reinterpret_cast<uint32_t*>(gb + 8 * NBARS);
  s.abort_flag = reinterpret_cast<volatile int*>(tslot + 1);
  s.status = p.status;
  const int warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  const uint32_t tcols = p.bn < 32 ? 32u : static_cast<uint32_t>(p.bn);

  // cluster c: tile c, rows the fast index (the weights of a column tile are
  // then in L2 for its other row tiles)
  const int split = p.split;
  const int rank = static_cast<int>(blockIdx.x) % split;
  const int tile = static_cast<int>(blockIdx.x) / split;
  const int tr = tile % p.tiles_r, tc = tile / p.tiles_r;
  const int row0 = tr * p.bn, col0 = tc * kTileCols;
  const int ksteps = (p.K + kGemmK - 1) / kGemmK;
  const int k0 = static_cast<int>(static_cast<int64_t>(ksteps) * rank / split);
  const int k1 = static_cast<int>(static_cast<int64_t>(ksteps) * (rank + 1) / split);
  const bool tile_ok =
      WSATTN_BOUNDS(p.status, tc < p.tiles_c && row0 < p.R && col0 < p.C && k1 > k0 &&
                                  k1 <= ksteps && p.stages >= 1 && p.stages <= kMaxStages &&
                                  (split == 1 || static_cast<uint32_t>(p.bn) * kTileCols * 4u <=
                                                     static_cast<uint32_t>(p.stages) * stage));

  if (threadIdx.x == 0) {
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(bar(s, FULL0 + i), 1);
      mbar_init(bar(s, EMPTY0 + i), 1);
    }
    mbar_init(bar(s, ACCFULL), 1);
    *s.abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&p.tm_p);
    prefetch_tensormap(&p.tm_q);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tslot), tcols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = *tslot;
  griddep_wait();
  // the next kernel's set-up may overlap this one (it waits for its results)
  griddep_launch_dependents();

  const int rows = static_cast<int>(min(static_cast<int64_t>(p.bn), p.R - row0));
  if (warp == 0) {
    if (lane == 0 && tile_ok) producer(p, s, row0, col0, k0, k1);
  } else if (warp == 1) {
    if (lane == 0 && tile_ok) mma_issuer(p, s, k1 - k0, tbase, !IsHalf<T>::value);
  } else {
    side_sums(p, static_cast<int>(blockIdx.x) * 128 + static_cast<int>(threadIdx.x) - 64,
              static_cast<int>(gridDim.x) * 128);
    __syncwarp();
    bool have = tile_ok && wait(s, bar(s, ACCFULL), 0, kStatusTimeoutSoftmax, p.K);
    have = __all_sync(0xffffffffu, have);
    tc_fence_after();
    if (have) {
      // the operand ring is idle now (every MMA of this CTA is complete): it
      // takes the tile, [row][128 columns] in fp32
      const int quad = warp & 3;
      const uint32_t tlane = tbase + (static_cast<uint32_t>(32 * quad) << 16);
      float* part = reinterpret_cast<float*>(smem_raw + (base - raw)) + 32 * quad + lane;
#pragma unroll 1
      for (int j = 0; j < rows; j += 16) {
        uint32_t a[16];
        tmem_ld16(tlane + j, a);
        tmem_wait_ld16(a);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (j + i < rows) part[(j + i) * kTileCols] = __uint_as_float(a[i]);
      }
    }
  }
  __syncwarp();
  if (split > 1) cluster_sync();  // every CTA's partial tile is in its shared memory
  else __syncthreads();
  if (warp >= 2 && tile_ok && *s.abort_flag == 0) {
    const int j0 = rows * rank / split, j1 = rows * (rank + 1) / split, col = col0 + 4 * lane;
    if (j1 - j0 <= 4)  // a row a warp: everything it needs at once
      finish_rows<T, O, 1, 8>(p, base, split, row0, j0, j1, col, warp - 2);
    else
      finish_rows<T, O, 4, 2>(p, base, split, row0, j0, j1, col, warp - 2);
  }
  if (split > 1) {
    __syncwarp();
    cluster_sync();  // no CTA leaves while others read its shared memory
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tbase, tcols);
}

template <typename T, typename O>
cudaError_t launch(const GemmParams& p, cudaStream_t s) {
  static bool attr_set[kMaxDevices] = {};
  const int dev = current_device();
  if (dev < 0) return cudaErrorInvalidDevice;
  if (!attr_set[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(gemm_tile_kernel<T, O>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(tile_smem_bytes(16, kMaxStages)));
    if (e != cudaSuccess) return e;
    attr_set[dev] = true;
  }
  const int64_t grid = static_cast<int64_t>(p.tiles_r) * p.tiles_c * p.split;
  if (grid > INT32_MAX || p.stages > kMaxStages) return cudaErrorInvalidValue;
  return launch_cluster(gemm_tile_kernel<T, O>, dim3(static_cast<unsigned>(grid)), dim3(kThreads),
                        p.split, tile_smem_bytes(p.bn, p.stages), s, p);
}

}  // namespace

size_t tile_smem_bytes(int bn, int stages) {
  return 1024 + static_cast<size_t>(stages) * (kQBytes + static_cast<size_t>(bn) * kGemmK * 2) +
         8 * NBARS + 16;
}

cudaError_t launch_gemm_tile(const GemmParams& p, int dtype, bool out_f32, cudaStream_t s) {
  if (dtype == WSATTN_BF16)
    return out_f32 ? launch<__nv_bfloat16, float>(p, s) : launch<__nv_bfloat16, __nv_bfloat16>(p, s);
  return out_f32 ? launch<__half, float>(p, s) : launch<__half, __half>(p, s);
}

}  // namespace wsattn
