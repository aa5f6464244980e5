// mok_ffn_tile.cu -- the feed-forward block's contractions, one output tile per CTA.
//
// A CTA computes a 128 x BN tile, or (split) one of S CTAs of a cluster computes a share of its K
// range; the S partial tiles meet in shared memory.  Warp 0 issues TMA loads into a ring of
// stages, warp 1 issues the tcgen05.mma (M = 128, N = BN, K = 16) into one TMEM accumulator; warps 2 to 5
// copy it to shared memory as fp32, and then all threads take 8 columns of a row at a time: they sum the
// cluster's partials in ascending order through distributed shared memory, apply the epilogue and write
// 16-byte vectors.  Every output has a fixed order of summation.
#include "mok_ffn.cuh"

namespace mok {
namespace {

constexpr int kTileThreads = 192;
constexpr int kTileMaxStages = 16;
constexpr uint32_t kTileMaxSmem = 232448;

struct TileArgs {
  FfnArgs f;
  int32_t split;    // CTAs per tile (the cluster's size)
  int32_t stages;
  int32_t a_rows;   // rows of one A box (K-major A): 128, or all of M rounded up to 8
  uint32_t b_off;   // shared memory: A stages, then B stages
};

struct TileMaps {
  CUtensorMap a, a2, b, b2;
};

template <int VAR, int BN>
struct TileCfg {
  static constexpr uint32_t kBBytes = BN * 128;
  static constexpr uint32_t kStride = BN + 4;  // fp32 per row of the staged tile
  static constexpr uint32_t kStaged = 128u * kStride * 4u;
};

// Bounded wait that ignores the abort flag: only while winding down.
__device__ __forceinline__ void wait_landed(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < kWaitLimitNs / 4) {
  }
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void store_bf16x8(void* p, int64_t i, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
// 8 columns of a saved g or u: two blocks of 4 columns, 128 elements apart.
__device__ __forceinline__ void saved_store8(float* p, int64_t off, const float (&v)[8]) {
  *reinterpret_cast<float4*>(p + off) = make_float4(v[0], v[1], v[2], v[3]);
  *reinterpret_cast<float4*>(p + off + 128) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void saved_load8(const float* p, int64_t off, float (&v)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p + off), b = *reinterpret_cast<const float4*>(p + off + 128);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

template <int VAR, int BN>
__device__ __forceinline__ void tile_load_a(const TileArgs& t, int m, int kb, uint32_t sa, uint32_t bar,
                                            const CUtensorMap* tA, const CUtensorMap* tA2) {
  const int k0 = kb * kFfnBK;
  if constexpr (VAR == F_DX) {
    const bool first = kb < t.f.kb_split;
    tma_load_2d(sa, first ? tA : tA2, bar, first ? k0 : k0 - t.f.kb_split * kFfnBK, m * 128);
  } else {
    tma_load_2d(sa, tA, bar, k0, m * 128);
  }
}
template <int VAR, int BN>
__device__ __forceinline__ void tile_load_b(const TileArgs& t, int n, int kb, uint32_t sb, uint32_t bar,
                                            const CUtensorMap* tB, const CUtensorMap* tB2) {
  const int k0 = kb * kFfnBK;
  if constexpr (VAR == F_GATEUP) {
    tma_load_2d(sb, tB, bar, k0, n * (BN / 2));
    tma_load_2d(sb + BN / 2 * 128, tB2, bar, k0, n * (BN / 2));
  } else if constexpr (!ffn_b_mn(VAR)) {
    tma_load_2d(sb, tB, bar, k0, n * BN);
  } else {
    const bool first = VAR != F_DX || kb < t.f.kb_split;
    const int kr = first ? k0 : k0 - t.f.kb_split * kFfnBK;
#pragma unroll
    for (int j = 0; j < BN / 64; ++j) tma_load_2d(sb + j * 8192, first ? tB : tB2, bar, n * BN + j * 64, kr);
  }
}

// Epilogue of 8 columns (GATEUP: v = 8 gate and w the same 8 up columns) at row m, column c of the output.
template <int VAR>
__device__ __forceinline__ void tile_epilogue8(const FfnArgs& f, int64_t m, int c, float (&v)[8], float (&w)[8]) {
  const int64_t i = m * f.N + c;
  if constexpr (VAR == F_GATEUP) {
    if (f.g) {
      saved_store8(f.g, ffn_saved_offset(m, c, f.N), v);
      saved_store8(f.u, ffn_saved_offset(m, c, f.N), w);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = act_fwd(v[k], f.act) * w[k];
    store_bf16x8(f.out0, i, v);
  } else if constexpr (VAR == F_DOWN) {
    if (f.residual) {
      const uint4 q = *reinterpret_cast<const uint4*>(f.residual + i);
      v[0] += bf16_lo(q.x), v[1] += bf16_hi(q.x), v[2] += bf16_lo(q.y), v[3] += bf16_hi(q.y);
      v[4] += bf16_lo(q.z), v[5] += bf16_hi(q.z), v[6] += bf16_lo(q.w), v[7] += bf16_hi(q.w);
    }
    store_bf16x8(f.out0, i, v);
  } else if constexpr (VAR == F_DACT) {
    float g[8], u[8];
    saved_load8(f.g, ffn_saved_offset(m, c, f.N), g);
    saved_load8(f.u, ffn_saved_offset(m, c, f.N), u);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      float a, da;
      act_bwd(g[k], f.act, a, da);
      g[k] = v[k] * u[k] * da;
      u[k] = v[k] * a;
    }
    store_bf16x8(f.out0, i, g);
    store_bf16x8(f.out1, i, u);
  } else {
    store_bf16x8(f.out0, i, v);
  }
}

template <int VAR, int BN>
__global__ void __launch_bounds__(kTileThreads)
    ffn_tile_kernel(const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tA2,
                    const __grid_constant__ CUtensorMap tB, const __grid_constant__ CUtensorMap tB2,
                    const TileArgs t) {
  using C = TileCfg<VAR, BN>;
  constexpr uint32_t kIdesc = idesc_bf16(128, BN, false, ffn_b_mn(VAR));
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kTileMaxStages + 1];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;  // swizzle atoms: 1024-byte aligned
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kTileMaxStages + s); };
  const uint32_t done = bar0 + 8u * (2 * kTileMaxStages);
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = t.split, rank = static_cast<int>(blockIdx.x) % S, tile = static_cast<int>(blockIdx.x) / S;
  const int n = tile / t.f.m_tiles, m = tile - n * t.f.m_tiles;
  const int kb0 = static_cast<int>(static_cast<int64_t>(t.f.k_blocks) * rank / S);
  const int kb1 = static_cast<int>(static_cast<int64_t>(t.f.k_blocks) * (rank + 1) / S);
  const uint32_t a_bytes = static_cast<uint32_t>(t.a_rows) * 128u;
  if (threadIdx.x == 0) {
    for (int s = 0; s < t.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    mbar_init(done, 1);
    abort_word = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tA);
    tma_prefetch_desc(&tB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_wait();
  const uint32_t tmem = tmem_slot;

  if (warp == 0) {
    if (lane == 0) {
      bool ok = true;
      int st = 0, issued = 0;
      uint32_t ph = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(empty(st), ph ^ 1u, abort_flag, t.f.status)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(full(st), a_bytes + C::kBBytes);
        tile_load_a<VAR, BN>(t, m, kb, base + st * a_bytes, full(st), &tA, &tA2);
        tile_load_b<VAR, BN>(t, n, kb, base + t.b_off + st * C::kBBytes, full(st), &tB, &tB2);
        ++issued;
        if (++st == t.stages) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (!ok) {  // let the copies in flight land: the last one of each stage
        for (int b = issued > t.stages ? issued - t.stages : 0; b < issued; ++b)
          wait_landed(full(b % t.stages), static_cast<uint32_t>(b / t.stages) & 1u);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (lane == 0) {
      int st = 0;
      uint32_t ph = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!mbar_wait(full(st), ph, abort_flag, t.f.status)) break;
        tc_fence_after();
        const uint32_t sa = base + st * a_bytes, sb = base + t.b_off + st * C::kBBytes;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint64_t ad = sdesc_sw128(sa + ks * 32, 16, 1024);
          const uint64_t bd = ffn_b_mn(VAR) ? sdesc_sw128(sb + ks * 2048, 8192, 1024) : sdesc_sw128(sb + ks * 32, 16, 1024);
          umma_bf16(tmem, ad, bd, kIdesc, (kb > kb0 || ks > 0) ? 1u : 0u);
        }
        umma_commit(empty(st));
        if (++st == t.stages) {
          st = 0;
          ph ^= 1u;
        }
      }
      umma_commit(done);  // also after an abort: what was issued completes before TMEM is freed
    }
    __syncwarp();
  }
  // the accumulator to shared memory, over the stages: every copy into them has been consumed
  bool ok = true;
  {
    int w = 0;
    if (lane == 0) {
      w = mbar_wait(done, 0, abort_flag, t.f.status) ? 1 : 0;
      // after an abort the MMAs already issued still end before TMEM is freed
      if (!w && warp == 1) wait_landed(done, 0);
    }
    ok = __shfl_sync(0xffffffffu, w, 0) != 0;
  }
  __syncthreads();
  if (*abort_flag) ok = false;
  tc_fence_after();
  const int rows = min(128, t.f.M - m * 128);
  if (warp >= 2 && ok) {
    const int q = warp & 3;  // this warp's TMEM lane quarter
    if (q * 32 < rows) {
      const uint32_t row = base + static_cast<uint32_t>(q * 32 + lane) * (C::kStride * 4u);
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 8; ++j)
          st_shared_v4(row + 4u * c + 16u * j, make_uint4(r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]));
      }
    }
  }
  tc_fence_before();
  if (S > 1) cluster_sync();
  else __syncthreads();
  if (ok) {
    const int64_t m0 = static_cast<int64_t>(m) * 128;
    constexpr int kCols = VAR == F_GATEUP ? BN / 2 : BN;  // output columns of a tile
    constexpr int kChunks = kCols / 8;
    const int c0 = n * kCols;
    const int items = rows * kChunks;
    for (int it = rank * kTileThreads + threadIdx.x; it < items; it += S * kTileThreads) {
      const int r = it / kChunks, c = (it - r * kChunks) * 8;
      if (c0 + c >= t.f.N) continue;
      float v[8], w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = w[k] = 0.0f;
      const uint32_t off = base + static_cast<uint32_t>(r) * (C::kStride * 4u) + 4u * c;
      for (int p = 0; p < S; ++p) {
        const uint32_t src = S > 1 ? mapa_shared(off, p) : off;
        const float4 x = ld_cluster_f4(src), y = ld_cluster_f4(src + 16);
        v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
        if constexpr (VAR == F_GATEUP) {
          const float4 z = ld_cluster_f4(src + kCols * 4), q = ld_cluster_f4(src + kCols * 4 + 16);
          w[0] += z.x, w[1] += z.y, w[2] += z.z, w[3] += z.w, w[4] += q.x, w[5] += q.y, w[6] += q.z, w[7] += q.w;
        }
      }
      tile_epilogue8<VAR>(t.f, m0 + r, c0 + c, v, w);
    }
  }
  if (S > 1) cluster_sync();  // no CTA leaves while a peer may read its partials
  else __syncthreads();
  if (warp == 1) tmem_dealloc(tmem, BN);
}

template <int VAR, int BN>
int launch_tile(const TileMaps& maps, TileArgs t, cudaStream_t stream) {
  using C = TileCfg<VAR, BN>;
  static DeviceOnce once;
  const int se = once.run([](int* d) { return static_cast<int>(cudaGetDevice(d)); },
                          [] {
                            return static_cast<int>(cudaFuncSetAttribute(ffn_tile_kernel<VAR, BN>,
                                                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                         static_cast<int>(kTileMaxSmem - 1024)));
                          },
                          static_cast<int>(cudaErrorInvalidDevice));
  if (se) return se;
  const uint32_t a_bytes = static_cast<uint32_t>(t.a_rows) * 128u;
  const uint32_t stage = a_bytes + C::kBBytes;
  const uint32_t budget = kTileMaxSmem - 4096;  // static shared memory and the alignment slack
  int stages = static_cast<int>((budget - 16384u) / stage);
  if (stages > kTileMaxStages) stages = kTileMaxStages;
  const int per = (t.f.k_blocks + t.split - 1) / t.split;
  if (stages > per) stages = per;
  t.stages = stages;
  t.b_off = (static_cast<uint32_t>(stages) * a_bytes + 1023u) & ~1023u;
  // the MMA reads 128 rows of A whatever was loaded: what a short box leaves out is other shared memory
  // (its results are rows past M, never stored), inside the allocation
  uint32_t smem = t.b_off + static_cast<uint32_t>(stages) * C::kBBytes;
  const uint32_t a_reach = static_cast<uint32_t>(stages - 1) * a_bytes + 16384u;
  if (smem < a_reach) smem = a_reach;
  if (smem < C::kStaged) smem = C::kStaged;
  smem += 1024;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(t.f.m_tiles) * t.f.n_tiles * t.split);
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = t.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = t.split > 1 ? 2 : 1;
  constexpr int kKind = K_FFN_GATEUP + VAR;
  trace_begin(stream, kKind);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, ffn_tile_kernel<VAR, BN>, maps.a, maps.a2, maps.b, maps.b2, t);
  trace_end(stream);
  return static_cast<int>(e);
}

template <int VAR, int BN>
int launch_var(int64_t M, int64_t N, int64_t K, int split, const FfnOperands& o, FfnArgs f, cudaStream_t stream) {
  TileArgs t{};
  constexpr int kCols = VAR == F_GATEUP ? BN / 2 : BN;
  const int64_t mt = (M + 127) / 128, nt = (N + kCols - 1) / kCols;
  f.M = static_cast<int32_t>(M);
  f.N = static_cast<int32_t>(N);
  f.m_tiles = static_cast<int32_t>(mt);
  f.n_tiles = static_cast<int32_t>(nt);
  const int64_t kb = (K + kFfnBK - 1) / kFfnBK;
  f.kb_split = static_cast<int32_t>(kb);
  f.k_blocks = static_cast<int32_t>(VAR == F_DX ? 2 * kb : kb);
  if (static_cast<int64_t>(f.m_tiles) * nt >= (int64_t{1} << 27)) return static_cast<int>(cudaErrorInvalidValue);
  t.f = f;
  t.a_rows = M >= 128 ? 128 : static_cast<int32_t>((M + 7) / 8 * 8);
  t.split = split;
  const uint64_t um = static_cast<uint64_t>(M), un = static_cast<uint64_t>(N), uk = static_cast<uint64_t>(K);
  TileMaps p;
  bool good = make_tmap_bf16(&p.a, o.a, uk, um, 64, static_cast<uint32_t>(t.a_rows));
  p.a2 = p.a;
  if constexpr (VAR == F_DX) good = good && make_tmap_bf16(&p.a2, o.a2, uk, um, 64, static_cast<uint32_t>(t.a_rows));
  if constexpr (ffn_b_mn(VAR)) good = good && make_tmap_bf16(&p.b, o.b, un, uk, 64, 64);
  else good = good && make_tmap_bf16(&p.b, o.b, uk, un, 64, kCols);
  p.b2 = p.b;
  if constexpr (VAR == F_GATEUP) good = good && make_tmap_bf16(&p.b2, o.b2, uk, un, 64, kCols);
  if constexpr (VAR == F_DX) good = good && make_tmap_bf16(&p.b2, o.b2, un, uk, 64, 64);
  if (!good) return static_cast<int>(cudaErrorInvalidValue);
  return launch_tile<VAR, BN>(p, t, stream);
}

// Columns of a tile and CTAs per tile.  With few tiles the K range is split over a cluster until about
// every SM has a CTA, leaving each at least four K blocks; 64-column tiles first, since they need fewer
// CTAs per tile.
template <int VAR>
int launch_tiles(int64_t M, int64_t N, int64_t K, const FfnOperands& o, const FfnArgs& f, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return static_cast<int>(cudaErrorInvalidDevice);
  auto tiles = [&](int bn) { return (M + 127) / 128 * ((N + bn - 1) / bn); };
  constexpr int kPer = VAR == F_GATEUP ? 2 : 1;  // tile columns per output column
  if (2 * tiles(64 / kPer) > 3 * sms) return launch_var<VAR, 128>(M, N, K, 1, o, f, stream);
  const int64_t kb = (K + kFfnBK - 1) / kFfnBK * (VAR == F_DX ? 2 : 1);
  int64_t split = sms / tiles(64 / kPer);
  if (split > kb / 4) split = kb / 4;
  split = split < 1 ? 1 : split > 8 ? 8 : split;
  return launch_var<VAR, 64>(M, N, K, static_cast<int>(split), o, f, stream);
}

}  // namespace

int launch_ffn_tile(int var, int64_t M, int64_t N, int64_t K, const FfnOperands& o, const FfnArgs& a,
                    cudaStream_t stream) {
  switch (var) {
    case F_GATEUP: return launch_tiles<F_GATEUP>(M, N, K, o, a, stream);
    case F_DOWN: return launch_tiles<F_DOWN>(M, N, K, o, a, stream);
    case F_DACT: return launch_tiles<F_DACT>(M, N, K, o, a, stream);
    default: return launch_tiles<F_DX>(M, N, K, o, a, stream);
  }
}

}  // namespace mok
