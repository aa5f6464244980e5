// mok_ffn_tile.cu -- the feed-forward block's contractions, one output tile per CTA.
//
// A CTA computes a 128 x BN tile, or (split) one of S CTAs of a cluster computes a share of its K
// range.  Warp 0 issues TMA loads into a ring of stages, warp 1 issues the tcgen05.mma (M = 128, N = BN,
// K = 16) into one TMEM accumulator.  Then warps 2 to 5 push the accumulator, 8 columns of a row at a
// time, into the shared memory of the CTA of the cluster that owns them (dealt out round robin), and every owner
// adds its sources in ascending order, applies the epilogue and writes 16-byte
// vectors.  Every output has a fixed order of summation.
//
// With few tokens the weights' bytes bound it, and what stands in the way is latency: so the loops of
// warps 0 and 1 are warp-uniform with one elected lane at each asynchronous instruction (issued from a
// single-lane branch, a K block took 240 ns to issue whatever its size), the first loads are issued
// before the CTA's set-up has finished, and the contractions that follow another of this block
// load their weights before they wait for it.  Measured (both forward contractions, weights from HBM): 16 tokens at
// H = 4096, I = 1536 14.0 us; 61 tokens at H = 7168, I = 2048 23.9, 25.0 with a residual (13.0 of weights: gate/up streams at 7.1 TB/s; the rest
// is first bytes, reductions and the launch between, when HBM idles).
#include "mok_ffn.cuh"

namespace mok {
namespace {

constexpr int kTileThreads = 192;
constexpr int kTileMaxStages = 16;
constexpr uint32_t kTileMaxSmem = 230400;  // what a launch may ask for
// Tokens up to which the partials are counted on the owners' mbarriers, each CTA waiting for its own only; above, a
// store that is counted costs more than the cluster barrier that orders plain ones: 16 tokens at H = 4096, I = 1536
// 14.0 and 14.5 us, 48 tokens 14.9 both, 64 tokens 16.8 and 16.0, 128 tokens 21.6 and 19.4; at H = 7168, I = 2048 48 tokens
// 22.0 and 22.5, 61 tokens 22.9 and 23.5, 128 tokens 31.6 and 28.9.  (Staged first and copied in bulk: 14.7 and 23.3 for 16
// and 128 tokens at the first, when counted ones took 14.4 and plain ones 22.5.)
constexpr int64_t kTileCounted = 48;
constexpr uint32_t kTileSmem = 116224;  // two CTAs per SM

struct TileArgs {
  FfnArgs f;
  int32_t split;    // CTAs per tile (the cluster's size)
  int32_t stages;
  int32_t a_rows;   // rows of one A box: 128, or all of M rounded up to 8
  int32_t early_b;  // the previous kernel of the stream is one of this block's: weights may be read before it ends
  uint32_t b_off;   // shared memory: A stages, then B stages, then (split) the pushed partials
  uint32_t push_off;
  uint32_t src_bytes;  // pushed bytes per source CTA
};

struct TileMaps {
  CUtensorMap a, a2, b, b2;
};

template <int VAR, int BN>
struct TileCfg {
  static constexpr uint32_t kBBytes = BN * 128;
  static constexpr int kCols = VAR == F_GATEUP ? BN / 2 : BN;  // output columns of a tile
  static constexpr int kChunks = kCols / 8;
  static constexpr uint32_t kChunkBytes = VAR == F_GATEUP ? 64 : 32;  // 8 fp32 columns (gate, then up)
  // chunk `slot` of a pushed or staged tile; 16 bytes between rows keep the lanes (rows) off each
  // other's banks
  static __host__ __device__ uint32_t slot_off(uint32_t slot) {
    return slot * kChunkBytes + slot / kChunks * 16u;
  }
};

__device__ __forceinline__ float4 ld_shared_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster_v4(uint32_t addr, const uint32_t* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]),
               "r"(v[3])
               : "memory");
}
// The same, counted on a barrier of that CTA when the bytes are there.
__device__ __forceinline__ void st_async_v4(uint32_t addr, const uint32_t* v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(
                   addr),
               "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void store_bf16x8(void* p, int64_t i, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
// 8 columns of a saved factor: two blocks of 4 columns, 128 elements apart.
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
    if (f.kg) {
      float kg[8], ku[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = act_saved(v[k], w[k], f.act, kg[k], ku[k]);
      saved_store8(f.kg, ffn_saved_offset(m, c, f.N), kg);
      saved_store8(f.ku, ffn_saved_offset(m, c, f.N), ku);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = act_fwd(v[k], f.act) * w[k];
    }
    store_bf16x8(f.out0, i, v);
  } else if constexpr (VAR == F_DOWN || VAR == F_DX) {
    if (f.residual) {
      const uint4 q = *reinterpret_cast<const uint4*>(f.residual + i);
      v[0] += bf16_lo(q.x), v[1] += bf16_hi(q.x), v[2] += bf16_lo(q.y), v[3] += bf16_hi(q.y);
      v[4] += bf16_lo(q.z), v[5] += bf16_hi(q.z), v[6] += bf16_lo(q.w), v[7] += bf16_hi(q.w);
    }
    store_bf16x8(f.out0, i, v);
  } else if constexpr (VAR == F_DACT) {
    float g[8], u[8];
    saved_load8(f.kg, ffn_saved_offset(m, c, f.N), g);
    saved_load8(f.ku, ffn_saved_offset(m, c, f.N), u);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      g[k] *= v[k];
      u[k] *= v[k];
    }
    store_bf16x8(f.out0, i, g);
    store_bf16x8(f.out1, i, u);
  }
}

// COUNTED (split): the pushed partials are counted on mbarriers; else a cluster barrier orders them.
template <int VAR, int BN, bool COUNTED>
__global__ void __launch_bounds__(kTileThreads)
    ffn_tile_kernel(const __grid_constant__ CUtensorMap tA, const __grid_constant__ CUtensorMap tA2,
                    const __grid_constant__ CUtensorMap tB, const __grid_constant__ CUtensorMap tB2,
                    const TileArgs t) {
  using C = TileCfg<VAR, BN>;
  constexpr uint32_t kIdesc = idesc_bf16(128, BN, false, ffn_b_mn(VAR));
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kTileMaxStages + 2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;  // swizzle atoms: 1024-byte aligned
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kTileMaxStages + s); };
  const uint32_t done = bar0 + 8u * (2 * kTileMaxStages), pushed = done + 8u;
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = t.split, rank = static_cast<int>(blockIdx.x) % S, tile = static_cast<int>(blockIdx.x) / S;
  const int n = tile / t.f.m_tiles, m = tile - n * t.f.m_tiles;
  const int kb0 = static_cast<int>(static_cast<int64_t>(t.f.k_blocks) * rank / S);
  const int count = static_cast<int>(static_cast<int64_t>(t.f.k_blocks) * (rank + 1) / S) - kb0;
  const uint32_t a_bytes = static_cast<uint32_t>(t.a_rows) * 128u;
  const int rows = min(128, t.f.M - m * 128), items = rows * C::kChunks;  // chunks of the tile's valid rows
  if (warp == 0) {
    if (elect_one()) {
      for (int s = 0; s < t.stages; ++s) {
        mbar_init(full(s), 1);
        mbar_init(empty(s), 1);
      }
      mbar_init(done, 1);
      mbar_init(pushed, 1);
      abort_word = 0;
      fence_barrier_init();
      const int mine = items > rank ? (items - rank + S - 1) / S : 0;  // this CTA's chunks, once from every source
      mbar_arrive_expect_tx(pushed, COUNTED ? static_cast<uint32_t>(S * mine) * C::kChunkBytes : 0u);
    }
    __syncwarp();
  } else if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), BN < 32 ? 32 : BN);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const uint32_t tmem = tmem_slot;

  if (warp == 0 || warp == 2) {  // weights and, by another warp, tokens: a load takes about 35 ns to issue
    const bool b_side = warp == 0;
    if (!b_side || !t.early_b) pdl_wait();
    if (!b_side) pdl_trigger();
    bool ok = true;
    int st = 0, i = 0;
    uint32_t ph = 1;  // parity of the empty barrier's phase to wait for: none in the first round
    for (; i < count; ++i) {
      if (i == t.stages) pdl_wait();  // (weights: the stages filled early; see warp 1)
      if (i >= t.stages && !warp_wait(empty(st), ph, abort_flag, t.f.status)) {
        ok = false;
        break;
      }
      if (elect_one()) {
        if (b_side) {
          mbar_arrive_expect_tx(full(st), a_bytes + C::kBBytes);
          tile_load_b<VAR, BN>(t, n, kb0 + i, base + t.b_off + st * C::kBBytes, full(st), &tB, &tB2);
        } else {
          tile_load_a<VAR, BN>(t, m, kb0 + i, base + st * a_bytes, full(st), &tA, &tA2);
        }
      }
      if (++st == t.stages) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (!ok && lane == 0) {  // let the copies in flight land: the last one of each stage
      for (int b = i > t.stages ? i - t.stages : 0; b < i; ++b)
        wait_landed(full(b % t.stages), static_cast<uint32_t>(b / t.stages) & 1u);
    }
    __syncwarp();
  } else if (warp == 1) {
    pdl_wait();  // the kernel in front may take its time: no bounded wait starts before its end
    int st = 0;
    uint32_t ph = 0;
    for (int i = 0; i < count; ++i) {
      if (!warp_wait(full(st), ph, abort_flag, t.f.status)) break;
      tc_fence_after();
      const uint32_t sa = base + st * a_bytes, sb = base + t.b_off + st * C::kBBytes;
      const uint64_t ad = sdesc_sw128(sa, 16, 1024);
      const uint64_t bd = ffn_b_mn(VAR) ? sdesc_sw128(sb, 8192, 1024) : sdesc_sw128(sb, 16, 1024);
      if (elect_one()) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)  // descriptors count 16-byte units
          umma_bf16(tmem, ad + ks * 2, bd + ks * (ffn_b_mn(VAR) ? 128 : 2), kIdesc, (i > 0 || ks > 0) ? 1u : 0u);
        umma_commit(empty(st));
      }
      if (++st == t.stages) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (elect_one()) umma_commit(done);  // also after an abort: what was issued completes before TMEM is freed
    __syncwarp();
  }
  pdl_wait();  // before anything is read or written below (at once for the warps that have passed it)
  bool ok = warp_wait(done, 0, abort_flag, t.f.status);
  if (!ok && warp == 1) wait_landed(done, 0);
  if (S > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // every peer has started
  tc_fence_after();
  // the accumulator's chunks to their owners: chunk j (row-major over the tile's valid rows) is slot j / S
  // of CTA j % S.  Without a split they are staged over the stages, every copy into which has been consumed.
  const uint32_t push = S > 1 ? base + t.push_off : base;
  if (warp >= 2) {
    const int q = warp & 3, r = q * 32 + lane;  // this warp's TMEM lane quarter; the lane's row
    if (q * 32 < rows) {
      const uint32_t src = push + static_cast<uint32_t>(rank) * t.src_bytes;
      const uint32_t j0 = static_cast<uint32_t>(r * C::kChunks);
      const uint32_t slot0 = j0 / static_cast<uint32_t>(S), own0 = j0 - slot0 * static_cast<uint32_t>(S);
      auto put = [&](const uint32_t* v, uint32_t chunk, uint32_t sub) {
        if (r >= rows) return;
        if (S == 1) {
          const uint32_t d = src + C::slot_off(j0 + chunk) + sub;
          st_shared_v4(d, make_uint4(v[0], v[1], v[2], v[3]));
          st_shared_v4(d + 16, make_uint4(v[4], v[5], v[6], v[7]));
        } else {
          uint32_t slot = slot0, own = own0 + chunk;
          while (own >= static_cast<uint32_t>(S)) own -= S, ++slot;
          const uint32_t d = mapa_shared(src + C::slot_off(slot) + sub, own);
          if constexpr (COUNTED) {
            const uint32_t bar = mapa_shared(pushed, own);
            st_async_v4(d, v, bar);
            st_async_v4(d + 16, v + 4, bar);
          } else {
            st_cluster_v4(d, v);
            st_cluster_v4(d + 16, v + 4);
          }
        }
      };
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        uint32_t v[32];
        tmem_ld_32x32b_x32(tmem + (static_cast<uint32_t>(q * 32) << 16) + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = c + 8 * j;
          if (VAR == F_GATEUP && col >= C::kCols) put(v + 8 * j, (col - C::kCols) / 8, 32);
          else put(v + 8 * j, col / 8, 0);
        }
      }
    }
  }
  tc_fence_before();
  if (S > 1 && !COUNTED) cluster_sync();  // release / acquire: the pushed chunks are there
  else __syncthreads();
  if constexpr (COUNTED) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA has pushed
  if (warp == 1) tmem_dealloc(tmem, BN < 32 ? 32 : BN);
  if constexpr (COUNTED) __all_sync(0xffffffffu, mbar_wait<true>(pushed, 0, abort_flag, t.f.status));
  const bool whole = *abort_flag == 0;  // (else recorded in the status word)
  const int64_t m0 = static_cast<int64_t>(m) * 128;
  const int c0 = n * C::kCols;
  for (int slot = threadIdx.x; whole && slot * S + rank < items; slot += kTileThreads) {
    const int j = slot * S + rank, r = j / C::kChunks, c = (j - r * C::kChunks) * 8;
    if (c0 + c >= t.f.N) continue;
    float v[8], w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = w[k] = 0.0f;
    uint32_t d = push + C::slot_off(static_cast<uint32_t>(slot));
    for (int p = 0; p < S; ++p, d += t.src_bytes) {
      const float4 x = ld_shared_f4(d), y = ld_shared_f4(d + 16);
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w, v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
      if constexpr (VAR == F_GATEUP) {
        const float4 z = ld_shared_f4(d + 32), q = ld_shared_f4(d + 48);
        w[0] += z.x, w[1] += z.y, w[2] += z.z, w[3] += z.w, w[4] += q.x, w[5] += q.y, w[6] += q.z, w[7] += q.w;
      }
    }
    tile_epilogue8<VAR>(t.f, m0 + r, c0 + c, v, w);
  }
  if constexpr (COUNTED) {
    if (!whole) {  // failure path: a peer's chunks may still be under way
      const uint64_t t0 = global_timer_ns();
      while (global_timer_ns() - t0 < kWaitLimitNs / 100) {
      }
    }
    __syncwarp();
    asm volatile("barrier.cluster.wait.aligned;" ::: "memory");  // no CTA leaves before every peer has pushed
  }
}

// Whether every CTA gets an SM of its own, with most of its shared memory: where they all fit in one go (clusters of 4
// and 8 leave SMs of a GPC without one: 36 and 15 of them fit).  Two per SM would be packed onto the SMs that the
// kernel in front leaves free: this one is launched while that one runs.  T = 128, H = 4096, I = 1536 22.5 -> 20.3 us
// forward, 58.8 -> 55.3 training; T = 100, H = 3000, I = 1000 16.0 -> 14.9 and 45.7 -> 42.3.
bool tiles_alone(int64_t tiles, int split) {
  const int sms = sm_count();
  return tiles <= (split == 1 ? sms : split == 2 ? sms / 2 : split == 4 ? sms / 4 - 2 : sms / 8 - 4);
}

template <int VAR, int BN, bool COUNTED>
int launch_tile(const TileMaps& maps, TileArgs t, cudaStream_t stream) {
  using C = TileCfg<VAR, BN>;
  static DeviceOnce once;
  const int se = once.run([](int* d) { return static_cast<int>(cudaGetDevice(d)); },
                          [] {
                            return static_cast<int>(cudaFuncSetAttribute(ffn_tile_kernel<VAR, BN, COUNTED>,
                                                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                         static_cast<int>(kTileMaxSmem)));
                          },
                          static_cast<int>(cudaErrorInvalidDevice));
  if (se) return se;
  const uint32_t a_bytes = static_cast<uint32_t>(t.a_rows) * 128u;
  const uint32_t stage = a_bytes + C::kBBytes;
  const uint32_t rows = static_cast<uint32_t>(t.f.M < 128 ? t.f.M : 128);
  const uint32_t slots = (rows * C::kChunks + t.split - 1) / t.split;
  t.src_bytes = (C::slot_off(slots) + 31u) & ~15u;
  const uint32_t push = t.split > 1 ? t.src_bytes * t.split : 0u;
  const bool alone = tiles_alone(static_cast<int64_t>(t.f.m_tiles) * t.f.n_tiles, t.split);
  const uint32_t budget = (alone ? kTileMaxSmem - 1024u : kTileSmem) - 3072u - push;  // alignment slack, static and reserved shared memory
  int stages = static_cast<int>(budget / stage);
  if (stages < 2) stages = 2;
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
  t.push_off = smem;
  smem += push;
  if (t.split == 1 && smem < t.src_bytes) smem = t.src_bytes;
  smem += 1024;
  if (alone && smem <= kTileSmem) smem = kTileSmem + 1024u;
  if (smem > kTileMaxSmem) return static_cast<int>(cudaErrorInvalidValue);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, ffn_tile_kernel<VAR, BN, COUNTED>, maps.a, maps.a2, maps.b, maps.b2, t);
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
  t.early_b = VAR == F_DOWN || VAR == F_DX;  // always behind GATEUP and DACT
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
  if constexpr (BN == 64) {
    if (split > 1 && M <= kTileCounted) return launch_tile<VAR, BN, true>(p, t, stream);
  }
  return launch_tile<VAR, BN, false>(p, t, stream);
}

// Columns of a tile and CTAs per tile.  64-column tiles, two CTAs resident per SM; with few tiles the K range is
// split over a cluster of 2, 4 or 8 while there are at most two CTAs per SM; from six rounds of tiles on, 128
// columns (H = 4096, I = 32768 forward: 16 tokens 123 us, 133 with 64 columns; 128 tokens 147 and 164; H = 60000, I =
// 4096, a training step of 128 tokens 973 and 1029).  What a split costs is its partials, so with the rows: up to 24 tokens each CTA keeps two K blocks or more, up
// to 64 four, above eight, and above 32 tokens clusters of four at most.  Measured, both forward contractions: H =
// I = 640, 16 tokens 7.0 us with two K blocks at least, 8.0 with four; H = I = 1000, 32 tokens 9.0 and 8.5; H = 4096,
// I = 1536, 61 tokens 16.3 with four at least, 17.1 with eight; H = 1000, I = 2000, 5 tokens 9.7 with clusters of
// eight allowed, 10.5 without; 128 tokens 19.8 and 18.1, and 13.6 with eight K blocks at least.
// (Clusters of 3, 5 or 6 leave SMs of a GPC without one.)
template <int VAR>
int launch_tiles(int64_t M, int64_t N, int64_t K, const FfnOperands& o, const FfnArgs& f, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return static_cast<int>(cudaErrorInvalidDevice);
  auto tiles = [&](int bn) { return (M + 127) / 128 * ((N + bn - 1) / bn); };
  constexpr int kPer = VAR == F_GATEUP ? 2 : 1;  // tile columns per output column
  if (tiles(64 / kPer) > 6 * sms) return launch_var<VAR, 128>(M, N, K, 1, o, f, stream);
  const int64_t kb = (K + kFfnBK - 1) / kFfnBK * (VAR == F_DX ? 2 : 1);
  int64_t split = 2 * sms / tiles(64 / kPer);
  const int64_t least = M > 64 ? 8 : M > 24 ? 4 : 2;  // K blocks per CTA
  if (split > kb / least) split = kb / least;
  split = split >= 8 && M <= 32 ? 8 : split >= 4 ? 4 : split >= 2 ? 2 : 1;
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
