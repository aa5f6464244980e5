// mok_ffn_pair.cu -- the feed-forward block's contractions for many tokens: persistent CTA pairs.
//
// A cluster of two CTAs computes 256 x BN tiles with tcgen05.mma.cta_group::2 (M = 256): each CTA loads its
// own 128 rows of A and half of B's columns, so a CTA takes in 32 KB per 64-wide K block of a 256 x 256
// tile and keeps six blocks in flight.  Two TMEM accumulators let one tile's epilogue run under the next
// tile's MMAs.  Per CTA: warp 0 issues TMA loads, warp 1 (of the first CTA) the MMAs, eight warps
// drain the accumulator, two per TMEM lane quarter with half of the columns each.
//
// Tiles are dealt out over one pair per two SMs, in an order that keeps the tiles running together in a
// near-square block of the output (ordered_tile), so that both operands are read from L2.
//
// The backward is two launches of two jobs each, so that one's tiles fill the pairs that the other's last round
// leaves idle: BWD1 = DACT, and dWd where that is shorter (it needs nothing of DACT's); BWD2 = DX and the other
// weight gradients.  One job's tiles go round robin; the other's are shared out behind them so that all pairs end
// as nearly together as whole tiles allow (make_plan).
//
// Bound by the tensor cores and, about as much, by the loads from L2; the power limit sets the pace of long runs.
// Measured: a training step of 8192 tokens at H = 4096, I = 1536 518 us, 1,790 TFLOP/s (1,930 for a plain library product
// in bursts), 603 us in a sustained loop; a forward of 4096 tokens at H = 2048, I = 1024 38.3 us, 1,350 TFLOP/s; a
// training step of 1003 tokens at H = 2056, I = 1000 61 us: its four launches cost 5 us each besides their tiles.
#include "mok_ffn.cuh"

namespace mok {
namespace {

constexpr int kPairThreads = 64 + 32 * 8;
constexpr uint32_t kPairTmemCols = 512;  // two accumulators, 256 columns apart
struct PairArgs {
  FfnArgs f;            // job 0
  PairPlan plan;
  // job 1: units [0, u1) are dWg, [u1, 2 u1) dWu (I x H), the rest dWd (H x I)
  int32_t H, I, u1;
  int32_t m_tiles_i, n_tiles_h, m_tiles_h, n_tiles_i;
  int32_t k_blocks1;
  // forward, MIX: from the M tile m_split on, tiles of bn1 columns
  int32_t bn1, m_split, n_tiles1;
};

struct PairMaps {
  CUtensorMap a[2], b[2], o[2];     // job 0
  CUtensorMap a1[3], b1[2], o1[3];  // job 1 (forward: b1)
};

enum PairVariant : int { P_GATEUP = 0, P_DOWN, P_BWD1, P_BWD2 };

template <int VAR, int BN>
struct PairCfg {
  static constexpr bool kBmn = VAR >= P_BWD1;
  static constexpr uint32_t kABytes = 128 * 128;
  // an MN-major B half is whole 64-column boxes (the columns past BN / 2 of the last one are not used)
  static constexpr uint32_t kBBoxes = (BN / 2 + 63) / 64;
  static constexpr uint32_t kBBytes = kBmn ? kBBoxes * 8192 : BN / 2 * 128;
  static constexpr uint32_t kStageBytes = kABytes + kBBytes;
  // both CTAs' loads of a tile of bn columns count on the first CTA's barrier
  static __device__ __forceinline__ uint32_t tx_bytes(int bn) {
    return kBmn ? 2 * kStageBytes : 2 * kABytes + static_cast<uint32_t>(bn) * 128u;
  }
  static constexpr uint32_t kStagingBytes = 8 * 2 * 2048;  // two 32-row x 64-byte tiles per epilogue warp
  static constexpr int kStages = static_cast<int>((232448u - 1024u - 512u - kStagingBytes) / kStageBytes);
  static constexpr uint32_t kStagingOff = kStages * kStageBytes;
  static constexpr uint32_t kBarOff = kStagingOff + kStagingBytes;
  static constexpr uint32_t kSmemBytes = 1024 + kBarOff + 256;
  static_assert(kSmemBytes <= 232448, "shared memory per CTA");
  static_assert(2 * kStages + 5 <= 24, "barriers fit");
  static_assert(kStageBytes % 1024 == 0, "swizzle atoms");
};

struct PairUnit {
  int m, n;      // tile of 256 rows x BN columns
  int bn;        // columns of the tile
  int job;       // 0, or 1: a weight gradient (forward: narrower tiles)
  int which;     // job 1: 0 dWg, 1 dWu, 2 dWd
  int k_blocks;
};

// The i-th unit of pair `pair`; false when that slot of the plan is empty.
template <int VAR, int BN, bool MIX>
__device__ __forceinline__ bool pair_unit(const PairArgs& p, int pair, int i, PairUnit& w) {
  int u;
  if (!plan_unit(p.plan, pair, i, w.job, u)) return false;
  w.which = 0;
  w.bn = BN;
  if constexpr (VAR < P_BWD1) {
    w.k_blocks = p.f.k_blocks;
    if (MIX && w.job) {
      w.bn = p.bn1;
      ordered_tile(u, p.f.m_tiles - p.m_split, p.n_tiles1, w.m, w.n);
      w.m += p.m_split;
    } else {
      w.job = 0;
      ordered_tile(u, MIX ? p.m_split : p.f.m_tiles, p.f.n_tiles, w.m, w.n);
    }
  } else if (w.job == 0) {
    w.k_blocks = p.f.k_blocks;
    ordered_tile(u, p.f.m_tiles, p.f.n_tiles, w.m, w.n);
  } else {
    w.k_blocks = p.k_blocks1;
    w.which = u >= 2 * p.u1 ? 2 : u >= p.u1 ? 1 : 0;
    u -= w.which * p.u1;
    if (w.which == 2) ordered_tile(u, p.m_tiles_h, p.n_tiles_i, w.m, w.n);
    else ordered_tile(u, p.m_tiles_i, p.n_tiles_h, w.m, w.n);
  }
  return true;
}

// This CTA's loads of one K block: its 128 rows of A, and its half of B's columns.
template <int VAR>
__device__ __forceinline__ void pair_load_a(const PairArgs& p, const PairMaps& t, const PairUnit& w, int kb,
                                            uint32_t sa, uint32_t bar, int rank) {
  const int k0 = kb * kFfnBK, m0 = w.m * 256 + rank * 128;
  if (VAR >= P_BWD1 && w.job) {
    const CUtensorMap* ta = &t.a1[w.which];
    tma_load_2d_pair(sa, ta, bar, m0, k0);
    tma_load_2d_pair(sa + 8192, ta, bar, m0 + 64, k0);
  } else if constexpr (VAR == P_BWD2) {
    const int half = kb < p.f.kb_split ? 0 : 1;
    tma_load_2d_pair(sa, &t.a[half], bar, k0 - half * p.f.kb_split * kFfnBK, m0);
  } else {
    tma_load_2d_pair(sa, &t.a[0], bar, k0, m0);
  }
}
template <int VAR, int BN, bool MIX>
__device__ __forceinline__ void pair_load_b(const PairArgs& p, const PairMaps& t, const PairUnit& w, int kb,
                                            uint32_t sb, uint32_t bar, int rank) {
  constexpr int HB = BN / 2;
  const int k0 = kb * kFfnBK;
  if constexpr (VAR == P_GATEUP) {  // the first CTA holds the gate rows, the second the same up rows
    tma_load_2d_pair(sb, MIX && w.job ? &t.b1[rank] : &t.b[rank], bar, k0, w.n * ((MIX ? w.bn : BN) / 2));
  } else if constexpr (VAR == P_DOWN) {
    const int bn = MIX ? w.bn : BN;
    tma_load_2d_pair(sb, MIX && w.job ? &t.b1[0] : &t.b[0], bar, k0, w.n * bn + rank * (bn / 2));
  } else {
    const int half = VAR == P_BWD2 && !w.job && kb >= p.f.kb_split ? 1 : 0;
    const CUtensorMap* tb = w.job ? &t.b1[w.which == 2 ? 1 : 0] : &t.b[half];
    const int kr = k0 - half * p.f.kb_split * kFfnBK;
#pragma unroll
    for (int j = 0; j < static_cast<int>(PairCfg<VAR, BN>::kBBoxes); ++j)
      tma_load_2d_pair(sb + j * 8192, tb, bar, w.n * BN + rank * HB + j * 64, kr);
  }
}

// One epilogue warp's output staging: two shared tiles of 32 rows x 64 bytes in the 64-byte TMA swizzle
// (chunk j of row r at j ^ ((r >> 1) & 3)), each stored by one TMA store that clips at the tensor's
// edges; a tile is refilled once its previous store has read it.
struct WarpStage {
  uint32_t base;
  int cur, lane;
  __device__ __forceinline__ void put(const uint4 (&ch)[4], const CUtensorMap* tm, int c0, int r0) {
    if (lane == 0) bulk_wait_read<1>();
    __syncwarp();
    const uint32_t b = base + static_cast<uint32_t>(cur) * 2048u;
    cur ^= 1;
    const uint32_t row = b + static_cast<uint32_t>(lane) * 64u;
#pragma unroll
    for (int j = 0; j < 4; ++j) st_shared_v4(row + (static_cast<uint32_t>(j ^ ((lane >> 1) & 3)) << 4), ch[j]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(tm, b, c0, r0);
      bulk_commit();
    }
  }
  __device__ __forceinline__ void put_bf16(const float (&v)[32], const CUtensorMap* tm, int c0, int r0) {
    uint4 ch[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      ch[j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                         pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
    put(ch, tm, c0, r0);
  }
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld_32x32b_x32(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// 32 columns of this lane's row of the saved factors (ffn_saved_offset), 4 columns per entry.  DACT keeps one
// chunk loaded ahead: its first one while the tile's MMAs run, the next one entry by entry as the current
// one is used (a chunk's loads issued and awaited in place took 2.3 us, four of them per warp and tile).
struct SavedChunk {
  float4 kg[8], ku[8];
};
__device__ __forceinline__ void saved_fetch(const FfnArgs& f, int row0, int lane, int col, int j, SavedChunk& s) {
  if (row0 < f.M && col + 4 * j < f.N) {
    const int64_t off = ffn_saved_offset(row0 + lane, col, f.N);
    s.kg[j] = __ldcs(reinterpret_cast<const float4*>(f.kg + off) + 32 * j);
    s.ku[j] = __ldcs(reinterpret_cast<const float4*>(f.ku + off) + 32 * j);
  }
}

// Epilogue of one tile for one warp: accumulator rows q * 32 ... (lane = row), column half h.
template <int VAR, int BN, bool MIX>
__device__ __forceinline__ void pair_epilogue(const PairArgs& p, const PairMaps& t, const PairUnit& w, int rank, int q,
                                              int h, int lane, uint32_t taddr, WarpStage& st, uint32_t tempty,
                                              SavedChunk& pre) {
  const FfnArgs& f = p.f;
  const int r0 = w.m * 256 + rank * 128 + q * 32;  // the warp's first row
  const bool rows = r0 < f.M;                       // (job 0)
  auto release = [&] {  // the accumulator's last column has been read
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive_cluster(tempty);
  };
  // this warp's 32-column chunks of the tile's: the first half (rounded up) or the rest
  const int bn = MIX ? w.bn : BN, chunks = (VAR == P_GATEUP ? bn / 2 : bn) / 32;
  const int c_beg = h ? (chunks + 1) / 2 * 32 : 0, c_end = h ? chunks * 32 : (chunks + 1) / 2 * 32;
  if constexpr (VAR == P_GATEUP) {
    const int c0 = w.n * (bn / 2);
#pragma unroll 1
    for (int c = c_beg; c < c_end; c += 32) {
      float g[32], u[32];
      tmem_ld32(taddr + c, g);
      tmem_ld32(taddr + bn / 2 + c, u);
      if (c + 32 >= c_end) release();
      if (!rows || c0 + c >= f.N) continue;
      if (f.kg) {
        const int64_t off = ffn_saved_offset(r0 + lane, c0 + c, f.N);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          float kg[4], ku[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) g[4 * j + k] = act_saved(g[4 * j + k], u[4 * j + k], f.act, kg[k], ku[k]);
          if (c0 + c + 4 * j < f.N) {
            __stcs(reinterpret_cast<float4*>(f.kg + off) + 32 * j, make_float4(kg[0], kg[1], kg[2], kg[3]));
            __stcs(reinterpret_cast<float4*>(f.ku + off) + 32 * j, make_float4(ku[0], ku[1], ku[2], ku[3]));
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) g[i] = act_fwd(g[i], f.act) * u[i];
      }
      st.put_bf16(g, &t.o[0], c0 + c, r0);
    }
    return;
  }
  if (VAR == P_BWD1 && !w.job) {  // DACT
    const int c0 = w.n * BN;
#pragma unroll 1
    for (int c = c_beg; c < c_end; c += 32) {
      uint4 dg[4], du[4];
      uint32_t* pg = reinterpret_cast<uint32_t*>(dg);
      uint32_t* pu = reinterpret_cast<uint32_t*>(du);
#pragma unroll
      for (int i = 0; i < 32; i += 16) {  // accumulator columns 16 at a time: registers
        float v[16];
        tmem_ld16(taddr + c + i, v);
        if (i == 16 && c + 32 >= c_end) release();
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int j = i / 4 + jj;
          float x[4] = {pre.kg[j].x, pre.kg[j].y, pre.kg[j].z, pre.kg[j].w};
          float y[4] = {pre.ku[j].x, pre.ku[j].y, pre.ku[j].z, pre.ku[j].w};
          if (c + 32 < c_end) saved_fetch(f, r0, lane, c0 + c + 32, j, pre);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[k] *= v[4 * jj + k];
            y[k] *= v[4 * jj + k];
          }
          pg[2 * j] = pack_bf16x2(x[0], x[1]);
          pg[2 * j + 1] = pack_bf16x2(x[2], x[3]);
          pu[2 * j] = pack_bf16x2(y[0], y[1]);
          pu[2 * j + 1] = pack_bf16x2(y[2], y[3]);
        }
      }
      if (!rows || c0 + c >= f.N) continue;
      st.put(dg, &t.o[0], c0 + c, r0);
      st.put(du, &t.o[1], c0 + c, r0);
    }
  } else {
    const bool dw = VAR >= P_BWD1 && w.job;
    const int M = !dw ? f.M : w.which == 2 ? p.H : p.I, N = !dw ? f.N : w.which == 2 ? p.I : p.H;
    const CUtensorMap* to = dw ? &t.o1[w.which] : &t.o[0];
    const uint16_t* add = dw ? nullptr : f.residual;
    const int c0 = w.n * bn;
#pragma unroll 1
    for (int c = c_beg; c < c_end; c += 32) {
      const bool in = r0 < M && c0 + c < N;
      uint4 res[4];
      if constexpr (VAR == P_DOWN || VAR == P_BWD2) {
        if (add && in && r0 + lane < M) {
          const uint4* s = reinterpret_cast<const uint4*>(add + static_cast<int64_t>(r0 + lane) * N + c0 + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) res[j] = c0 + c + 8 * j < N ? s[j] : make_uint4(0, 0, 0, 0);
        }
      }
      float v[32];
      tmem_ld32(taddr + c, v);
      if (c + 32 >= c_end) release();
      if (!in) continue;
      if constexpr (VAR == P_DOWN || VAR == P_BWD2) {
        if (add && r0 + lane < M) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t r[4] = {res[j].x, res[j].y, res[j].z, res[j].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              v[8 * j + 2 * k] += bf16_lo(r[k]);
              v[8 * j + 2 * k + 1] += bf16_hi(r[k]);
            }
          }
        }
      }
      if (dw && f.out_f32) {
#pragma unroll
        for (int k = 0; k < 32; k += 16) {
          uint4 ch[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            ch[j] = make_uint4(__float_as_uint(v[k + 4 * j]), __float_as_uint(v[k + 4 * j + 1]),
                               __float_as_uint(v[k + 4 * j + 2]), __float_as_uint(v[k + 4 * j + 3]));
          if (c0 + c + k < N) st.put(ch, to, c0 + c + k, r0);
        }
      } else {
        st.put_bf16(v, to, c0 + c, r0);
      }
    }
  }
}

template <int VAR, int BN, bool MIX>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    ffn_pair_kernel(const __grid_constant__ PairMaps t, const PairArgs p) {
  using C = PairCfg<VAR, BN>;
  constexpr int S = C::kStages;
  constexpr bool kBmn = C::kBmn;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // swizzle atoms: 1024-byte aligned
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem_raw + (base - raw) + C::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 24);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  // the pair counts loads and accumulator releases on the first CTA's full / tempty barriers; each
  // CTA has its own empty, tfull and drain barriers, on which the first CTA's commits arrive
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (S + s); };
  auto tfull = [&](int a) { return bar0 + 8u * (2 * S + a); };
  auto tempty = [&](int a) { return bar0 + 8u * (2 * S + 2 + a); };
  const uint32_t drain = bar0 + 8u * (2 * S + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = static_cast<int>(blockIdx.x >> 1), steps = plan_steps(p.plan, pair);
  uint32_t* status = p.f.status;
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(tfull(a), 1);
      mbar_init(tempty(a), 16);  // eight warps of each CTA
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_barrier_init();
    if (p.plan.units[0]) {  // (a backward's launch may have weight gradients only)
      tma_prefetch_desc(&t.a[0]);
      tma_prefetch_desc(&t.b[0]);
      tma_prefetch_desc(&t.o[0]);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kPairTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // the peer's barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // DOWN and DX always follow another kernel of this block, which runs once everything before it has ended:
  // their first weights are loaded before its end
  constexpr bool kEarlyB = VAR == P_DOWN || VAR == P_BWD2;

  if (warp == 0) {
    int ahead = 0;
    if constexpr (kEarlyB) {
      PairUnit w;
      if (steps > 0 && pair_unit<VAR, BN, MIX>(p, pair, 0, w) && (VAR == P_DOWN || !w.job)) {
        ahead = min(w.k_blocks, S);
        for (int kb = 0; kb < ahead; ++kb)
          if (elect_one()) {
            if (rank == 0) mbar_arrive_expect_tx(full(kb), C::tx_bytes(MIX ? w.bn : BN));
            pair_load_b<VAR, BN, MIX>(p, t, w, kb, base + kb * C::kStageBytes + C::kABytes, mapa_shared(full(kb), 0), rank);
          }
      }
    }
    pdl_wait();
    pdl_trigger();
    int st = 0, issued = 0;
    uint32_t ph = 0;
    bool ok = true;
    for (int i = 0; i < steps && ok; ++i) {
      PairUnit w;
      if (!pair_unit<VAR, BN, MIX>(p, pair, i, w)) continue;
      for (int kb = 0; kb < w.k_blocks; ++kb) {
        if (!warp_wait(empty(st), ph ^ 1u, abort_flag, status)) {
          ok = false;
          break;
        }
        const uint32_t sa = base + st * C::kStageBytes, bar = mapa_shared(full(st), 0);
        if (elect_one()) {
          if (issued >= ahead) {
            if (rank == 0) mbar_arrive_expect_tx(full(st), C::tx_bytes(MIX ? w.bn : BN));
            pair_load_b<VAR, BN, MIX>(p, t, w, kb, sa + C::kABytes, bar, rank);
          }
          pair_load_a<VAR>(p, t, w, kb, sa, bar, rank);
        }
        ++issued;
        if (++st == S) {
          st = 0;
          ph ^= 1u;
        }
      }
    }
    if (!ok && rank == 0 && lane == 0)  // let the copies in flight land: the last one of each stage
      for (int b = issued > S ? issued - S : 0; b < issued; ++b)
        wait_landed(full(b % S), static_cast<uint32_t>(b / S) & 1u);
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      pdl_wait();  // the kernel in front may take its time: no bounded wait starts before its end
      int st = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int i = 0; i < steps && ok; ++i) {
        PairUnit w;
        if (!pair_unit<VAR, BN, MIX>(p, pair, i, w)) continue;
        const bool amn = VAR >= P_BWD1 && w.job;  // A's layout goes by the job
        const uint32_t idesc = MIX        ? idesc_bf16(256, w.bn, false, kBmn)
                               : amn        ? idesc_bf16(256, BN, true, kBmn)
                                            : idesc_bf16(256, BN, false, kBmn);
        const uint32_t a_step = amn ? 128 : 2, a_lbo = amn ? 8192 : 16;  // steps count 16-byte units
        if (!__all_sync(0xffffffffu, mbar_wait<true>(tempty(acc), aph ^ 1u, abort_flag, status))) break;
        tc_fence_after();
        const uint32_t d = tmem + static_cast<uint32_t>(acc) * 256u;
        for (int kb = 0; kb < w.k_blocks; ++kb) {
          if (!warp_wait(full(st), ph, abort_flag, status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t sa = base + st * C::kStageBytes, sb = sa + C::kABytes;
          const uint64_t ad = sdesc_sw128(sa, a_lbo, 1024);
          const uint64_t bd = kBmn ? sdesc_sw128(sb, 8192, 1024) : sdesc_sw128(sb, 16, 1024);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              umma_bf16_pair(d, ad + ks * a_step, bd + ks * (kBmn ? 128 : 2), idesc, (kb | ks) != 0 ? 1u : 0u);
            umma_commit_pair(empty(st));
          }
          if (++st == S) {
            st = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        if (elect_one()) umma_commit_pair(tfull(acc));
        if (++acc == 2) {
          acc = 0;
          aph ^= 1u;
        }
      }
      // every MMA issued has ended before TMEM is freed, in both CTAs
      if (elect_one()) umma_commit_pair(drain);
    }
    __syncwarp();
    if (lane == 0) wait_landed(drain, 0);
    __syncwarp();
  } else {
    const int q = warp & 3, h = (warp - 2) >> 2;
    pdl_wait();  // the residual, the saved factors, and outputs that an earlier kernel may still read
    WarpStage st{base + C::kStagingOff + static_cast<uint32_t>(warp - 2) * 4096u, 0, lane};
    int acc = 0;
    uint32_t aph = 0;
    for (int i = 0; i < steps; ++i) {
      PairUnit w;
      if (!pair_unit<VAR, BN, MIX>(p, pair, i, w)) continue;
      SavedChunk pre;
      if (VAR == P_BWD1 && !w.job) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          saved_fetch(p.f, w.m * 256 + rank * 128 + q * 32, lane, w.n * BN + (h ? (BN / 32 + 1) / 2 * 32 : 0), j, pre);
      }
      int ok = 0;
      if (lane == 0) ok = mbar_wait_tile(tfull(acc), aph, w.k_blocks, abort_flag, status) ? 1 : 0;
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      tc_fence_after();
      pair_epilogue<VAR, BN, MIX>(p, t, w, rank, q, h, lane,
                             tmem + (static_cast<uint32_t>(q * 32) << 16) + static_cast<uint32_t>(acc) * 256u, st,
                             mapa_shared(tempty(acc), 0), pre);
      if (++acc == 2) {
        acc = 0;
        aph ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_read<0>();  // the staging tiles have been read; the grid's end waits for the writes
    __syncwarp();
  }
  if (*abort_flag) {  // failure path: copies or arrivals of the peer may still be in flight
    const uint64_t t0 = global_timer_ns();
    while (global_timer_ns() - t0 < kWaitLimitNs / 100) {
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // neither CTA leaves while the other may still address it
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kPairTmemCols);
  }
}

template <int VAR, int BN, bool MIX>
int launch_pair(const PairMaps& maps, const PairArgs& p, cudaStream_t stream) {
  using C = PairCfg<VAR, BN>;
  static DeviceOnce once;
  const int se = once.run([](int* d) { return static_cast<int>(cudaGetDevice(d)); },
                          [] {
                            return static_cast<int>(cudaFuncSetAttribute(ffn_pair_kernel<VAR, BN, MIX>,
                                                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                         static_cast<int>(C::kSmemBytes)));
                          },
                          static_cast<int>(cudaErrorInvalidDevice));
  if (se) return se;
  constexpr int kKind = VAR == P_BWD1 ? static_cast<int>(K_FFN_BWD1)
                        : VAR == P_BWD2 ? static_cast<int>(K_FFN_BWD2) : K_FFN_GATEUP + VAR;
  trace_begin(stream, kKind);
  const cudaError_t e =
      launch_pdl(ffn_pair_kernel<VAR, BN, MIX>, dim3(2 * p.plan.pairs), dim3(kPairThreads), C::kSmemBytes, stream, maps, p);
  trace_end(stream);
  return static_cast<int>(e);
}

bool fits(const int64_t (&units)[2]) { return units[0] + units[1] < (int64_t{1} << 30); }

// GATEUP or DOWN: M rows, N output columns, K, in the widths of `d`.
template <int VAR, int BN>
int pair_fwd(int64_t M, int64_t N, int64_t K, const FwdSplit& d, int pairs, const FfnOperands& o, const FfnArgs& f,
             cudaStream_t stream) {
  auto out_cols = [](int bn) { return VAR == P_GATEUP ? bn / 2 : bn; };
  const int64_t mt = tiles_of(M, 256), kb = tiles_of(K, kFfnBK);
  PairArgs p{};
  p.f = f;
  p.f.M = static_cast<int32_t>(M);
  p.f.N = static_cast<int32_t>(N);
  p.f.m_tiles = static_cast<int32_t>(mt);
  p.f.n_tiles = static_cast<int32_t>(tiles_of(N, out_cols(BN)));
  p.f.k_blocks = static_cast<int32_t>(kb);
  p.bn1 = d.bn1;
  p.m_split = static_cast<int32_t>(d.m_split);
  p.n_tiles1 = d.bn1 ? static_cast<int32_t>(tiles_of(N, out_cols(d.bn1))) : 0;
  const int64_t units[2] = {d.m_split * p.f.n_tiles, (mt - d.m_split) * p.n_tiles1};
  if (!fits(units)) return static_cast<int>(cudaErrorInvalidValue);
  make_plan(units, {fwd_cost(kb, BN), d.bn1 ? fwd_cost(kb, d.bn1) : 1}, true, pairs, &p.plan);
  const uint64_t um = static_cast<uint64_t>(M), un = static_cast<uint64_t>(N), uk = static_cast<uint64_t>(K);
  PairMaps t{};
  const uint32_t h0 = BN / 2, h1 = static_cast<uint32_t>(d.bn1) / 2;
  bool good = make_tmap_bf16(&t.a[0], o.a, uk, um, 64, 128) && make_tmap_bf16(&t.b[0], o.b, uk, un, 64, h0) &&
              make_tmap_bf16_sw64(&t.o[0], f.out0, un, um, 32, 32);
  if constexpr (VAR == P_GATEUP) good = good && make_tmap_bf16(&t.b[1], o.b2, uk, un, 64, h0);
  if (d.bn1) {
    good = good && make_tmap_bf16(&t.b1[0], o.b, uk, un, 64, h1);
    if constexpr (VAR == P_GATEUP) good = good && make_tmap_bf16(&t.b1[1], o.b2, uk, un, 64, h1);
  }
  if (!good) return static_cast<int>(cudaErrorInvalidValue);
  if constexpr (BN > 128) {
    if (d.bn1) return launch_pair<VAR, BN, true>(t, p, stream);
  }
  return launch_pair<VAR, BN, false>(t, p, stream);
}

template <int VAR>
int pair_fwd_any(int64_t M, int64_t N, int64_t K, const FfnOperands& o, const FfnArgs& f, cudaStream_t stream) {
  const int pairs = sm_count() / 2;
  if (pairs <= 0) return static_cast<int>(cudaErrorInvalidDevice);
  const FwdSplit d = fwd_split(VAR == P_GATEUP, M, N, K, pairs);
  if constexpr (VAR == P_DOWN) {
    if (d.bn0 == 224) return pair_fwd<VAR, 224>(M, N, K, d, pairs, o, f, stream);
  }
  if (d.bn0 == 256) return pair_fwd<VAR, 256>(M, N, K, d, pairs, o, f, stream);
  if (d.bn0 == 192) return pair_fwd<VAR, 192>(M, N, K, d, pairs, o, f, stream);
  return pair_fwd<VAR, 128>(M, N, K, d, pairs, o, f, stream);
}

template <int VAR>
constexpr int phase_of() { return VAR == P_BWD1 ? 1 : 2; }

template <int VAR, int BN>
int pair_bwd(const FfnBackward& b, const BwdJobs& j, int pairs, cudaStream_t stream) {
  const int64_t cols = VAR == P_BWD1 ? b.I : b.H;
  PairArgs p{};
  p.f.M = static_cast<int32_t>(b.T);
  p.f.N = static_cast<int32_t>(cols);
  p.f.m_tiles = static_cast<int32_t>(tiles_of(b.T, 256));
  p.f.n_tiles = static_cast<int32_t>(tiles_of(cols, BN));
  p.f.kb_split = static_cast<int32_t>(tiles_of(VAR == P_BWD1 ? b.H : b.I, kFfnBK));
  p.f.k_blocks = p.f.kb_split * (VAR == P_BWD2 ? 2 : 1);
  p.f.act = b.act;
  p.f.out_f32 = b.dw_f32;
  p.f.status = b.status;
  p.f.kg = const_cast<float*>(b.kg);
  p.f.ku = const_cast<float*>(b.ku);
  p.f.residual = static_cast<const uint16_t*>(b.dx_add);
  p.H = static_cast<int32_t>(b.H);
  p.I = static_cast<int32_t>(b.I);
  p.m_tiles_i = static_cast<int32_t>(tiles_of(b.I, 256));
  p.n_tiles_h = static_cast<int32_t>(tiles_of(b.H, BN));
  p.m_tiles_h = static_cast<int32_t>(tiles_of(b.H, 256));
  p.n_tiles_i = static_cast<int32_t>(tiles_of(b.I, BN));
  p.u1 = j.gate_up ? p.m_tiles_i * p.n_tiles_h : 0;
  p.k_blocks1 = static_cast<int32_t>(tiles_of(b.T, kFfnBK));
  int64_t units[2];
  bwd_tiles(phase_of<VAR>(), b.T, b.H, b.I, j, BN, units);
  if (!fits(units)) return static_cast<int>(cudaErrorInvalidValue);
  make_plan(units, {p.f.k_blocks, p.k_blocks1}, rows_first(phase_of<VAR>()), pairs, &p.plan);
  const uint64_t t = static_cast<uint64_t>(b.T), h = static_cast<uint64_t>(b.H), i = static_cast<uint64_t>(b.I);
  PairMaps m{};
  auto dw_map = [&](CUtensorMap* tm, void* d, uint64_t inner, uint64_t outer) {
    return b.dw_f32 ? make_tmap_f32_sw64(tm, d, inner, outer, 16, 32)
                    : make_tmap_bf16_sw64(tm, d, inner, outer, 32, 32);
  };
  bool good = true;
  if (j.rows && VAR == P_BWD1)
    good = make_tmap_bf16(&m.a[0], b.dy, h, t, 64, 128) && make_tmap_bf16(&m.b[0], b.w_down, i, h, 64, 64) &&
           make_tmap_bf16_sw64(&m.o[0], b.dg, i, t, 32, 32) && make_tmap_bf16_sw64(&m.o[1], b.du, i, t, 32, 32);
  else if (j.rows)
    good = make_tmap_bf16(&m.a[0], b.dg, i, t, 64, 128) && make_tmap_bf16(&m.a[1], b.du, i, t, 64, 128) &&
           make_tmap_bf16(&m.b[0], b.w_gate, h, i, 64, 64) && make_tmap_bf16(&m.b[1], b.w_up, h, i, 64, 64) &&
           make_tmap_bf16_sw64(&m.o[0], b.dx, h, t, 32, 32);
  if (good && j.gate_up)
    good = make_tmap_bf16(&m.a1[0], b.dg, i, t, 64, 64) && make_tmap_bf16(&m.a1[1], b.du, i, t, 64, 64) &&
           make_tmap_bf16(&m.b1[0], b.x, h, t, 64, 64) && dw_map(&m.o1[0], b.dw_gate, h, i) &&
           dw_map(&m.o1[1], b.dw_up, h, i);
  if (good && j.down)
    good = make_tmap_bf16(&m.a1[2], b.dy, h, t, 64, 64) && make_tmap_bf16(&m.b1[1], b.a, i, t, 64, 64) &&
           dw_map(&m.o1[2], b.dw_down, i, h);
  if (!good) return static_cast<int>(cudaErrorInvalidValue);
  return launch_pair<VAR, BN, false>(m, p, stream);
}

template <int VAR>
int pair_bwd_any(const FfnBackward& b, const BwdJobs& j, int pairs, cudaStream_t stream) {
  switch (bwd_width(phase_of<VAR>(), b.T, b.H, b.I, j, pairs).bn) {
    case 0: return 0;
    case 256: return pair_bwd<VAR, 256>(b, j, pairs, stream);
    case 224: return pair_bwd<VAR, 224>(b, j, pairs, stream);
    case 192: return pair_bwd<VAR, 192>(b, j, pairs, stream);
    default: return pair_bwd<VAR, 128>(b, j, pairs, stream);
  }
}

}  // namespace

int launch_ffn_pair_fwd(int var, int64_t M, int64_t N, int64_t K, const FfnOperands& o, const FfnArgs& a,
                        cudaStream_t stream) {
  return var == F_GATEUP ? pair_fwd_any<P_GATEUP>(M, N, K, o, a, stream)
                         : pair_fwd_any<P_DOWN>(M, N, K, o, a, stream);
}

int launch_ffn_pair_bwd(int phase, const FfnBackward& b, cudaStream_t stream) {
  const int pairs = sm_count() / 2;
  if (pairs <= 0) return static_cast<int>(cudaErrorInvalidDevice);
  BwdJobs one, two;
  bwd_jobs(b.T, b.H, b.I, b.dact, b.dx_rows, b.dw_gate != nullptr, b.dw_down != nullptr, pairs, &one, &two);
  return phase == 1 ? pair_bwd_any<P_BWD1>(b, one, pairs, stream) : pair_bwd_any<P_BWD2>(b, two, pairs, stream);
}

}  // namespace mok
