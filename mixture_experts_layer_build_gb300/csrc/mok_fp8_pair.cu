// mok_fp8_pair.cu -- 8-bit products with a scale per 128 values for many rows: persistent CTA pairs.
//
// A cluster of two CTAs computes 256 x BN tiles (BN 256 or 128, of row-scaled products 192 as well) with
// tcgen05.mma.cta_group::2: each CTA loads its own 128 rows of P and half of Q's rows, 32 KB per K block of 128 of a 256 x 256
// tile.  The scales belong to whole K blocks, so every block's products go to a TMEM accumulator of their own, one of
// 512 / BN in turn; eight warps per CTA drain it, two per TMEM lane quarter with half of the columns each, times the
// block's scales into fp32 registers (BN / 2 per thread), while the MMAs fill the next one.  A tile's output goes through
// shared memory and leaves by TMA while the next tile's blocks are in the tensor cores.
//
// Modes: dense rows; a schedule's rows against one matrix per expert (the units of 256 rows are counted from the
// expert counts on the device, by every CTA for itself); weight gradients, whose K blocks are the 128-row blocks
// of an expert's rows.
//
// What bounds it: an accumulator is free for new MMAs once all of its columns have been read, and there are two of 256
// columns, so a K block takes half of MMAs + commit + drain + release: 0.43 us (0.30 where nothing is drained: the loads
// from L2), of which the reads of TMEM are 0.04 and the multiply-adds 0.05.  Measured: 4096 x 7168 x 2048 54 us (2,210
// TFLOP/s; a library product with one scale for all 43), 8192 x 8192 x 8192 395 to 404 us (2,750; 282), both operands row-scaled
// 71 and 542: twice the multiply-adds, and column scales from shared memory.  Per tile 1.2 us more for its output.
// Measured and not kept: a release at cluster scope per K block (a memory barrier: 110 us for 56); four accumulators of 128
// columns, two MMA groups per block (504 us for 8192 cubed: A is read from shared memory twice); scales fetched by the
// drain warps (a column-scaled block waits 0.15 us more); column scales broadcast to a thread per row (588 us for 550); four
// or six stages for five (with one staging box per warp; with two there is room for four), the schedule's tables in shared memory, or read a tile ahead (no change); the next
// kernel let start early (its waiting CTAs: a training step of 64 experts 490 us for 459).
#include "mok_ffn.cuh"  // warp_wait, wait_landed, elect_one, ordered_tile
#include "mok_fp8_gemm.cuh"
#include "mok_stage.cuh"

namespace mok {
namespace {

// Warpgroup 0: warp 0 loads, warp 1 issues MMAs; warpgroups 1 and 2 drain.  A drain thread of a 256-column tile needs more
// registers than a third of the SM's (168 of 384 threads): the first group gives up of its own.  What the groups have is at
// most what the launch had: 128 x 72 + 256 x 216 = 384 x 168.  208 for threads of 128 columns: 8192 x 8192 x 8192 409 us, 414 with
// 224, 453 with 200 (with one staging box).
constexpr int kThreads = 384;
constexpr int kDrain = 4;  // the first drain warp
constexpr int kMaxExperts = 1024;

struct PairArgs {
  Fp8Problem g;
  int32_t pairs;
  int32_t units;  // dense, weight gradients; a schedule's are counted on the device
};
struct PairMaps {
  CUtensorMap p, q, out;
};

// 16 TMEM lanes x 64 columns: register 4 n + k of thread t holds lane t / 4 + 8 (k / 2), column 8 n + 2 (t % 4) + k % 2.
__device__ __forceinline__ void tmem_ld_16x256b_x8(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x8.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

// The same for 32 columns.
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

// ALT: the two drain warpgroups take tiles of 128 columns in turn, each with accumulators and scale slots of its own, so that
// one's output leaves while the other drains: for row-scaled products with few K blocks, such as experts' weight gradients
// (64 experts with 384 rows each, 1024 x 2048: 139 us in tiles of 256, 112 to 116 so; without any output 91, without
// multiply-adds either 71; with one staging box per warp 121, stores straight from registers 140).
template <int BN, bool COLVEC, bool ALT>
struct Cfg {
  static_assert(!ALT || BN == 128, "a thread of an alternating group holds all of a tile's columns");
  static constexpr int kGroups = ALT ? 2 : 1;
  static constexpr int HB = ALT ? BN : BN / 2;  // columns of a drain thread
  static constexpr int kLow = 72, kHigh = HB == 128 ? 208 : 216;  // registers per thread
  static_assert(COLVEC || HB == 64 || HB == 128, "a thread's columns are in one block of 128");
  static constexpr int kBox = HB % 64 == 0 ? 64 : 32;  // columns of a box of bf16 output (128 or 64 bytes)
  static constexpr int kAccs = 512 / BN / kGroups;     // accumulators in TMEM, of a group
  static constexpr uint32_t kQBytes = BN / 2 * 128, kStage = 16384 + kQBytes, kTx = 2 * kStage;
  // boxes of 32 rows x 128 bytes that a drain warp stages output in: with two, a box is written while the other one is read, for a
  // stage of loads less (8192 x 8192 x 8192 407 us with one, 395 with two; tiles of 192 columns, 1536 x 4096 over 8192, 70.6 and
  // 71.8; 128 columns alike)
  static constexpr int kBoxes = ALT || BN == 256 ? 2 : 1;
  static constexpr uint32_t kStaging = kBoxes * 4096;
  // scales of a K block: the CTA's 128 rows', and (COLVEC) the tile's columns'.  A group's slot is filled again once the MMAs of
  // kStages blocks before have ended, and so the group's blocks kAccs further back have been drained.
  static constexpr int kSlots = ALT ? 8 : BN == 256 ? 8 : 12;
  static constexpr uint32_t kScales = 512 + (COLVEC ? BN * 4 : 0);
  static constexpr uint32_t kMost = 227328;      // 5 KB of 227 are static
  static constexpr uint32_t kFixed = 1024 + 8 * kStaging + kGroups * kSlots * kScales + 512;
  static constexpr int kStages = (kMost - kFixed) / kStage < 8 ? (kMost - kFixed) / kStage : 8;
  static constexpr uint32_t kStagingOff = kStages * kStage;
  static constexpr uint32_t kScaleOff = kStagingOff + 8 * kStaging;
  static constexpr uint32_t kBarOff = kScaleOff + kGroups * kSlots * kScales;
  static constexpr uint32_t kSmem = 1024 + kBarOff + 512;
  static_assert(2 * kStages + kGroups * (2 * kAccs + kSlots) + 1 <= 48, "barriers fit");
  static_assert(kSlots > kStages + kAccs, "scales stay until they are used");
};

struct Unit {
  int32_t p0, q0;           // first rows of the pair's tile in the operands' tensor maps
  int32_t row0, row_end;    // output rows: row0 + r for tile row r, below row_end
  int32_t j0;
  int32_t kb0, count;
  int32_t batch;
};

// Unit u: p0 is the pair's first row of P, rank adds 128.  `prefix`: (grouped) units of 256 rows before each expert.
__device__ __forceinline__ void pair_unit(const Fp8Problem& g, const int* prefix, int u, int bn, Unit& w) {
  w.kb0 = 0;
  w.count = g.k_blocks;
  w.batch = 0;
  if (g.mode == FP8_DENSE) {
    int m, n;
    ordered_tile(u, g.p_tiles, g.q_tiles, m, n);
    w.p0 = w.row0 = m * 256;
    w.row_end = g.p_rows;
    w.j0 = w.q0 = n * bn;
  } else if (g.mode == FP8_WGRAD) {
    const int per = g.p_tiles * g.q_tiles, e = u / per;
    int m, n;
    ordered_tile(u - e * per, g.p_tiles, g.q_tiles, m, n);
    w.batch = e;
    w.kb0 = __ldg(g.poff + e) / 128;
    w.count = __ldg(g.poff + e + 1) / 128 - w.kb0;
    w.p0 = m * 256;
    w.row0 = e * g.p_rows + w.p0;
    w.row_end = (e + 1) * g.p_rows;
    w.j0 = w.q0 = n * bn;
  } else {
    const int mu = u / g.q_tiles, n = u - mu * g.q_tiles;
    int lo = 0, hi = g.experts - 1;  // the last expert whose units begin at or before mu
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (prefix[mid] <= mu) lo = mid;
      else hi = mid - 1;
    }
    const int first = __ldg(g.poff + lo);
    w.batch = lo;
    w.p0 = w.row0 = first + (mu - prefix[lo]) * 256;
    w.row_end = first + __ldg(g.counts + lo);
    w.j0 = n * bn;
    w.q0 = lo * g.q_rows + w.j0;
  }
}

// prefix[e] = units of 256 rows of the experts before e; returns their number.  All threads.
__device__ __forceinline__ int count_units(const Fp8Problem& g, int* prefix, int* wsum) {
  constexpr int kPer = (kMaxExperts + kThreads - 1) / kThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, e0 = threadIdx.x * kPer;
  int v[kPer], sum = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    v[i] = e0 + i < g.experts ? (__ldg(g.counts + e0 + i) + 255) / 256 : 0;
    sum += v[i];
  }
  int incl = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) wsum[warp] = incl;
  __syncthreads();
  int at = incl - sum, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) at += wsum[w];
    total += wsum[w];
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (e0 + i < g.experts) prefix[e0 + i] = at;
    at += v[i];
  }
  __syncthreads();
  return total;
}

template <int BN, bool COLVEC, bool ALT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ PairMaps t, const PairArgs a) {
  using C = Cfg<BN, COLVEC, ALT>;
  constexpr int S = C::kStages, HB = C::HB, kAccs = C::kAccs, kAll = C::kGroups * kAccs;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int prefix[kMaxExperts];
  __shared__ int wsum[kThreads / 32];
  const Fp8Problem& g = a.g;
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;  // swizzle atoms: 1024-byte aligned
  uint8_t* smem = smem_raw + (base - raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 48);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const uint32_t bar0 = smem_u32(bars);
  // the pair counts loads and drained accumulators on the first CTA's full / tempty barriers; each CTA has its own
  // empty, tfull and drain barriers, on which the first CTA's commits arrive
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (S + s); };
  auto tfull = [&](int b) { return bar0 + 8u * (2 * S + b); };
  auto tempty = [&](int b) { return bar0 + 8u * (2 * S + kAll + b); };
  const uint32_t drain = bar0 + 8u * (2 * S + 2 * kAll);
  auto sfull = [&](int i) { return drain + 8u * (1 + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int pair = static_cast<int>(blockIdx.x >> 1);
  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < kAll; ++b) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), 16 / C::kGroups);  // the warps that drain it, of both CTAs
    }
    mbar_init(drain, 1);
    for (int i = 0; i < C::kGroups * C::kSlots; ++i) mbar_init(sfull(i), 1);
    *abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&t.p);
    tma_prefetch_desc(&t.q);
    tma_prefetch_desc(&t.out);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  int units = a.units;
  if (g.mode != FP8_DENSE) pdl_wait();  // the schedule's tables
  if (g.mode == FP8_GROUPED) units = count_units(g, prefix, wsum) * g.q_tiles;
  tc_fence_before();
  cluster_sync();  // the peer's barriers exist before anything arrives on them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // (roles in one branch with their setmaxnreg: only then does the compiler give the drain code its registers)
  if (warp < kDrain) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLow));
  if (warp == 0) {
    int ahead = 0;
    auto load_q = [&](const Unit& w, int kb, int st) {
      tma_load_2d_pair(base + st * C::kStage + 16384, &t.q, mapa_shared(full(st), 0), (w.kb0 + kb) * 128, w.q0 + rank * (BN / 2));
    };
    if (g.early_q && pair < units) {  // weights: nothing that still runs writes them
      Unit w;
      pair_unit(g, prefix, pair, BN, w);
      ahead = min(w.count, S);
      for (int kb = 0; kb < ahead; ++kb)
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(full(kb), C::kTx);
          load_q(w, kb, kb);
        }
    }
    pdl_wait();
    int st = 0, issued = 0, slot = 0, slot2 = C::kSlots;  // (the other group's next one)
    uint32_t ph = 0;
    bool ok = true;
    for (int u = pair; u < units && ok; u += a.pairs) {
      Unit w;
      pair_unit(g, prefix, u, BN, w);
      // the scales that go with a block: this CTA's rows' and all columns', as many as there are (rounded up to four)
      const int row = w.p0 + rank * 128;
      const int64_t rows = g.p_pitch - row, cols = g.q_pitch - w.j0;
      const uint32_t pb = rows <= 0 ? 0u : rows < 128 ? static_cast<uint32_t>(rows) * 4u : 512u;
      const uint32_t qb = !COLVEC ? 0u : cols < BN ? static_cast<uint32_t>(cols) * 4u : BN * 4u;
      for (int kb = 0; kb < w.count; ++kb) {
        if (!warp_wait(empty(st), ph ^ 1u, abort_flag, g.status)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          if (issued >= ahead) {
            if (rank == 0) mbar_arrive_expect_tx(full(st), C::kTx);
            load_q(w, kb, st);
          }
          tma_load_2d_pair(base + st * C::kStage, &t.p, mapa_shared(full(st), 0), (w.kb0 + kb) * 128, row);
          const uint32_t to = base + C::kScaleOff + slot * C::kScales;
          const int64_t k = w.kb0 + kb;
          mbar_arrive_expect_tx(sfull(slot), pb + qb);
          if (pb) bulk_load(to, g.sp + k * g.p_pitch + row, pb, sfull(slot));
          if (qb) bulk_load(to + 512, g.sq + k * g.q_pitch + w.j0, qb, sfull(slot));
        }
        ++issued;
        if (!ALT) slot = slot + 1 == C::kSlots ? 0 : slot + 1;
        else slot = slot + 1 == C::kSlots ? 0 : slot + 1 == 2 * C::kSlots ? C::kSlots : slot + 1;
        if (++st == S) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (ALT) {
        const int x = slot;
        slot = slot2;
        slot2 = x;
      }
    }
    if (!ok && rank == 0 && lane == 0)  // let the copies in flight land: the last one of each stage
      for (int b = issued > S ? issued - S : 0; b < issued; ++b) wait_landed(full(b % S), static_cast<uint32_t>(b / S) & 1u);
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      pdl_wait();  // the kernel in front may take its time: no bounded wait starts before its end
      int st = 0, n = 0, n2 = 0, first = 0;  // the group's blocks, and the other's; the group's first accumulator
      uint32_t ph = 0;
      bool ok = true;
      for (int u = pair; u < units && ok; u += a.pairs) {
        Unit w;
        pair_unit(g, prefix, u, BN, w);
        for (int kb = 0; kb < w.count; ++kb, ++n) {
          const int b = first + n % kAccs;
          const uint32_t read = static_cast<uint32_t>(n / kAccs - 1) & 1u;  // parity of that accumulator's last drain
          ok = (n < kAccs || warp_wait(tempty(b), read, abort_flag, g.status)) && warp_wait(full(st), ph, abort_flag, g.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sp = base + st * C::kStage;
          const uint64_t pd = sdesc_sw128(sp, 16, 1024), qd = sdesc_sw128(sp + 16384, 16, 1024);
          if (elect_one()) {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)  // 32 bytes of K; descriptors count 16-byte units
              umma_fp8_pair(tmem + b * BN, pd + ks * 2, qd + ks * 2, idesc_fp8(256, BN), ks > 0 ? 1u : 0u);
            umma_commit_pair(tfull(b));
            umma_commit_pair(empty(st));
          }
          if (++st == S) {
            st = 0;
            ph ^= 1u;
          }
        }
        if (ALT) {
          const int x = n;
          n = n2;
          n2 = x;
          first ^= kAccs;
        }
      }
      if (elect_one()) umma_commit_pair(drain);  // every MMA issued has ended before TMEM is freed, in both CTAs
    }
    __syncwarp();
    if (lane == 0) wait_landed(drain, 0);
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kHigh));
    const int q = warp & 3, dw = warp - kDrain, h = ALT ? 0 : dw >> 2, group = ALT ? dw >> 2 : 0;
    pdl_wait();
    const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16) + h * HB;
    const uint32_t stage0 = base + C::kStagingOff + static_cast<uint32_t>(dw) * C::kStaging;
    uint32_t stage = stage0;
    int n = 0;
    bool ok = true;
    for (int u = pair + group * a.pairs; u < units; u += C::kGroups * a.pairs) {
      Unit w;
      pair_unit(g, prefix, u, BN, w);
      const int j0 = w.j0 + h * HB;
      float acc[HB];
#pragma unroll
      for (int j = 0; j < HB; ++j) acc[j] = 0.0f;
      // the tile's column blocks' scales (one per thread's columns), 32 K blocks at a time and one lot ahead, a lane each
      const float* qs = g.sq + w.batch * g.q_batch + static_cast<int64_t>(min(j0, g.q_rows - 1) / 128) * g.k_blocks;
      float q_now = 0.0f, q_next = !COLVEC && lane < w.count ? __ldg(qs + lane) : 0.0f;
      for (int kb = 0; kb < w.count; ++kb, ++n) {
        if (!COLVEC && kb % 32 == 0) {
          q_now = q_next;
          if (kb + 32 + lane < w.count) q_next = __ldg(qs + kb + 32 + lane);
        }
        const int slot = group * C::kSlots + n % C::kSlots;
        ok = warp_wait(sfull(slot), static_cast<uint32_t>(n / C::kSlots) & 1u, abort_flag, g.status);
        if (!ok) break;
        const float* sc = reinterpret_cast<const float*>(smem + C::kScaleOff + slot * C::kScales);
        const int b = group * kAccs + n % kAccs;
        ok = warp_wait(tfull(b), static_cast<uint32_t>(n / kAccs) & 1u, abort_flag, g.status);
        if (!ok) break;
        tc_fence_after();
        auto release = [&] {  // the accumulator has been read whole: the MMAs may write it again
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(tempty(b), 0));
        };
        // chunks, the next one on its way while this one is added
        if constexpr (COLVEC) {
          // a thread holds 4 rows x HB / 4 columns, so that it needs few of the column scales (all of them, for a row per
          // thread, are 1024 cycles of shared memory per block: 8192 x 8192 x 8192 588 us)
          constexpr int kW = HB % 64 == 0 ? 64 : 32, kChunks = 2 * HB / kW;  // 16 lanes x kW columns, lanes first
          uint32_t v[2][kW / 2];
          const float* cs = sc + 128 + h * HB + (lane & 3) * 2;
          float rs[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) rs[i] = sc[q * 32 + (lane >> 2) + 8 * i];
          auto load = [&](int i, uint32_t(&x)[kW / 2]) {
            const uint32_t at = lanes + (static_cast<uint32_t>(i & 1) * 16u << 16) + b * BN + (i >> 1) * kW;
            if constexpr (kW == 64) tmem_ld_16x256b_x8(at, x);
            else tmem_ld_16x256b_x4(at, x);
          };
          load(0, v[0]);
          float2 y[kW / 8];
#pragma unroll
          for (int i = 0; i < kChunks; ++i) {
            if (!(i & 1)) {
#pragma unroll
              for (int k = 0; k < kW / 8; ++k) y[k] = *reinterpret_cast<const float2*>(cs + (i >> 1) * kW + k * 8);
            }
            uint32_t(&x)[kW / 2] = v[i & 1];
            tmem_ld_wait_for(x);
            if (i + 1 < kChunks) load(i + 1, v[(i + 1) & 1]);
            else release();
#pragma unroll
            for (int k = 0; k < kW / 8; ++k)
#pragma unroll
              for (int o = 0; o < 2; ++o) {
                float f0, f1;
                const float s = rs[(i & 1) * 2 + o];
                mul_f32x2(f0, f1, s, s, y[k].x, y[k].y);
                const int at = i * (kW / 2) + k * 4 + o * 2;
                fma_f32x2(acc[at], acc[at + 1], __uint_as_float(x[k * 4 + o * 2]), __uint_as_float(x[k * 4 + o * 2 + 1]), f0, f1,
                          acc[at], acc[at + 1]);
              }
          }
        } else {
          const float s = sc[q * 32 + lane] * __shfl_sync(0xffffffffu, q_now, kb % 32);
          uint32_t v[2][32];
          tmem_ld_32x32b_x32(lanes + b * BN, v[0]);
#pragma unroll
          for (int c = 0; c < HB; c += 32) {
            uint32_t(&x)[32] = v[c / 32 & 1];
            tmem_ld_wait_for(x);
            if (c + 32 < HB) tmem_ld_32x32b_x32(lanes + b * BN + c + 32, v[(c / 32 + 1) & 1]);
            else release();
#pragma unroll
            for (int j = 0; j < 32; j += 2)
              fma_f32x2(acc[c + j], acc[c + j + 1], __uint_as_float(x[j]), __uint_as_float(x[j + 1]), s, s, acc[c + j],
                        acc[c + j + 1]);
          }
        }
      }
      if (!ok) break;
      // The tile's 32 rows of this warp.  Where all of them are there: through shared memory, a box of 32 rows x 128 bytes
      // at a time (in the 128-byte TMA swizzle: 16-byte chunk k of row r at k ^ (r & 7); bf16 boxes of 32 columns in the 64-byte
      // one, k ^ (r >> 1 & 3)); else straight from the registers.
      const int row0 = w.row0 + rank * 128 + q * 32;
      if (row0 >= w.row_end) continue;
      const bool boxes = row0 + 32 <= w.row_end;
      auto bf16_at = [&](int r, int k) {  // chunk k of row r
        return static_cast<uint32_t>(C::kBox == 64 ? r * 128 + ((k ^ (r & 7)) << 4) : r * 64 + ((k ^ (r >> 1 & 3)) << 4));
      };
      auto begin = [&] {
        if (lane == 0) bulk_wait_read<C::kBoxes - 1>();  // what was stored from here before has been read
        __syncwarp();
      };
      auto send = [&](int c0) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&t.out, stage, c0, row0);
          bulk_commit();
        }
        if (C::kBoxes == 2) stage = 2 * stage0 + 4096 - stage;
      };
      if constexpr (COLVEC) {
        const int fr = lane >> 2, fc = lane & 3;  // row of the thread's first; its pair of columns in 8
        constexpr int kW = HB % 64 == 0 ? 64 : 32;
        auto value = [&](int c, int o) {  // the thread's pair of columns in the 8 from c on, row fr + 8 o
          return &acc[(c / kW * 2 + (o >> 1)) * (kW / 2) + c % kW / 8 * 4 + (o & 1) * 2];
        };
        if (boxes && !g.out_f32) {
#pragma unroll
          for (int i = 0; i < HB; i += C::kBox) {
            if (j0 + i >= g.q_rows) continue;
            begin();
#pragma unroll
            for (int o = 0; o < 4; ++o)
#pragma unroll
              for (int k = 0; k < C::kBox / 8; ++k) {
                const float* x = value(i + k * 8, o);
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(stage + bf16_at(fr + 8 * o, k) + fc * 4),
                             "r"(pack_bf16x2(x[0], x[1]))
                             : "memory");
              }
            send(j0 + i);
          }
        } else if (boxes) {
#pragma unroll
          for (int i = 0; i < HB; i += 32) {
            if (j0 + i >= g.q_rows) continue;
            begin();
#pragma unroll
            for (int o = 0; o < 4; ++o)
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float* x = value(i + k * 8, o);
                const int r = fr + 8 * o;
                asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(
                                 stage + static_cast<uint32_t>(r * 128 + ((k * 2 + (fc >> 1)) ^ (r & 7)) * 16 + (fc & 1) * 8)),
                             "f"(x[0]), "f"(x[1])
                             : "memory");
              }
            send(j0 + i);
          }
        } else {
#pragma unroll
          for (int i = 0; i < HB; i += 8)
#pragma unroll
            for (int o = 0; o < 4; ++o) {
              const int row = row0 + fr + 8 * o, col = j0 + i + fc * 2;
              if (row >= w.row_end || col >= g.q_rows) continue;
              const float* x = value(i, o);
              const int64_t at = static_cast<int64_t>(row) * g.ldo + col;
              if (g.out_f32) *reinterpret_cast<float2*>(static_cast<float*>(g.out) + at) = make_float2(x[0], x[1]);
              else *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(g.out) + at) = pack_bf16x2(x[0], x[1]);
            }
        }
      } else if (boxes) {
        if (!g.out_f32) {
#pragma unroll
          for (int c = 0; c < HB; c += C::kBox) {
            if (j0 + c >= g.q_rows) continue;
            begin();
#pragma unroll
            for (int k = 0; k < C::kBox / 8; ++k) {
              const float* x = &acc[c + 8 * k];
              st_shared_v4(stage + bf16_at(lane, k), make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]),
                                                                pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])));
            }
            send(j0 + c);
          }
        } else {
#pragma unroll
          for (int c = 0; c < HB; c += 32) {
            if (j0 + c >= g.q_rows) continue;
            begin();
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float* x = &acc[c + 4 * k];
              st_shared_v4(stage + static_cast<uint32_t>(lane * 128 + ((k ^ (lane & 7)) << 4)),
                           make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])));
            }
            send(j0 + c);
          }
        }
      } else if (row0 + lane < w.row_end) {
        const int64_t at = static_cast<int64_t>(row0 + lane) * g.ldo + j0;
        if (g.out_f32) {
          float* o = static_cast<float*>(g.out) + at;
#pragma unroll
          for (int j = 0; j < HB; j += 4)
            if (j0 + j < g.q_rows) *reinterpret_cast<float4*>(o + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        } else {
          uint16_t* o = static_cast<uint16_t*>(g.out) + at;
#pragma unroll
          for (int j = 0; j < HB; j += 8)
            if (j0 + j < g.q_rows)
              *reinterpret_cast<uint4*>(o + j) =
                  make_uint4(pack_bf16x2(acc[j], acc[j + 1]), pack_bf16x2(acc[j + 2], acc[j + 3]),
                             pack_bf16x2(acc[j + 4], acc[j + 5]), pack_bf16x2(acc[j + 6], acc[j + 7]));
        }
      }
      __syncwarp();
    }
    if (lane == 0) bulk_wait_read<0>();  // the staging has been read; the grid's end waits for the writes
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
    tmem_dealloc_pair(tmem, 512);
  }
}

template <int BN, bool COLVEC, bool ALT>
int launch_pair(const PairMaps& maps, const PairArgs& a, int kind, cudaStream_t stream) {
  using C = Cfg<BN, COLVEC, ALT>;
  static DeviceOnce once;
  const int se = once.run([](int* d) { return static_cast<int>(cudaGetDevice(d)); },
                          [] {
                            // what setmaxnreg hands round must be what the launch has: a wait for more would not end
                            cudaFuncAttributes f;
                            const cudaError_t e = cudaFuncGetAttributes(&f, fp8_pair_kernel<BN, COLVEC, ALT>);
                            if (e != cudaSuccess) return static_cast<int>(e);
                            if (f.numRegs * kThreads < 128 * C::kLow + 256 * C::kHigh)
                              return static_cast<int>(cudaErrorInvalidConfiguration);
                            return static_cast<int>(cudaFuncSetAttribute(fp8_pair_kernel<BN, COLVEC, ALT>,
                                                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                         static_cast<int>(C::kSmem)));
                          },
                          static_cast<int>(cudaErrorInvalidDevice));
  if (se) return se;
  trace_begin(stream, kind);
  const cudaError_t e = launch_pdl(fp8_pair_kernel<BN, COLVEC, ALT>, dim3(2 * a.pairs), dim3(kThreads), C::kSmem, stream, maps, a);
  trace_end(stream);
  return static_cast<int>(e);
}

template <int BN, bool ALT = false>
int pair_width(const Fp8Operand& p, const Fp8Operand& q, PairArgs a, int64_t out_rows, int kind, cudaStream_t stream) {
  Fp8Problem& g = a.g;
  g.q_tiles = static_cast<int32_t>((q.rows + BN - 1) / BN);
  int64_t units = static_cast<int64_t>(g.p_tiles) * g.q_tiles * (g.mode == FP8_WGRAD ? g.experts : 1);
  if (units == 0) return 0;
  if (units >= (int64_t{1} << 30)) return static_cast<int>(cudaErrorInvalidValue);
  a.units = static_cast<int32_t>(units);
  if (units < a.pairs) a.pairs = static_cast<int32_t>(units);
  PairMaps m;
  const uint64_t N = static_cast<uint64_t>(q.rows), R = static_cast<uint64_t>(out_rows);
  const bool good =
      make_tmap_fp8(&m.p, p.q, static_cast<uint64_t>(p.cols), static_cast<uint64_t>(p.rows), static_cast<uint64_t>(p.ld), 128) &&
      make_tmap_fp8(&m.q, q.q, static_cast<uint64_t>(q.cols), static_cast<uint64_t>(q.rows) * q.batch,
                    static_cast<uint64_t>(q.ld), BN / 2) &&
      (g.out_f32      ? make_tmap_f32(&m.out, g.out, N, R, 32, 32)
       : BN / 2 % 64 ? make_tmap_bf16_sw64(&m.out, g.out, N, R, 32, 32)
                     : make_tmap_bf16(&m.out, g.out, N, R, 64, 32));
  if (!good) return static_cast<int>(cudaErrorInvalidValue);
  if constexpr (BN != 192 && !ALT) {
    if (!q.row_scales) return launch_pair<BN, false, false>(m, a, kind, stream);
  }
  return launch_pair<BN, true, ALT>(m, a, kind, stream);
}

}  // namespace

int launch_fp8_pair(const Fp8Operand& p, const Fp8Operand& q, Fp8Problem g, int64_t row_units, int kind, cudaStream_t stream) {
  const int pairs = sm_count() / 2;
  if (pairs <= 0) return static_cast<int>(cudaErrorInvalidDevice);
  g.sp = p.s;
  g.p_pitch = fp8_pitch(p.rows);
  g.p_rows = static_cast<int32_t>(p.rows);
  g.sq = q.s;
  g.q_pitch = fp8_pitch(q.rows);
  g.q_batch = fp8_blocks(q.rows) * g.k_blocks;
  g.q_rows = static_cast<int32_t>(q.rows);
  g.p_tiles = static_cast<int32_t>(g.mode == FP8_GROUPED ? row_units : (p.rows + 255) / 256);
  PairArgs a{};
  a.g = g;
  a.pairs = pairs;
  const int64_t mats = g.mode == FP8_WGRAD ? g.experts : 1;
  const int64_t out_rows = p.rows * mats;
  // The tile width whose rounds of tiles take least.  A round takes its K blocks and what its output adds; with outputs beyond L2
  // at least its bytes at the rate at which they were seen to leave.  (192 columns in row-scaled products only: with a scale per
  // 128 x 128 values a block takes 420 ns of 192, hardly less than of 256.)  A schedule's rows count as spread evenly, a
  // weight gradient's K likewise.
  auto rounds = [&](int bn) {
    return (static_cast<int64_t>(g.p_tiles) * ((q.rows + bn - 1) / bn) * mats + pairs - 1) / pairs;
  };
  if (!q.row_scales) {
    if (rounds(256) * (g.k_blocks * int64_t{450} + 1000) <= rounds(128) * (g.k_blocks * int64_t{310} + 1000))
      return pair_width<256>(p, q, a, out_rows, kind, stream);
    return pair_width<128>(p, q, a, out_rows, kind, stream);
  }
  // Row-scaled, us of 256, 192 and 128 columns, and of 128 in turn (ALT), fp32 output (bf16 output); the weight gradients are 64
  // experts' of 1024 x 2048, their rows per expert:
  //   1536 x 4096 over 8192         84.3        70.3        82.9       105
  //   4096 x 4096 over 512          24.0 (19.0) 24.1 (20.1) 22.4 (19.4) 19.4 (17.7)
  //   4096 x 4096 over 2048         52.3 (47.0) 52.9 (49.2) 56.4 (52.4) 62.7 (61.4)
  //   1000 x 2056 over 1003         11.2        9.8         8.4        9.5
  //   weight gradient, 96 rows      102 (53)    105 (66)    98 (69)    106 (53)
  //   weight gradient, 384 rows     139 (106)   154 (123)   139 (121)  112 (96)
  //   weight gradient, 768 rows     184 (151)   209 (176)   222 (186)  184 (180)
  const int64_t esize = g.out_f32 ? 4 : 2;
  const bool beyond_l2 = out_rows * q.rows * esize > (int64_t{1} << 27);
  auto cost = [&](int bn, int64_t ns, int64_t out_ns, int64_t gbs) {
    const int64_t blocks = g.mode == FP8_WGRAD ? ns * g.k_blocks / g.experts - ns / 2 : ns * g.k_blocks;
    const int64_t least = beyond_l2 ? 256 * bn * esize * pairs / gbs : 0;
    return rounds(bn) * (blocks + out_ns > least ? blocks + out_ns : least);
  };
  const bool f32 = g.out_f32;
  const int64_t c256 = cost(256, 615, f32 ? 2800 : 1600, 5200), c192 = cost(192, 505, f32 ? 2300 : 1300, 5200),
                c128 = cost(128, 400, f32 ? 1400 : 800, 5200), alt = cost(128, 520, f32 ? 300 : 0, 4800) + 1500;
  const int64_t others = c256 < c192 ? (c256 < c128 ? c256 : c128) : (c192 < c128 ? c192 : c128);
  if (alt < others) return pair_width<128, true>(p, q, a, out_rows, kind, stream);
  if (c256 == others) return pair_width<256>(p, q, a, out_rows, kind, stream);
  if (c192 == others) return pair_width<192>(p, q, a, out_rows, kind, stream);
  return pair_width<128>(p, q, a, out_rows, kind, stream);
}

}  // namespace mok
