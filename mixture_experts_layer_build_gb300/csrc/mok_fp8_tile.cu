// mok_fp8_tile.cu -- 8-bit products with a scale per 128 values, one 128 x BN tile per CTA.
//
// With P = b, whose rows are the accumulator's 128 lanes, and Q = a, whose rows are its BN columns, a CTA computes out[j, i] =
// sum over K blocks of sq[j] sp[i] (Q[j, :] . P[i, :]): few rows of a take few columns, and the weights' bytes bound it.  A
// K block is 128 bytes of a row, one
// swizzle atom: four tcgen05.mma (M = 128, K = 32) into a TMEM accumulator of its own, one of four or eight in turn, which four
// warps then drain, scale and add into their registers.  Row scales come to shared memory in lots of 16 K blocks, the next
// lot on its way while one is used (fetched block by block, their latency set the pace: 1.6 us per block, one row at N =
// 2048, K = 7168 14 us).
//
// XQ: a is bf16 and quantised on the way, by four more warps, each K block's rows by one of them, straight into the stage's
// swizzled shared memory: a launch less, and its latency under the weights'.
//
// With few tiles their K range is split over a cluster, whose CTAs add up their partials through shared memory in rank
// order.  Up to 32 columns two CTAs share an SM: clusters of eight, of which 15 fit at one CTA per SM, then fit twice as often.
//
// The weights' bytes and the latencies of a start, a load, a chain of K blocks and a reduction bound it.  Measured: one row at
// N = 2048, K = 7168 6.1 us with its quantisation (14.7 MB: 2.2), 61 rows at N = 7168, K = 2048 7.0, 128 rows 8.9; one token's eight
// experts of 1536 x 4096 9.2 us (50 MB: 7.4); 128 experts of them with 8 rows each 125 (119).
#include "mok_ffn.cuh"  // warp_wait, wait_landed, elect_one
#include "mok_fp8.cuh"
#include "mok_fp8_gemm.cuh"

namespace mok {
namespace {

constexpr int kThreads = 192, kThreadsXq = 320;
constexpr int kSlots = 24;  // (XQ) K blocks whose column scales are kept: stages + accumulators + 1 at least
constexpr int kMaxStages = 12;
constexpr uint32_t kHalfSmem = 114688;  // two CTAs
constexpr uint32_t kMaxSmem = 227328;  // dynamic: 5 KB of 227 KB are left for what is static

constexpr int kLot = 16;  // K blocks whose scales are fetched together

struct TileArgs {
  Fp8Problem g;
  int32_t split;   // CTAs of a cluster that share a tile's K range 
  int32_t stages;
  uint32_t scale_off, push_off;
  const uint16_t* x;  // (XQ) a's values
  int32_t K;
};

template <int BN, bool PVEC, bool XQ>
struct Cfg {
  static_assert(!(PVEC && XQ), "a forward's weights have scales per 128 x 128 values");
  static constexpr uint32_t kStage = 16384 + BN * 128;
  static constexpr int kAccs = BN <= 32 ? 8 : 4;
  static constexpr int kPerSm = BN <= 32 ? 2 : 1;  // CTAs of an SM
  static constexpr uint32_t kRows = PVEC ? 128 : 0;  // of P with a scale each
  static constexpr uint32_t kLotBytes = kLot * (kRows + BN) * 4;
  static constexpr uint32_t kScaleBytes = XQ ? kSlots * BN * 4 : 2 * kLotBytes;
};

// 32 or 16 columns of this lane's accumulator row.
template <int W>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[W]) {
  if constexpr (W == 32) {
    tmem_ld_32x32b_x32(taddr, r);
  } else {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr));
  }
}

// A tile: where its operands' rows start, the output's rows and columns it holds, its K blocks.
struct Tile {
  int32_t p0, q0;        // rows of P and Q in their tensor maps
  int32_t i0, j0;        // output column and row
  int32_t i_end, j_end;
  int32_t count;         // K blocks
  int32_t batch;         // of BLOCKS-scaled operands
};

__device__ __forceinline__ bool fp8_tile(const Fp8Problem& g, int u, int bn, Tile& t) {
  t.count = g.k_blocks;
  t.batch = 0;
  const int pt = u % g.p_tiles;
  const int rest = u / g.p_tiles;
  if (g.mode == FP8_DENSE) {
    t.p0 = t.i0 = pt * 128;
    t.q0 = t.j0 = rest * bn;
    t.i_end = g.p_rows;
    t.j_end = g.q_rows;
    return true;
  }
  // one 128-row block of an expert's rows, against a tile of its weights
  const int blocks = __ldg(g.meta + 2);  // (both loads at once: the table has an entry for every CTA of the grid)
  const int4 b = __ldg(reinterpret_cast<const int4*>(g.mblocks) + rest);  // {expert, first row, valid rows, tile}
  if (rest >= blocks) return false;
  t.batch = b.x;
  t.i0 = pt * 128;
  t.p0 = b.x * g.p_rows + t.i0;
  t.i_end = g.p_rows;
  t.q0 = t.j0 = b.y;
  t.j_end = b.y + b.z;
  return true;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// This thread's row r of the accumulator to the CTAs of a cluster of S that own its columns.
template <int BN, int S>
__device__ __forceinline__ void push_partials(uint32_t push, const float (&acc)[BN], int rank, int r) {
  constexpr int kPer = BN / S;
#pragma unroll
  for (int own = 0; own < S; ++own) {
    const uint32_t local = push + static_cast<uint32_t>(rank * kPer * 128 + r) * 4u;
    const uint32_t to = S > 1 ? mapa_shared(local, own) : local;
#pragma unroll
    for (int jj = 0; jj < kPer; ++jj) {
      if constexpr (S > 1)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(to + jj * 512), "f"(acc[own * kPer + jj]) : "memory");
      else
        asm volatile("st.shared.f32 [%0], %1;" ::"r"(to + jj * 512), "f"(acc[jj]) : "memory");
    }
  }
}

template <int BN, bool PVEC, bool XQ>
__global__ void __launch_bounds__(XQ ? kThreadsXq : kThreads, Cfg<BN, PVEC, XQ>::kPerSm)
    fp8_tile_kernel(const __grid_constant__ CUtensorMap tP, const __grid_constant__ CUtensorMap tQ, const TileArgs a) {
  using C = Cfg<BN, PVEC, XQ>;
  constexpr uint32_t kTx = 16384 + (XQ ? 0 : BN * 128), kStage = C::kStage, kCols = C::kAccs * BN;
  constexpr int kAccs = C::kAccs;
  constexpr int W = BN < 32 ? 16 : 32;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 17 + (XQ ? kSlots : 0)];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  const Fp8Problem& g = a.g;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull = [&](int b) { return bar0 + 8u * (2 * kMaxStages + b); };
  auto tempty = [&](int b) { return bar0 + 8u * (2 * kMaxStages + kAccs + b); };
  const uint32_t done = bar0 + 8u * (2 * kMaxStages + 2 * kAccs);
  auto qfull = [&](int i) { return done + 8u * (1 + i); };  // (XQ) the block's column scales are there
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = a.split;
  const int rank = static_cast<int>(blockIdx.x) % S, unit = static_cast<int>(blockIdx.x) / S;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full(s), XQ ? 2 : 1);  // the loads; (XQ) the warp that quantised the block
      mbar_init(empty(s), 1);
    }
    if (XQ)
      for (int i = 0; i < kSlots; ++i) mbar_init(qfull(i), 1);
    for (int b = 0; b < kAccs; ++b) {
      mbar_init(tfull(b), 1);
      mbar_init(tempty(b), 4);
    }
    mbar_init(done, 1);
    abort_word = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_slot), kCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  if (S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA has started
  if (g.mode != FP8_DENSE) pdl_wait();  // the schedule's tables
  Tile t;
  const bool have = fp8_tile(g, unit, BN, t);
  const int subs = !have ? 0 : (min(t.j_end - t.j0, g.mode == FP8_DENSE ? BN : 128) + BN - 1) / BN;
  // this CTA's share of the K blocks
  const int kb0 = static_cast<int>(static_cast<int64_t>(t.count) * rank / S);
  const int count = static_cast<int>(static_cast<int64_t>(t.count) * (rank + 1) / S) - kb0;
  const int total = subs * count;  // K blocks that pass through the stages
  if (S > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  bool ok = true;
  int ahead = 0;  // (warp 0) K blocks of P that were loaded early
  if (warp == 0 && g.early_p) {  // weights: nothing that still runs writes them
    ahead = min(total, a.stages);
    for (int n = 0; n < ahead; ++n)
      if (elect_one()) {
        mbar_arrive_expect_tx(full(n), kTx);
        tma_load_2d(base + n * kStage, &tP, full(n), (kb0 + n % count) * 128, t.p0);
      }
  }
  pdl_wait();  // (the kernel in front may take its time: no bounded wait starts before its end)
  pdl_trigger();
  const int q = warp & 3, r = q * 32 + lane;  // (warps 2 to 5) TMEM lane quarter; the lane's row
  const uint32_t lanes = tmem + (static_cast<uint32_t>(q * 32) << 16);
  int n = 0, st = 0;     // K blocks so far; (warps 0 and 1) the next one's stage
  uint32_t ph = 0;       // parity of the stage's round
  // The roles take the sub-tiles in step where a cluster's barriers separate them; without a split each runs ahead of
  // the next as far as stages and accumulators go.
  for (int sub = 0; sub < subs; ++sub) {
    float acc[BN];
    if (warp == 0) {
      for (int kb = 0; kb < count && ok; ++kb) {
        if (n >= a.stages && !warp_wait(empty(st), ph ^ 1u, abort_flag, g.status)) {
          ok = false;
          break;
        }
        const uint32_t sp = base + st * kStage;
        if (elect_one()) {
          if (n >= ahead) {
            mbar_arrive_expect_tx(full(st), kTx);
            tma_load_2d(sp, &tP, full(st), (kb0 + kb) * 128, t.p0);
          }
          if (!XQ) tma_load_2d(sp + 16384, &tQ, full(st), (kb0 + kb) * 128, t.q0 + sub * BN);
        }
        ++n;
        if (++st == a.stages) {
          st = 0;
          ph ^= 1u;
        }
      }
    } else if (warp == 1) {
      for (int kb = 0; kb < count && ok; ++kb, ++n) {
        const int b = n % kAccs;
        ok = (n < kAccs || warp_wait(tempty(b), static_cast<uint32_t>(n / kAccs - 1) & 1u, abort_flag, g.status)) &&
             warp_wait(full(st), ph, abort_flag, g.status);
        if (!ok) break;
        tc_fence_after();
        const uint32_t sp = base + st * kStage;
        const uint64_t pd = sdesc_sw128(sp, 16, 1024), qd = sdesc_sw128(sp + 16384, 16, 1024);
        if (elect_one()) {
#pragma unroll
          for (int ks = 0; ks < 4; ++ks)  // 32 bytes of K; descriptors count 16-byte units
            umma_fp8(tmem + b * BN, pd + ks * 2, qd + ks * 2, idesc_fp8(128, BN), ks > 0 ? 1u : 0u);
          umma_commit(empty(st));
          umma_commit(tfull(b));
        }
        if (++st == a.stages) {
          st = 0;
          ph ^= 1u;
        }
      }
    } else if (XQ && warp >= 6) {
      // K blocks warp - 6, + 4, ...: two rows at a time, 16 lanes x 8 columns each, the next rows on their way
      const int rows = t.j_end - t.j0, half = lane >> 4, c = (lane & 15) * 8;
      for (int kb = warp - 6; kb < count && ok; kb += 4) {
        const int slot = kb % kSlots, at = kb % a.stages, col = (kb0 + kb) * 128 + c;
        auto load = [&](int r) {
          return r < rows && col < a.K
                     ? __ldg(reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(t.j0 + r) * a.K + col))
                     : make_uint4(0, 0, 0, 0);
        };
        uint4 v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = load(2 * i + half);
        if (kb >= a.stages) ok = warp_wait(empty(at), static_cast<uint32_t>(kb / a.stages - 1) & 1u, abort_flag, g.status);
        if (!ok) break;
        const uint32_t to = base + at * kStage + 16384;
        float* sc = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)) + a.scale_off) + slot * BN;
        for (int r0 = 0; r0 < rows; r0 += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = r0 + 2 * i + half;
            const uint4 w = v[i];
            v[i] = load(r + 8);
            uint32_t m = absmax2(absmax2(w.x, w.y), absmax2(w.z, w.w));
#pragma unroll
            for (int d = 8; d >= 1; d >>= 1) m = absmax2(m, __shfl_xor_sync(0xffffffffu, m, d));
            m = absmax2(m, m >> 16) & 0x7FFFu;
            float up;
            const float scale = fp8_scale(m, up);
            uint2 o = make_uint2(fp8_codes(w.x, up) | fp8_codes(w.y, up) << 16, fp8_codes(w.z, up) | fp8_codes(w.w, up) << 16);
            if (m >= 0x7F80u) o = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
            if (r < rows) {  // 16-byte chunk k of row r at k ^ (r & 7); the rows past the last one's columns are not stored
              asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(to + static_cast<uint32_t>(r * 128 + (((c >> 4) ^ (r & 7)) << 4) + (c & 8))),
                           "r"(o.x), "r"(o.y)
                           : "memory");
              if ((lane & 15) == 0) sc[r] = scale;
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(full(at));
          mbar_arrive(qfull(slot));
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < BN; ++j) acc[j] = 0.0f;
      const int j0 = t.j0 + sub * BN;
      // 16-byte pieces of a lot's row scales (their rows are padded to four); what lies past the matrix is not used
      const int tid = static_cast<int>(threadIdx.x) - 64;
      [[maybe_unused]] auto fetch = [&](int lot) {
        const uint32_t to = base + a.scale_off + (lot & 1) * C::kLotBytes;
        const int k0 = kb0 + lot * kLot, blocks = min(kLot, count - lot * kLot);
        if constexpr (PVEC) {
          for (int x = tid; x < blocks * 32; x += 128) {
            const int k = x >> 5, i = (x & 31) * 4;
            if (t.i0 + i < g.p_pitch)
              cp_async16(to + (k * 128 + i) * 4, g.sp + static_cast<int64_t>(k0 + k) * g.p_pitch + t.i0 + i);
          }
        }
        for (int x = tid; x < blocks * (BN / 4); x += 128) {
          const int k = x / (BN / 4), j = (x % (BN / 4)) * 4;
          if (j0 + j < g.q_pitch)
            cp_async16(to + kLot * C::kRows * 4 + (k * BN + j) * 4, g.sq + static_cast<int64_t>(k0 + k) * g.q_pitch + j0 + j);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      // scales of 128 x 128 values: a lot's, a lane each
      const float* ps = g.sp + t.batch * g.p_batch + static_cast<int64_t>(t.i0 / 128) * g.k_blocks + kb0;
      auto block_scales = [&](int lot) {
        const int k = lot * kLot + (lane & (kLot - 1));
        return k < count ? __ldg(ps + k) : 0.0f;
      };
      if constexpr (!XQ) {
        asm volatile("bar.sync 1, 128;" ::: "memory");  // the lots of the sub-tile before have been used
        if (count > 0) fetch(0);
      }
      float s_now = 0.0f, s_next = PVEC ? 0.0f : block_scales(0);
      for (int kb = 0; kb < count; ++kb, ++n) {  // (also after a failed wait: the barriers count every warp)
        const int b = n % kAccs, lot = kb / kLot, in = kb % kLot;
        if (in == 0) {
          if constexpr (!XQ) {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            asm volatile("bar.sync 1, 128;" ::: "memory");  // everybody's pieces are there, and the other lot has been used
            if (kb + kLot < count) fetch(lot + 1);
          }
          s_now = s_next;
          if (!PVEC) s_next = block_scales(lot + 1);
        }
        const float* lots = reinterpret_cast<const float*>(smem_raw + (base - smem_u32(smem_raw)) + a.scale_off);
        if constexpr (!XQ) lots += (lot & 1) * (C::kLotBytes / 4);
        const float* cs = XQ ? lots + kb % kSlots * BN : lots + kLot * C::kRows + in * BN;
        const float s = PVEC ? lots[in * 128 + r] : __shfl_sync(0xffffffffu, s_now, in);
        if constexpr (XQ) ok = ok && warp_wait(qfull(kb % kSlots), static_cast<uint32_t>(kb / kSlots) & 1u, abort_flag, g.status);
        ok = ok && warp_wait(tfull(b), static_cast<uint32_t>(n / kAccs) & 1u, abort_flag, g.status);
        if (!ok) continue;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < BN; c += W) {
          uint32_t v[W];
          tmem_ld<W>(lanes + b * BN + c, v);
          tmem_ld_wait();
          if (c + W == BN) {  // read whole: the MMAs may write it again
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(tempty(b));
          }
#pragma unroll
          for (int j = 0; j < W; j += 4) {
            const float4 x = *reinterpret_cast<const float4*>(cs + c + j);
            float f0, f1, f2, f3;
            mul_f32x2(f0, f1, s, s, x.x, x.y);
            mul_f32x2(f2, f3, s, s, x.z, x.w);
            fma_f32x2(acc[c + j], acc[c + j + 1], __uint_as_float(v[j]), __uint_as_float(v[j + 1]), f0, f1, acc[c + j],
                      acc[c + j + 1]);
            fma_f32x2(acc[c + j + 2], acc[c + j + 3], __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]), f2, f3,
                      acc[c + j + 2], acc[c + j + 3]);
          }
        }
      }
    }
    const bool drains = warp >= 2 && warp < 6;
    const int j0 = t.j0 + sub * BN;
    // Column j belongs to CTA j / (BN / S) of the cluster: each sends it its partials, [source][column][row], and the owner
    // adds them in rank order, 8 rows of a column per thread: 16 bytes of a row of the output.
    const uint32_t push = base + a.push_off;
    if (drains) {
      if (S == 1) push_partials<BN, 1>(push, acc, rank, r);
      else if (S == 2) push_partials<BN, 2>(push, acc, rank, r);
      else if (S == 4) push_partials<BN, 4>(push, acc, rank, r);
      else push_partials<BN, 8>(push, acc, rank, r);
    }
    __syncwarp();
    if (S > 1) cluster_sync();
    else if (drains) asm volatile("bar.sync 1, 128;" ::: "memory");
    if (drains && *abort_flag == 0) {
      const int per = BN / S;
      const float* parts = reinterpret_cast<const float*>(smem_raw + (push - smem_u32(smem_raw)));
      for (int x = static_cast<int>(threadIdx.x) - 64; x < per * 16; x += 128) {
        const int jj = x >> 4, i = (x & 15) * 8, j = j0 + rank * per + jj;
        if (t.i0 + i >= t.i_end || j >= t.j_end) continue;
        float4 lo = make_float4(0, 0, 0, 0), hi = lo;
        for (int c = 0; c < S; ++c) {
          const float4* p = reinterpret_cast<const float4*>(parts + (c * per + jj) * 128 + i);
          const float4 y = p[0], z = p[1];
          lo.x += y.x, lo.y += y.y, lo.z += y.z, lo.w += y.w, hi.x += z.x, hi.y += z.y, hi.z += z.z, hi.w += z.w;
        }
        const int64_t at = static_cast<int64_t>(j) * g.ldo + t.i0 + i;
        if (g.out_f32) {
          float4* o = reinterpret_cast<float4*>(static_cast<float*>(g.out) + at);
          o[0] = lo;
          o[1] = hi;
        } else {
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(g.out) + at) =
              make_uint4(pack_bf16x2(lo.x, lo.y), pack_bf16x2(lo.z, lo.w), pack_bf16x2(hi.x, hi.y), pack_bf16x2(hi.z, hi.w));
        }
      }
    }
    __syncwarp();
    if (S > 1 && sub + 1 < subs) cluster_sync();  // the partials have been read (without a split: bar.sync above)
  }
  __syncwarp();
  if (warp == 0 && *abort_flag && lane == 0)  // let the copies in flight land: the last one of each stage
    for (int b = n > a.stages ? n - a.stages : 0; b < n; ++b)
      wait_landed(full(b % a.stages), static_cast<uint32_t>(b / a.stages) & 1u);
  if (warp == 1) {
    if (elect_one()) umma_commit(done);  // also after an abort: what was issued completes before TMEM is freed
    __syncwarp();
    if (lane == 0) wait_landed(done, 0);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
}

template <int BN, bool PVEC, bool XQ>
int launch_tile(const CUtensorMap& tP, const CUtensorMap& tQ, const Fp8Problem& g, int64_t units, int split, const void* x,
                int64_t K, int kind, cudaStream_t stream) {
  static DeviceOnce once;
  const int se = once.run([](int* d) { return static_cast<int>(cudaGetDevice(d)); },
                          [] {
                            return static_cast<int>(cudaFuncSetAttribute(fp8_tile_kernel<BN, PVEC, XQ>,
                                                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                         static_cast<int>(kMaxSmem)));
                          },
                          static_cast<int>(cudaErrorInvalidDevice));
  if (se) return se;
  if (units * split >= (int64_t{1} << 31)) return static_cast<int>(cudaErrorInvalidValue);
  using C = Cfg<BN, PVEC, XQ>;
  constexpr uint32_t kStage = C::kStage;
  TileArgs a{};
  a.g = g;
  a.x = static_cast<const uint16_t*>(x);
  a.K = static_cast<int32_t>(K);
  a.split = split;
  constexpr uint32_t push = BN * 512u;
  static_assert(!XQ || kSlots > kMaxStages + C::kAccs, "scales stay until they are used");
  constexpr uint32_t fixed = 1024u + C::kScaleBytes + push;  // alignment; scales; partials
  a.stages = static_cast<int32_t>(((C::kPerSm == 2 ? kHalfSmem : kMaxSmem) - fixed) / kStage);
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  a.scale_off = static_cast<uint32_t>(a.stages) * kStage;
  a.push_off = a.scale_off + C::kScaleBytes;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * split));
  cfg.blockDim = dim3(XQ ? kThreadsXq : kThreads);
  cfg.dynamicSmemBytes = a.push_off + push + 1024u;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  trace_begin(stream, kind);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_tile_kernel<BN, PVEC, XQ>, tP, tQ, a);
  trace_end(stream);
  return static_cast<int>(e);
}

}  // namespace

int launch_fp8_tile(const Fp8Operand& a, const void* x, const Fp8Operand& b, Fp8Problem g, int64_t rows, int64_t row_blocks,
                    int kind, cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return static_cast<int>(cudaErrorInvalidDevice);
  const bool grouped = g.mode == FP8_GROUPED;
  g.sp = b.s;
  g.p_pitch = fp8_pitch(b.rows);
  g.p_batch = fp8_blocks(b.rows) * g.k_blocks;
  g.p_rows = static_cast<int32_t>(b.rows);
  g.sq = a.s;
  g.q_pitch = fp8_pitch(a.rows);
  g.q_rows = static_cast<int32_t>(a.rows);
  // Columns for the rows of a block.  A schedule's blocks get twice their average (one with more takes its weights twice: 128
  // experts with 16 rows on average, K = 4096, N = 1536 177 us with 16 columns, 131 with 32), but 64 only from 24 rows on,
  // where an SM has one CTA (64 experts with 24 rows, K = 2048, N = 1024 43 us with 64, 35 with 32).
  const int64_t per = grouped ? 2 * rows / (row_blocks > 0 ? row_blocks : 1) : rows;
  const int bn = per <= 16 ? 16 : per <= (grouped ? 48 : 32) ? 32 : per <= 64 ? 64 : 128;
  g.p_tiles = static_cast<int32_t>(fp8_blocks(b.rows));
  g.q_tiles = static_cast<int32_t>(grouped ? row_blocks : (rows + bn - 1) / bn);
  const int64_t units = static_cast<int64_t>(g.p_tiles) * g.q_tiles;
  if (units == 0) return 0;
  int64_t split = (bn <= 32 ? 2 : 1) * sms / units;
  if (split > g.k_blocks / 2) split = g.k_blocks / 2;
  split = split >= 8 && bn <= 32 ? 8 : split >= 4 ? 4 : split >= 2 ? 2 : 1;
  CUtensorMap tp, tq;
  if (!make_tmap_fp8(&tp, b.q, static_cast<uint64_t>(b.cols), static_cast<uint64_t>(b.rows) * b.batch,
                     static_cast<uint64_t>(b.ld), 128))
    return static_cast<int>(cudaErrorInvalidValue);
  if (x) tq = tp;
  else if (!make_tmap_fp8(&tq, a.q, static_cast<uint64_t>(a.cols), static_cast<uint64_t>(a.rows), static_cast<uint64_t>(a.ld),
                          static_cast<uint32_t>(bn)))
    return static_cast<int>(cudaErrorInvalidValue);
  const int s = static_cast<int>(split);
  auto width = [&](auto vec) {
    constexpr bool V = decltype(vec)::value;
    switch (bn) {
      case 16: return launch_tile<16, V, false>(tp, tq, g, units, s, nullptr, 0, kind, stream);
      case 32: return launch_tile<32, V, false>(tp, tq, g, units, s, nullptr, 0, kind, stream);
      case 64: return launch_tile<64, V, false>(tp, tq, g, units, s, nullptr, 0, kind, stream);
      default: return launch_tile<128, V, false>(tp, tq, g, units, s, nullptr, 0, kind, stream);
    }
  };
  if (x) return launch_tile<16, false, true>(tp, tq, g, units, s, x, a.cols, kind, stream);
  return b.row_scales ? width(std::true_type{}) : width(std::false_type{});
}

}  // namespace mok
