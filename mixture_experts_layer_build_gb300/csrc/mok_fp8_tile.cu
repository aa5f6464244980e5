// mok_fp8_tile.cu -- 8-bit products with a scale per 128 values, one 128 x BN tile per CTA.
//
// With P the operand whose rows are the accumulator's 128 lanes and Q the one whose rows are its BN columns, a CTA
// computes D[i, j] = sum over K blocks of sp[i] sq[j] (P[i, :] . Q[j, :]).  A K block is 128 bytes of a row, one
// swizzle atom: four tcgen05.mma (M = 128, K = 32) into one of two TMEM accumulators, which four warps then drain,
// scale and add into their registers while the next block's MMAs run into the other one.
//
// SWAP: P holds the weights and Q the tokens, whose number picks BN: few tokens take few columns, and the weights'
// bytes bound it.  Their K range is then split over a cluster, whose CTAs add up their partials through shared memory
// in rank order.
#include "mok_ffn.cuh"  // warp_wait, wait_landed, elect_one
#include "mok_fp8.cuh"
#include "mok_fp8_gemm.cuh"

namespace mok {
namespace {

constexpr int kThreads = 192;
constexpr int kMaxStages = 12;
constexpr uint32_t kMaxSmem = 227328;  // dynamic: 5 KB of 227 KB are left for what is static

struct TileArgs {
  Fp8Problem g;
  int32_t split;   // CTAs of a cluster that share a tile's K range (SWAP)
  int32_t stages;
  uint32_t push_off;
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
  int32_t i0, j0;        // output position (SWAP: i is the output's column)
  int32_t i_end, j_end;
  int32_t kb0, count;    // K blocks
  int64_t out;           // element offset of the matrix written
  int32_t batch;         // of BLOCKS-scaled operands
};

__device__ __forceinline__ bool fp8_tile(const Fp8Problem& g, int u, bool swap, int bn, Tile& t) {
  t.kb0 = 0;
  t.count = g.k_blocks;
  t.out = 0;
  t.batch = 0;
  const int pt = u % g.p_tiles;
  int rest = u / g.p_tiles;
  if (g.mode == FP8_DENSE) {
    t.p0 = t.i0 = pt * 128;
    t.q0 = t.j0 = rest * bn;
    t.i_end = g.p_rows;
    t.j_end = g.q_rows;
    return true;
  }
  if (g.mode == FP8_WGRAD) {
    const int qt = rest % g.q_tiles;
    t.batch = rest / g.q_tiles;
    t.kb0 = __ldg(g.poff + t.batch) / 128;
    t.count = __ldg(g.poff + t.batch + 1) / 128 - t.kb0;
    t.p0 = t.i0 = pt * 128;
    t.q0 = t.j0 = qt * bn;
    t.i_end = g.p_rows;
    t.j_end = g.q_rows;
    t.out = static_cast<int64_t>(t.batch) * g.p_rows * g.q_rows;
    return true;
  }
  // one 128-row block of an expert's rows, against a tile of its weights
  int wt = pt, blk = rest;
  if (!swap) {
    wt = u % g.q_tiles;
    blk = u / g.q_tiles;
  }
  if (blk >= __ldg(g.meta + 2)) return false;
  const int4 b = __ldg(reinterpret_cast<const int4*>(g.mblocks) + blk);  // {expert, first row, valid rows, tile}
  t.batch = b.x;
  if (swap) {
    t.i0 = wt * 128;
    t.p0 = b.x * g.p_rows + t.i0;
    t.i_end = g.p_rows;
    t.q0 = t.j0 = b.y;
    t.j_end = b.y + b.z;
  } else {
    t.p0 = t.i0 = b.y;
    t.i_end = b.y + b.z;
    t.j0 = wt * bn;
    t.q0 = b.x * g.q_rows + t.j0;
    t.j_end = g.q_rows;
  }
  return true;
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ float ld_shared_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

template <int BN, bool COLVEC, bool SWAP>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_tile_kernel(const __grid_constant__ CUtensorMap tP, const __grid_constant__ CUtensorMap tQ, const TileArgs a) {
  constexpr uint32_t kQBytes = BN * 128, kStage = 16384 + (kQBytes < 1024 ? 1024 : kQBytes);
  constexpr uint32_t kCols = BN <= 16 ? 32 : 2 * BN;  // two accumulators
  constexpr int W = BN < 32 ? 16 : 32;
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t bars[2 * kMaxStages + 5];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  __shared__ __align__(16) float colbuf[COLVEC ? 4 : 1][2][COLVEC ? BN : 4];  // per warp, of the current and next block
  const Fp8Problem& g = a.g;
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t bar0 = smem_u32(bars);
  auto full = [&](int s) { return bar0 + 8u * s; };
  auto empty = [&](int s) { return bar0 + 8u * (kMaxStages + s); };
  auto tfull = [&](int b) { return bar0 + 8u * (2 * kMaxStages + b); };
  auto tempty = [&](int b) { return bar0 + 8u * (2 * kMaxStages + 2 + b); };
  const uint32_t done = bar0 + 8u * (2 * kMaxStages + 4);
  volatile int* abort_flag = &abort_word;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = SWAP ? a.split : 1;
  const int rank = SWAP ? static_cast<int>(blockIdx.x) % S : 0, unit = static_cast<int>(blockIdx.x) / S;
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int b = 0; b < 2; ++b) {
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
  if (SWAP && S > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");  // this CTA has started
  if (g.mode != FP8_DENSE) pdl_wait();  // the schedule's tables
  Tile t;
  const bool have = fp8_tile(g, unit, SWAP, BN, t);
  const int subs = !have ? 0 : SWAP ? (min(t.j_end - t.j0, g.mode == FP8_DENSE ? BN : 128) + BN - 1) / BN : 1;
  // this CTA's share of the K blocks
  const int kb0 = t.kb0 + static_cast<int>(static_cast<int64_t>(t.count) * rank / S);
  const int count = t.kb0 + static_cast<int>(static_cast<int64_t>(t.count) * (rank + 1) / S) - kb0;
  const int total = subs * count;  // K blocks that pass through the stages
  if (SWAP && S > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
  bool ok = true;
  int ahead = 0;  // (warp 0) K blocks of P that were loaded early
  if (warp == 0 && g.early_p) {  // weights: nothing that still runs writes them
    ahead = min(total, a.stages);
    for (int n = 0; n < ahead; ++n)
      if (elect_one()) {
        mbar_arrive_expect_tx(full(n), 16384 + kQBytes);
        tma_load_2d(base + n * kStage, &tP, full(n), (kb0 + n % count) * 128, t.p0);
      }
  }
  pdl_wait();  // (the kernel in front may take its time: no bounded wait starts before its end)
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
            mbar_arrive_expect_tx(full(st), 16384 + kQBytes);
            tma_load_2d(sp, &tP, full(st), (kb0 + kb) * 128, t.p0);
          }
          tma_load_2d(sp + 16384, &tQ, full(st), (kb0 + kb) * 128, t.q0 + sub * BN);
        }
        ++n;
        if (++st == a.stages) {
          st = 0;
          ph ^= 1u;
        }
      }
    } else if (warp == 1) {
      for (int kb = 0; kb < count && ok; ++kb, ++n) {
        const int b = n & 1;
        ok = (n < 2 || warp_wait(tempty(b), static_cast<uint32_t>(n / 2 - 1) & 1u, abort_flag, g.status)) &&
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
    } else {
#pragma unroll
      for (int j = 0; j < BN; ++j) acc[j] = 0.0f;
      const int i = min(t.i0 + r, t.i_end - 1), j0 = t.j0 + sub * BN;
      const float* ps = g.p_vec ? g.sp + i : g.sp + t.batch * g.p_batch + static_cast<int64_t>(i / 128) * g.k_blocks;
      const float* qs = COLVEC ? g.sq : g.sq + t.batch * g.q_batch + static_cast<int64_t>(j0 / 128) * g.k_blocks;
      const int64_t p_step = g.p_vec ? g.p_pitch : 1;
      float p_next = count > 0 ? __ldg(ps + kb0 * p_step) : 0.0f;
      // column scales: each lane its share of the warp's BN, four at a time (rows of scales are padded to four)
      float4 q_next = make_float4(0, 0, 0, 0);
      const int cq = lane * 4;
      auto fetch_q = [&](int kb) {
        if constexpr (COLVEC) {
          if (cq < BN && j0 + cq < g.q_pitch)
            q_next = __ldg(reinterpret_cast<const float4*>(qs + static_cast<int64_t>(kb) * g.q_pitch + j0 + cq));
        } else {
          q_next.x = __ldg(qs + kb);
        }
      };
      if (count > 0) fetch_q(kb0);
      for (int kb = 0; kb < count && ok; ++kb, ++n) {
        const int b = n & 1;
        float s = p_next;
        const float* cs = colbuf[COLVEC ? warp - 2 : 0][COLVEC ? b : 0];
        if constexpr (COLVEC) {
          if (cq < BN) *reinterpret_cast<float4*>(&colbuf[warp - 2][b][cq]) = q_next;
          __syncwarp();
        } else {
          s *= q_next.x;
        }
        if (kb + 1 < count) {
          p_next = __ldg(ps + (kb0 + kb + 1) * p_step);
          fetch_q(kb0 + kb + 1);
        }
        ok = warp_wait(tfull(b), static_cast<uint32_t>(n / 2) & 1u, abort_flag, g.status);
        if (!ok) break;
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
            float f0 = s, f1 = s, f2 = s, f3 = s;
            if constexpr (COLVEC) {
              const float4 x = *reinterpret_cast<const float4*>(cs + c + j);
              mul_f32x2(f0, f1, s, s, x.x, x.y);
              mul_f32x2(f2, f3, s, s, x.z, x.w);
            }
            fma_f32x2(acc[c + j], acc[c + j + 1], __uint_as_float(v[j]), __uint_as_float(v[j + 1]), f0, f1, acc[c + j],
                      acc[c + j + 1]);
            fma_f32x2(acc[c + j + 2], acc[c + j + 3], __uint_as_float(v[j + 2]), __uint_as_float(v[j + 3]), f2, f3,
                      acc[c + j + 2], acc[c + j + 3]);
          }
        }
      }
    }
    const int j0 = t.j0 + sub * BN;
    if constexpr (SWAP) {
      uint16_t* out = static_cast<uint16_t*>(g.out) + t.i0 + r;
      const bool mine = warp >= 2 && t.i0 + r < t.i_end;
      if (S == 1) {
        if (mine && ok) {
#pragma unroll
          for (int j = 0; j < BN; ++j)
            if (j0 + j < t.j_end) {
              if (g.out_f32) static_cast<float*>(g.out)[static_cast<int64_t>(j0 + j) * g.ldo + t.i0 + r] = acc[j];
              else out[static_cast<int64_t>(j0 + j) * g.ldo] = static_cast<uint16_t>(pack_bf16x2(acc[j], 0.0f));
            }
        }
      } else {
        // column j belongs to CTA j / per of the cluster: each sends it its partial, the owner adds them in rank order
        const int per = BN / S;
        const uint32_t push = base + a.push_off;
        if (warp >= 2) {
#pragma unroll
          for (int j = 0; j < BN; ++j) {
            const int own = j / per, jj = j - own * per;
            st_cluster_f32(mapa_shared(push + static_cast<uint32_t>((rank * per + jj) * 128 + r) * 4u, own), acc[j]);
          }
        }
        __syncwarp();
        cluster_sync();
        if (mine && *abort_flag == 0)
          for (int jj = 0; jj < per; ++jj) {
            const int j = j0 + rank * per + jj;
            float v = 0.0f;
            for (int c = 0; c < S; ++c) v += ld_shared_f32(push + static_cast<uint32_t>((c * per + jj) * 128 + r) * 4u);
            if (j < t.j_end) {
              if (g.out_f32) static_cast<float*>(g.out)[static_cast<int64_t>(j) * g.ldo + t.i0 + r] = v;
              else out[static_cast<int64_t>(j) * g.ldo] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f));
            }
          }
        __syncwarp();
        if (sub + 1 < subs) cluster_sync();  // the partials have been read
      }
    } else if (warp >= 2 && ok && t.i0 + r < t.i_end) {
      const int64_t at = t.out + static_cast<int64_t>(t.i0 + r) * g.ldo + j0;
      if (g.out_f32) {
        float* o = static_cast<float*>(g.out) + at;
#pragma unroll
        for (int j = 0; j < BN; j += 4)
          if (j0 + j < t.j_end) *reinterpret_cast<float4*>(o + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
      } else {
        uint16_t* o = static_cast<uint16_t*>(g.out) + at;
#pragma unroll
        for (int j = 0; j < BN; j += 8)
          if (j0 + j < t.j_end)
            *reinterpret_cast<uint4*>(o + j) =
                make_uint4(pack_bf16x2(acc[j], acc[j + 1]), pack_bf16x2(acc[j + 2], acc[j + 3]),
                           pack_bf16x2(acc[j + 4], acc[j + 5]), pack_bf16x2(acc[j + 6], acc[j + 7]));
      }
    }
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

template <int BN, bool COLVEC, bool SWAP>
int launch_tile(const CUtensorMap& tP, const CUtensorMap& tQ, const Fp8Problem& g, int64_t units, int split, int kind,
                cudaStream_t stream) {
  static DeviceOnce once;
  const int se = once.run([](int* d) { return static_cast<int>(cudaGetDevice(d)); },
                          [] {
                            return static_cast<int>(cudaFuncSetAttribute(fp8_tile_kernel<BN, COLVEC, SWAP>,
                                                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                                         static_cast<int>(kMaxSmem)));
                          },
                          static_cast<int>(cudaErrorInvalidDevice));
  if (se) return se;
  if (units * split >= (int64_t{1} << 31)) return static_cast<int>(cudaErrorInvalidValue);
  constexpr uint32_t kStage = 16384 + (BN * 128 < 1024 ? 1024 : BN * 128);
  TileArgs a{};
  a.g = g;
  a.split = split;
  const uint32_t push = split > 1 ? BN * 512u : 0u;
  const uint32_t fixed = 1024u + push;  // alignment; partials
  a.stages = static_cast<int32_t>((kMaxSmem - fixed) / kStage);
  if (a.stages > kMaxStages) a.stages = kMaxStages;
  a.push_off = static_cast<uint32_t>(a.stages) * kStage;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * split));
  cfg.blockDim = dim3(kThreads);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_tile_kernel<BN, COLVEC, SWAP>, tP, tQ, a);
  trace_end(stream);
  return static_cast<int>(e);
}

}  // namespace

int launch_fp8_tile(const Fp8Operand& a, const Fp8Operand& b, Fp8Problem g, int64_t rows, int64_t row_blocks, int kind,
                    cudaStream_t stream) {
  const int sms = sm_count();
  if (sms <= 0) return static_cast<int>(cudaErrorInvalidDevice);
  const int64_t N = b.rows;
  auto maps = [&](const Fp8Operand& p, const Fp8Operand& q, int bn, CUtensorMap* tp, CUtensorMap* tq) {
    return make_tmap_fp8(tp, p.q, static_cast<uint64_t>(p.cols), static_cast<uint64_t>(p.rows) * p.batch,
                         static_cast<uint64_t>(p.ld), 128) &&
           make_tmap_fp8(tq, q.q, static_cast<uint64_t>(q.cols), static_cast<uint64_t>(q.rows) * q.batch,
                         static_cast<uint64_t>(q.ld), static_cast<uint32_t>(bn));
  };
  auto sides = [&](const Fp8Operand& p, const Fp8Operand& q) {
    g.sp = p.s;
    g.p_vec = p.row_scales;
    g.p_pitch = fp8_pitch(p.rows);
    g.p_batch = fp8_blocks(p.rows) * g.k_blocks;
    g.p_rows = static_cast<int32_t>(p.rows);
    g.sq = q.s;
    g.q_pitch = fp8_pitch(q.rows);
    g.q_batch = fp8_blocks(q.rows) * g.k_blocks;
    g.q_rows = static_cast<int32_t>(q.rows);
  };
  CUtensorMap tp, tq;
  const bool swap = !b.row_scales && rows <= 128 * (g.mode == FP8_GROUPED ? row_blocks : 1);
  if (swap) {
    sides(b, a);
    g.p_tiles = static_cast<int32_t>(fp8_blocks(N));
    const int64_t per = g.mode == FP8_GROUPED ? (rows + row_blocks - 1) / (row_blocks > 0 ? row_blocks : 1) : rows;
    const int bn = per <= 16 ? 16 : per <= 32 ? 32 : per <= 64 ? 64 : 128;
    g.q_tiles = static_cast<int32_t>(g.mode == FP8_GROUPED ? row_blocks : (rows + bn - 1) / bn);
    const int64_t units = static_cast<int64_t>(g.p_tiles) * g.q_tiles;
    int64_t split = sms / (units > 0 ? units : 1);
    if (split > g.k_blocks / 2) split = g.k_blocks / 2;
    split = split >= 8 ? 8 : split >= 4 ? 4 : split >= 2 ? 2 : 1;
    if (units == 0) return 0;
    if (!maps(b, a, bn, &tp, &tq)) return static_cast<int>(cudaErrorInvalidValue);
    const int s = static_cast<int>(split);
    switch (bn) {
      case 16: return launch_tile<16, true, true>(tp, tq, g, units, s, kind, stream);
      case 32: return launch_tile<32, true, true>(tp, tq, g, units, s, kind, stream);
      case 64: return launch_tile<64, true, true>(tp, tq, g, units, s, kind, stream);
      default: return launch_tile<128, true, true>(tp, tq, g, units, s, kind, stream);
    }
  }
  sides(a, b);
  g.early_p = 0;
  g.q_tiles = static_cast<int32_t>(fp8_blocks(N));
  g.p_tiles = static_cast<int32_t>(g.mode == FP8_GROUPED ? row_blocks : fp8_blocks(a.rows));
  const int64_t units = static_cast<int64_t>(g.p_tiles) * g.q_tiles * (g.mode == FP8_WGRAD ? g.experts : 1);
  if (units == 0) return 0;
  if (!maps(a, b, 128, &tp, &tq)) return static_cast<int>(cudaErrorInvalidValue);
  return b.row_scales ? launch_tile<128, true, false>(tp, tq, g, units, 1, kind, stream)
                      : launch_tile<128, false, false>(tp, tq, g, units, 1, kind, stream);
}

}  // namespace mok
