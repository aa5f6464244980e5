// mok_ffn.cuh -- the dense gated feed-forward block: what its kernels share (sizes, arguments, the
// activations).
//
// Six contractions over tokens t, hidden h and intermediate i (row-major operands; K is the summed
// index):
//   GATEUP  [g | u] = x [Wg | Wu]^T, epilogue a = act(g) u           M = T, N = I (twice), K = H
//   DOWN    out = a Wd^T + residual                                  M = T, N = H, K = I
//   DACT    da = dy Wd, epilogue dg = da u act'(g), du = da act(g)   M = T, N = I, K = H
//           (both factors are made and saved by GATEUP's epilogue, where the sigmoid is at hand)
//   DX      dx = dg Wg + du Wu + dx_add                              M = T, N = H, K = I twice
//   DW      dWg = dg^T x, dWu = du^T x                               M = I, N = H, K = T
//           dWd = dy^T a                                             M = H, N = I, K = T
// An operand whose rows run along K is K-major for the MMA, one whose rows run along M or N is
// MN-major: weights in DACT and DX, both operands in DW.
#pragma once
#include <cuda.h>

#include "mok_ffn_plan.h"
#include "mok_internal.cuh"
#include "mok_once.h"
#include "mok_ptx.cuh"

namespace mok {

__host__ __device__ constexpr bool ffn_b_mn(int v) { return v >= F_DACT; }

struct FfnArgs {
  int32_t M, N;         // rows and columns of the output
  int32_t m_tiles, n_tiles;
  int32_t k_blocks;
  int32_t kb_split;     // DX: K blocks over (dg, Wg), then the same over (du, Wu)
  int32_t act;
  int32_t out_f32;      // weight gradients: fp32 instead of bf16
  void* out0;           // a | out | dg | dx
  void* out1;           // - | -   | du | -
  float* kg;            // u act'(g) and act(g), fp32.  GATEUP: saved when not null; DACT: read
  float* ku;
  const uint16_t* residual;  // DOWN (the residual), DX (dx_add): added to the output, may be null
  uint32_t* status;
};

// Element offset of (row, column) of the saved factors, columns a multiple of 4 wide: blocks of 32 rows x 4
// columns, so that a warp whose lanes hold 32 rows of an accumulator moves 512 contiguous bytes per
// 4 columns straight from and to its registers.  Rows are padded to a multiple of 32.
__host__ __device__ __forceinline__ int64_t ffn_saved_offset(int64_t row, int col, int I) {
  return ((row >> 5) * (I >> 2) + (col >> 2)) * 128 + (row & 31) * 4 + (col & 3);
}

#ifdef __CUDACC__
// Bounded wait that ignores the abort flag: only while winding down.
__device__ __forceinline__ void wait_landed(uint32_t bar, uint32_t parity) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity) && global_timer_ns() - t0 < kWaitLimitNs / 4) {
  }
}
// mbar_wait for a barrier that completes when all k_blocks MMAs of a tile have: the tokens of a weight gradient may be
// more K blocks than the limit of a single wait allows.
__device__ __forceinline__ bool mbar_wait_tile(uint32_t bar, uint32_t parity, int k_blocks, volatile int* abort,
                                               uint32_t* status) {
  const uint64_t limit = tile_wait_ns(kWaitLimitNs, k_blocks), t0 = global_timer_ns();
  for (uint32_t spins = 1; !mbar_try_wait(bar, parity); ++spins) {
    if (spins & 63u) continue;
    if (*abort) return false;
    if (global_timer_ns() - t0 > limit) {
      *abort = 1;
      record_status(status, MOK_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}
// The whole warp waits; the same answer on every lane.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, status));
}
// Let the stream's next kernel be scheduled.  Only after this thread's pdl_wait() -- all kernels before this
// one have then ended, so that one that follows knows that of everything but this one -- and after the
// CTA's TMEM is allocated: a CTA of the next kernel that took the columns first would wait for this
// grid while holding them.
__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

__device__ __forceinline__ float sigmoid_fast(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

// act(g) and, for the backward, act'(g).  The tanh form of GELU is g sigmoid(2 z), z = c (g + k g^3),
// since (1 + tanh z) / 2 = sigmoid(2 z): no cancellation for negative g.  The exponential and the
// division are the fast approximations (a few ulp of fp32): what they feed is rounded to bf16 (2^-9).
__device__ __forceinline__ float act_fwd(float g, int act) {
  if (act == MOK_ACT_SILU) return g * sigmoid_fast(g);
  return g * sigmoid_fast(1.5957691216057308f * g * fmaf(0.044715f * g, g, 1.0f));
}
__device__ __forceinline__ void act_bwd(float g, int act, float& f, float& df) {
  if (act == MOK_ACT_SILU) {
    const float s = sigmoid_fast(g);
    f = g * s;
    df = s * fmaf(g, 1.0f - s, 1.0f);
  } else {
    const float s = sigmoid_fast(1.5957691216057308f * g * fmaf(0.044715f * g, g, 1.0f));
    f = g * s;
    df = fmaf(f * (1.0f - s), 1.5957691216057308f * fmaf(3.0f * 0.044715f * g, g, 1.0f), s);
  }
}
// a = act(g) u, with the factors of dg and du.
__device__ __forceinline__ float act_saved(float g, float u, int act, float& kg, float& ku) {
  float df;
  act_bwd(g, act, ku, df);
  kg = u * df;
  return ku * u;
}
#endif

bool make_tmap_bf16(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint32_t box_inner,
                    uint32_t box_outer);
bool make_tmap_bf16_sw64(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint32_t box_inner,
                         uint32_t box_outer);
bool make_tmap_f32_sw64(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint32_t box_inner,
                        uint32_t box_outer);

struct FfnOperands {
  const void* a;   // x  | a  | dy | dg
  const void* a2;  // -    -    -    du
  const void* b;   // Wg | Wd | Wd | Wg
  const void* b2;  // Wu   -    -    Wu
};
// The backward's operands.  dw_gate == nullptr, dw_down == nullptr: not computed.
struct FfnBackward {
  int64_t T, H, I;
  int32_t act, dw_f32;
  bool dact, dx_rows;  // DACT, DX in the phases' launches (else before them on the tile kernel, or not wanted)
  const void* x;
  const void* w_gate;
  const void* w_up;
  const void* w_down;
  const void* a;
  const float* kg;
  const float* ku;
  const void* dy;
  void* dg;
  void* du;
  void* dx;
  const void* dx_add;
  void* dw_gate;
  void* dw_up;
  void* dw_down;
  uint32_t* status;
};
// One row-tiled contraction: M, N, K of the variant (K of one half for DX), operands and the epilogue's
// fields of `a` set.  The tile kernel (one tile per CTA, K split when there are few tiles; mok_ffn_tile.cu)
// and persistent CTA pairs (mok_ffn_pair.cu).
int launch_ffn_tile(int var, int64_t M, int64_t N, int64_t K, const FfnOperands& o, const FfnArgs& a,
                    cudaStream_t stream);
// GATEUP and DOWN for at most kFfnRowTokens tokens (mok_ffn_row.cu).
constexpr int kFfnRowTokens = 4;
int launch_ffn_row(int var, int64_t M, int64_t N, int64_t K, const FfnOperands& o, const FfnArgs& a,
                   cudaStream_t stream);
int launch_ffn_pair_fwd(int var, int64_t M, int64_t N, int64_t K, const FfnOperands& o, const FfnArgs& a,
                        cudaStream_t stream);
// Phase 1: DACT (if b.dact), perhaps dWd; phase 2, after it: DX (if b.dx_rows) and the other weight gradients.
int launch_ffn_pair_bwd(int phase, const FfnBackward& b, cudaStream_t stream);

}  // namespace mok
