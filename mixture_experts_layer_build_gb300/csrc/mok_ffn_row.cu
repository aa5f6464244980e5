// mok_ffn_row.cu -- the feed-forward block's forward contractions for one to four tokens: every weight is
// read once, straight into registers, and multiplied on the CUDA cores.
//
//   GATEUP  a[t, i] = act(<x_t, Wg_i>) <x_t, Wu_i>        DOWN  out[t, h] = <a_t, Wd_h> + residual[t, h]
//
// Bound by the weights' bytes.  A CTA of four warps takes four weight rows (GATEUP: two of Wg and the same
// two of Wu); the warps take 256-column chunks of K in turn, a lane 8 neighbouring columns of each row
// (512 contiguous bytes per warp and load), two chunks ahead of the arithmetic: eight 16-byte loads of
// weights in flight per lane.  Products and sums in fp32, two neighbouring columns per instruction
// (fma.rn.f32x2): along each lane's columns, the even and the odd ones apart, then a butterfly over the
// warp, then the warps in ascending order.
//
// Measured (H = 4096, I = 1536, weights from HBM, both contractions): 9.1 us for one token, 10.7 for two, 13.3 for four,
// against 13.6 to 14.1 on the tensor cores (mok_ffn_tile.cu) for any of 5 to 32; at H = 7168, I = 2048 16.3 (5.4 TB/s) for
// one, 22.2 for four against 21.7.  For eight tokens it took 22.6 and 41.1 at the two: the tokens' loads and the
// arithmetic, once per four weight rows, then outweigh the weights.
// Hence kFfnRowTokens.
#include "mok_ffn.cuh"

namespace mok {
namespace {

constexpr int kRowWarps = 4;
constexpr int kRowRows = 4;  // weight rows per CTA

struct RowArgs {
  FfnArgs f;
  const uint16_t* x;   // [T, K]
  const uint16_t* w0;  // [N, K]
  const uint16_t* w1;  // GATEUP: Wu
  int32_t K;
};

__device__ __forceinline__ uint4 ld_stream(const uint16_t* p) { return __ldcs(reinterpret_cast<const uint4*>(p)); }

// (bf16 low, bf16 high) of a word as a pair of fp32.
__device__ __forceinline__ uint64_t bf16_pair(uint32_t v) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(v << 16), "r"(v & 0xFFFF0000u));
  return r;
}
__device__ __forceinline__ void fma_pair(uint64_t& d, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ float pair_sum(uint64_t v) {
  float lo, hi;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
  return lo + hi;
}

template <int VAR, int TT>
__global__ void __launch_bounds__(32 * kRowWarps) ffn_row_kernel(const RowArgs a) {
  constexpr bool kGate = VAR == F_GATEUP;
  constexpr int kAhead = 2;                              // chunks in flight
  constexpr int kStep = kRowWarps * 256;                 // columns between a warp's chunks
  constexpr int kOut = kGate ? kRowRows / 2 : kRowRows;  // output columns per CTA
  __shared__ float part[kRowWarps][kRowRows * TT];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n0 = static_cast<int>(blockIdx.x) * kOut;
  const int K = a.K, T = a.f.M, N = a.f.N;
  const uint16_t* rows[kRowRows];
#pragma unroll
  for (int r = 0; r < kRowRows; ++r) {
    const int n = min(n0 + (kGate ? r >> 1 : r), N - 1);  // past the last column: its row again, not stored
    rows[r] = (kGate && (r & 1) ? a.w1 : a.w0) + static_cast<int64_t>(n) * K;
  }
  const uint4 zero = make_uint4(0, 0, 0, 0);
  uint4 w[kAhead][kRowRows];
  auto load_w = [&](int u, int k) {
#pragma unroll
    for (int r = 0; r < kRowRows; ++r) w[u][r] = k < K ? ld_stream(rows[r] + k) : zero;
  };
  const int k0 = warp * 256 + lane * 8;
  if (kGate) pdl_wait();
  // (DOWN: always behind GATEUP, which runs once everything before it has ended: weights may be read)
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load_w(u, k0 + u * kStep);
  if (!kGate) pdl_wait();
  pdl_trigger();
  uint64_t acc[kRowRows][TT];
#pragma unroll
  for (int r = 0; r < kRowRows; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = 0;
  for (int c = k0; c - lane * 8 < K; c += kAhead * kStep) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int k = c + u * kStep;
      uint64_t wp[kRowRows][4];
#pragma unroll
      for (int r = 0; r < kRowRows; ++r) {
        wp[r][0] = bf16_pair(w[u][r].x), wp[r][1] = bf16_pair(w[u][r].y);
        wp[r][2] = bf16_pair(w[u][r].z), wp[r][3] = bf16_pair(w[u][r].w);
      }
      load_w(u, k + kAhead * kStep);
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const uint4 x =
            k < K && t < T ? *reinterpret_cast<const uint4*>(a.x + static_cast<int64_t>(t) * K + k) : zero;
        const uint64_t xp[4] = {bf16_pair(x.x), bf16_pair(x.y), bf16_pair(x.z), bf16_pair(x.w)};
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int r = 0; r < kRowRows; ++r) fma_pair(acc[r][t], wp[r][i], xp[i]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRowRows; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      float v = pair_sum(acc[r][t]);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
      if (lane == 0) part[warp][r * TT + t] = v;
    }
  __syncthreads();
  const int t = static_cast<int>(threadIdx.x) / kOut, j = static_cast<int>(threadIdx.x) - t * kOut, n = n0 + j;
  if (t >= T || n >= N || t >= TT) return;
  auto sum = [&](int r) {
    float v = part[0][r * TT + t];
#pragma unroll
    for (int i = 1; i < kRowWarps; ++i) v += part[i][r * TT + t];
    return v;
  };
  const int64_t o = static_cast<int64_t>(t) * N + n;
  float v;
  if constexpr (kGate) {
    const float g = sum(2 * j), u = sum(2 * j + 1);
    if (a.f.kg) {
      const int64_t s = ffn_saved_offset(t, n, N);
      v = act_saved(g, u, a.f.act, a.f.kg[s], a.f.ku[s]);
    } else {
      v = act_fwd(g, a.f.act) * u;
    }
  } else {
    v = sum(j);
    if (a.f.residual) v += bf16_lo(a.f.residual[o]);
  }
  static_cast<uint16_t*>(a.f.out0)[o] = static_cast<uint16_t>(pack_bf16x2(v, 0.0f));
}

template <int VAR>
int launch_rows(const RowArgs& a, cudaStream_t stream) {
  constexpr int kOut = VAR == F_GATEUP ? kRowRows / 2 : kRowRows;
  const dim3 grid((a.f.N + kOut - 1) / kOut), block(32 * kRowWarps);
  trace_begin(stream, K_FFN_GATEUP + VAR);
  cudaError_t e;
  if (a.f.M <= 1) e = launch_pdl(ffn_row_kernel<VAR, 1>, grid, block, 0, stream, a);
  else if (a.f.M <= 2) e = launch_pdl(ffn_row_kernel<VAR, 2>, grid, block, 0, stream, a);
  else e = launch_pdl(ffn_row_kernel<VAR, kFfnRowTokens>, grid, block, 0, stream, a);
  trace_end(stream);
  return static_cast<int>(e);
}

}  // namespace

int launch_ffn_row(int var, int64_t M, int64_t N, int64_t K, const FfnOperands& o, const FfnArgs& f,
                   cudaStream_t stream) {
  RowArgs a{};
  a.f = f;
  a.f.M = static_cast<int32_t>(M);
  a.f.N = static_cast<int32_t>(N);
  a.K = static_cast<int32_t>(K);
  a.x = static_cast<const uint16_t*>(o.a);
  a.w0 = static_cast<const uint16_t*>(o.b);
  a.w1 = static_cast<const uint16_t*>(o.b2);
  return var == F_GATEUP ? launch_rows<F_GATEUP>(a, stream) : launch_rows<F_DOWN>(a, stream);
}

}  // namespace mok
