// mok_norm.cu -- the residual stream's kernels: root-mean-square norm with the branch's (dropped-out)
// addition and a bf16 or MXFP8 output, its backward, and dropout with the residual's addition alone.
//
//   forward   h = residual + dropout(x),  rstd = (mean h^2 + eps)^-1/2,  y = h rstd weight
//   backward  xh = h rstd, g = dy weight: dh = rstd (g - xh mean(g xh)) + dres, dx = factors * dh,
//             dweight = sum over rows of dy xh
//
// All of it is bound by HBM: every value is read once and written once, and a row stays in its
// threads' registers between the row reduction and the outputs.  fp32 arithmetic throughout, one
// rounding per output.  No atomics: the row sums and dweight are reduced in fixed orders.
//
// Measured, every operand in memory of its own (of 6,784 GB/s copy): forward 8192 x 4096 bf16 40.6 us (6.6 TB/s), with
// dropout and an MXFP8 output 40.4 (5.8: issue slots); backward 47.6 (5.6), with dropout 57.3 (5.9), 16384 x 7168 with an
// fp32 stream 289 (6.5); dropout 32.8 (6.1), its backward at 16384 x 7168 74.2 (6.3), with an fp32 stream 105 (6.7).
#include <cmath>
#include <type_traits>

#include "mok_internal.cuh"
#include "mok_philox.cuh"
#include "mok_ptx.cuh"

namespace mok {
namespace {

constexpr int kNormMaxH = 16384;
constexpr int kNormThreads = 512;  // most threads of a block
constexpr int kNormParts = 304;  // most partial dweight rows: two blocks of 256 threads on each of 152 SMs

// fp32 values in pairs: one instruction for two (add, mul, fma .f32x2), each rounded as the scalar one.
using Pair = uint64_t;
__device__ __forceinline__ Pair pair_of(uint32_t lo, uint32_t hi) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ Pair splat(float v) { return pair_of(__float_as_uint(v), __float_as_uint(v)); }
__device__ __forceinline__ float2 floats_of(Pair p) {
  float2 v;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(p));
  return v;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_pair(Pair p) {
  const float2 v = floats_of(p);
  return pack_bf16x2(v.x, v.y);
}
__device__ __forceinline__ uint4 pack_pairs(const Pair (&v)[4]) {
  return make_uint4(pack_pair(v[0]), pack_pair(v[1]), pack_pair(v[2]), pack_pair(v[3]));
}
// 8 bf16 as fp32 bit patterns, or as pairs.
__device__ __forceinline__ void bits_of(uint4 q, uint32_t (&b)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) b[2 * i] = w[i] << 16, b[2 * i + 1] = w[i] & 0xFFFF0000u;
}
__device__ __forceinline__ void pairs_of(uint4 q, Pair (&v)[4]) {
  uint32_t b[8];
  bits_of(q, b);
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = pair_of(b[2 * i], b[2 * i + 1]);
}

// 8 values of a bf16 or fp32 tensor, as loaded.  The loads are streaming (evict-first: no kernel
// of the call reads them again) and coherent, since an output may be an input's buffer.
template <bool F32>
struct Vec8;
template <>
struct Vec8<false> {
  uint4 q;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    q = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i));
  }
  __device__ __forceinline__ void bits(uint32_t (&b)[8]) const { bits_of(q, b); }
  __device__ __forceinline__ void get(Pair (&v)[4]) const { pairs_of(q, v); }
  static __device__ __forceinline__ void store(void* p, int64_t i, const Pair (&v)[4]) {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = pack_pairs(v);
  }
  // the values as the type stores them
  static __device__ __forceinline__ void round(Pair (&v)[4]) { pairs_of(pack_pairs(v), v); }
};
template <>
struct Vec8<true> {
  uint4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const uint4* s = reinterpret_cast<const uint4*>(static_cast<const float*>(p) + i);
    a = __ldcs(s);
    b = __ldcs(s + 1);
  }
  __device__ __forceinline__ void bits(uint32_t (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void get(Pair (&v)[4]) const {
    v[0] = pair_of(a.x, a.y), v[1] = pair_of(a.z, a.w), v[2] = pair_of(b.x, b.y), v[3] = pair_of(b.z, b.w);
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, const Pair (&v)[4]) {
    ulonglong2* d = reinterpret_cast<ulonglong2*>(static_cast<float*>(p) + i);
    d[0] = make_ulonglong2(v[0], v[1]);
    d[1] = make_ulonglong2(v[2], v[3]);
  }
  static __device__ __forceinline__ void round(Pair (&)[4]) {}
};

// Sum over the tpr threads of one row, in a fixed order; every thread gets it.  A row is a power of two of
// lanes of a warp, or whole warps: a butterfly within the warp, then the warps' sums in ascending order.
// All threads of the block call it; `buf` (32 words) may be used again after the next call's first
// barrier, so two calls in a row need two buffers.
__device__ __forceinline__ float row_sum(float v, int tpr, float* buf) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
    if (off < tpr) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (tpr <= 32) return v;  // the same for the whole grid
  if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = v;
  __syncthreads();
  const int nw = tpr >> 5, w0 = static_cast<int>(threadIdx.x >> 5) / nw * nw;
  float s = 0.0f;
  for (int i = 0; i < nw; ++i) s += buf[w0 + i];
  return s;
}

struct NormFwdArgs {
  const void* x;
  const void* residual;
  const uint16_t* w;
  void* h;
  uint16_t* y;
  uint8_t* yq;
  uint8_t* ys;
  float* rstd;
  int64_t T;
  int32_t H, tpr;
  float eps;
  DropArgs drop;
};

// Largest magnitude of three fp32, NaN if any is NaN.
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// MXFP8 of the 32 values held by four neighbouring lanes (8 each): shared = floor(log2 max) - 8,
// clamped at -127; codes E4M3 of v 2^-shared, saturating; a block with an Inf or a NaN gets scale 0xFF
// and codes 0x7F.
__device__ __forceinline__ void mx_store8(const Pair (&v)[4], uint8_t* q, uint8_t* s, int64_t off, int64_t soff,
                                          int c, bool in) {
  const float2 f0 = floats_of(v[0]), f1 = floats_of(v[1]), f2 = floats_of(v[2]), f3 = floats_of(v[3]);
  float m = max3_abs_nan(f0.x, f0.y, f1.x);
  m = max3_abs_nan(m, f1.y, f2.x);
  m = max3_abs_nan(m, f2.y, max3_abs_nan(f3.x, f3.y, 0.0f));
  m = fmax_abs_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmax_abs_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t amax = __float_as_uint(m) & 0x7FFFFFFFu;
  if (!in) return;  // after the shuffles
  const bool bad = amax > 0x7F7FFFFFu;
  // scale byte = max(exponent field - 8, 0); 2^-shared has exponent field 254 - byte, at least 7 here
  const int byte = max(static_cast<int>(amax >> 23) - 8, 0);
  const Pair dn = splat(__uint_as_float(static_cast<uint32_t>(254 - byte) << 23));
  uint16_t e[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 t = floats_of(mul2(v[j], dn));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e[j]) : "f"(t.y), "f"(t.x));
  }
  uint2 o = make_uint2(e[0] | static_cast<uint32_t>(e[1]) << 16, e[2] | static_cast<uint32_t>(e[3]) << 16);
  if (bad) o = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  *reinterpret_cast<uint2*>(q + off + c) = o;
  if ((c & 31) == 0) s[soff + c / 32] = static_cast<uint8_t>(bad ? 0xFF : byte);
}

// Facts of one call that a kernel's type may hold.  kFull: every thread has V vectors of an existing row, no bounds to
// test; kStream: every tensor of the residual stream is there (forward: residual and h; backward: dres, dh and dx);
// kDrop: with dropout.
enum { kFull = 1, kStream = 2, kDrop = 4 };
template <int KNOWN>
using Known = std::integral_constant<int, KNOWN>;

// Block = blockDim.x / tpr rows of tpr threads; thread t of a row holds vectors t, t + tpr, ... of 8 values.
// The draws need no data: they are made while the row's loads fly.  What a call is known to have
// is in the type: issue slots are what the MXFP8 output with dropout runs out of (at 8192 x 4096: 45.9 us with nothing
// known, 42.4 with kFull and kDrop, 40.5 with all three).
template <int V, bool F32, int MAXT, int MINB, int KNOWN>
__global__ void __launch_bounds__(MAXT, MINB) rmsnorm_fwd_kernel(const NormFwdArgs a) {
  constexpr bool FULL = KNOWN & kFull, STREAM = KNOWN & kStream, DROP = KNOWN & kDrop;
  pdl_wait();
  __shared__ float buf[32];
  const int rows = static_cast<int>(blockDim.x) / a.tpr;
  const int rl = static_cast<int>(threadIdx.x) / a.tpr, t = static_cast<int>(threadIdx.x) - rl * a.tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * rows + rl, off = row * a.H;
  auto has = [&](int c) { return FULL || (row < a.T && c < a.H); };  // column c of this thread's row exists
  uint4 x[V];
  Vec8<F32> r[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * a.tpr + t) * 8;
    if (has(c)) {
      x[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + off + c));
      if (STREAM || a.residual) r[j].load(a.residual, off + c);
    }
  }
  uint32_t draws[V][4];
  if constexpr (DROP) {
    DropState ds;
    ds.load(a.drop);
#pragma unroll
    for (int j = 0; j < V; ++j) philox8(ds, static_cast<uint64_t>(off + (j * a.tpr + t) * 8) >> 3, draws[j]);
  }
  const Pair scale = splat(a.drop.scale);
  Pair v[V][4];
  Pair ss = 0;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * a.tpr + t) * 8;
#pragma unroll
    for (int k = 0; k < 4; ++k) v[j][k] = 0;
    if (has(c)) {
      uint32_t xb[8];
      bits_of(x[j], xb);
      if constexpr (DROP) drop_bits(xb, a.drop, draws[j]);
      Pair rr[4];
      if (STREAM || a.residual) {
        r[j].get(rr);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) rr[k] = pair_of(0x80000000u, 0x80000000u);  // -0: x + -0 is x
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) v[j][k] = fma2(pair_of(xb[2 * k], xb[2 * k + 1]), scale, rr[k]);
      if (STREAM || a.h) {
        Vec8<F32>::store(a.h, off + c, v[j]);
        Vec8<F32>::round(v[j]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) ss = fma2(v[j][k], v[j][k], ss);
    }
  }
  uint4 wq[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * a.tpr + t) * 8;
    wq[j] = FULL || c < a.H ? __ldg(reinterpret_cast<const uint4*>(a.w + c)) : make_uint4(0, 0, 0, 0);
  }
  const float2 s2 = floats_of(ss);
  const float rs = rsqrtf(row_sum(s2.x + s2.y, a.tpr, buf) / static_cast<float>(a.H) + a.eps);
  if (has(0) && t == 0 && a.rstd) a.rstd[row] = rs;
  const Pair rs2 = splat(rs);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * a.tpr + t) * 8;
    const bool in = has(c);
    Pair w[4];
    pairs_of(wq[j], w);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[j][k] = mul2(mul2(v[j][k], rs2), w[k]);
    if (a.y && in) *reinterpret_cast<uint4*>(a.y + off + c) = pack_pairs(v[j]);
    if (a.yq) mx_store8(v[j], a.yq, a.ys, off, off >> 5, c, in);
  }
}

struct NormBwdArgs {
  const void* h;
  const float* rstd;
  const uint16_t* w;
  const uint16_t* dy;
  const void* dres;
  void* dh;
  uint16_t* dx;
  float* part;  // [gridDim.x, H]
  int64_t T;
  int32_t H, tpr;
  DropArgs drop;
};

// The same layout, the grid striding over the rows, and the next row loaded while one is worked on (not at four
// vectors per thread: registers).  A row is kept as loaded and unpacked twice, before and after the row
// reduction.  Every thread sums dy xh of its columns over its rows in ascending order, the row groups
// of a block are added in ascending order at the end: one partial row of dweight per block.  (Rows copied ahead into
// shared memory by cp.async, for four blocks per SM instead of two, were slower: 59 against 57 us at
// 8192 x 4096 bf16 with dropout, 375 against 230 at 16384 x 7168 with an fp32 stream, both with dres in h's buffer.)
// KNOWN (see above) takes 4096 x 2048 bf16 with dropout from 19.2 to 17.1 us (dres in h's buffer; in its own 17.5 to
// 19.4 us, the more the further apart the calls' outputs are); with an fp32 stream or four vectors its registers do not
// suffice (16384 x 7168: 357 us against 289), so those never have it.
template <int V, bool F32, int MAXT, int MINB, int KNOWN>
__global__ void __launch_bounds__(MAXT, MINB) rmsnorm_bwd_kernel(const NormBwdArgs a) {
  constexpr bool FULL = KNOWN & kFull, STREAM = KNOWN & kStream;
  pdl_wait();
  __shared__ float buf[2][32];
  extern __shared__ float group_dw[];  // [rows, H] when the block holds several rows
  const int rows = static_cast<int>(blockDim.x) / a.tpr;
  const int rl = static_cast<int>(threadIdx.x) / a.tpr, t = static_cast<int>(threadIdx.x) - rl * a.tpr;
  const int64_t step = static_cast<int64_t>(gridDim.x) * rows, hop = step * a.H;
  int64_t r0 = static_cast<int64_t>(blockIdx.x) * rows, row = r0 + rl, off = row * a.H;
  constexpr bool kAhead = V < 4;
  struct Row {
    Vec8<F32> h[V], d[V];
    uint4 dy[V];
    float rs;
  } next;
  auto fetch = [&](int64_t at, int64_t rw) {
    if (rw >= a.T) return;  // past the end: nothing of it is used
    next.rs = __ldg(a.rstd + rw);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * a.tpr + t) * 8;
      if (FULL || c < a.H) {
        next.h[j].load(a.h, at + c);
        next.dy[j] = __ldcs(reinterpret_cast<const uint4*>(a.dy + at + c));
        if (STREAM || a.dres) next.d[j].load(a.dres, at + c);
      }
    }
  };
  if constexpr (kAhead) fetch(off, row);
  DropState ds;
  ds.load(a.drop);
  Pair dw[V][4];
  uint4 wq[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * a.tpr + t) * 8;
    wq[j] = FULL || c < a.H ? __ldg(reinterpret_cast<const uint4*>(a.w + c)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[j][k] = 0;
  }
  const Pair scale = splat(a.drop.scale);
  const float inv_h = 1.0f / static_cast<float>(a.H);
  for (int ph = 0; r0 < a.T; r0 += step, row += step, off += hop, ph ^= 1) {
    const bool live = FULL || row < a.T;
    if constexpr (!kAhead) fetch(off, row);
    const Row cur = next;
    if constexpr (kAhead) fetch(off + hop, row + step);
    Pair ss = 0;
    const Pair rs2 = splat(cur.rs);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * a.tpr + t) * 8;
      if (live && (FULL || c < a.H)) {
        Pair dy[4], xh[4], w[4];
        cur.h[j].get(xh);
        pairs_of(cur.dy[j], dy);
        pairs_of(wq[j], w);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          xh[k] = mul2(xh[k], rs2);
          dw[j][k] = fma2(dy[k], xh[k], dw[j][k]);
          ss = fma2(mul2(dy[k], w[k]), xh[k], ss);
        }
      }
    }
    const float2 s2 = floats_of(ss);
    const Pair c2 = splat(-row_sum(s2.x + s2.y, a.tpr, buf[ph]) * inv_h);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * a.tpr + t) * 8;
      if (live && (FULL || c < a.H)) {
        Pair g[4], xh[4], w[4], e[4];
        cur.h[j].get(xh);
        pairs_of(cur.dy[j], g);
        pairs_of(wq[j], w);
        if (STREAM || a.dres) {
          cur.d[j].get(e);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) e[k] = pair_of(0x80000000u, 0x80000000u);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) g[k] = fma2(fma2(mul2(xh[k], rs2), c2, mul2(g[k], w[k])), rs2, e[k]);
        if (STREAM || a.dh) Vec8<F32>::store(a.dh, off + c, g);
        if (STREAM || a.dx) {
          if (a.drop.rng) {
            uint32_t b[8], dr[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = floats_of(g[k]);
              b[2 * k] = __float_as_uint(f.x), b[2 * k + 1] = __float_as_uint(f.y);
            }
            philox8(ds, static_cast<uint64_t>(off + c) >> 3, dr);
            drop_bits(b, a.drop, dr);
#pragma unroll
            for (int k = 0; k < 4; ++k) g[k] = mul2(pair_of(b[2 * k], b[2 * k + 1]), scale);
          }
          *reinterpret_cast<uint4*>(a.dx + off + c) = pack_pairs(g);
        }
      }
    }
  }
  float* part = a.part + static_cast<int64_t>(blockIdx.x) * a.H;
  float* p = rows > 1 ? group_dw + rl * a.H : part;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * a.tpr + t) * 8;
    if (FULL || c < a.H) Vec8<true>::store(p, c, dw[j]);
  }
  if (rows > 1) {
    __syncthreads();
    for (int c = threadIdx.x; c < a.H; c += blockDim.x) {
      float v = group_dw[c];
      for (int i = 1; i < rows; ++i) v += group_dw[i * a.H + c];
      part[c] = v;
    }
  }
}

// dweight[c] = sum of the partial rows: block of 32 columns x 32 slices of the rows, each slice summed in
// ascending order, then the slices in ascending order.
__global__ void __launch_bounds__(1024) rmsnorm_dw_kernel(const float* __restrict__ part, int parts, int H,
                                                          float* __restrict__ dw) {
  pdl_wait();
  __shared__ float sm[32][33];
  const int c = static_cast<int>(blockIdx.x) * 32 + threadIdx.x;
  float s = 0.0f;
  if (c < H) {
#pragma unroll 10
    for (int p = threadIdx.y; p < parts; p += 32) s += part[static_cast<int64_t>(p) * H + c];
  }
  sm[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && c < H) {
    float r = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) r += sm[i][threadIdx.x];
    dw[c] = r;
  }
}

constexpr int kDropThreads = 256;

// Groups a thread holds at a time, and blocks per SM of the grid, which strides over the groups (0: one block
// for every 256 groups).  Measured at 16384 x 7168 values: forward bf16 108 us with two groups and four
// blocks, 112 to 118 with one group; fp32 stream 166 with one group and no stride, 182 to 215 with strides;
// backward 74.5 with one group and 32 blocks, 84 with two and eight.
template <bool F32, bool BWD>
constexpr int drop_unroll() { return !F32 && !BWD ? 2 : 1; }
template <bool F32, bool BWD>
constexpr int drop_blocks() { return BWD ? 32 : F32 ? 0 : 4; }

// Forward (BWD = false): out = residual + dropout(x).  Backward: out (bf16) = factors * x, x of the
// stream's type.  A thread loads its groups, draws, then uses them.
template <bool F32, bool BWD>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const void* x, const void* residual, void* out,
                                                               int64_t groups, DropArgs d) {
  constexpr int kU = drop_unroll<F32, BWD>();
  pdl_wait();
  DropState ds;
  ds.load(d);
  const Pair scale = splat(d.scale);
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kDropThreads * kU);
  for (int64_t g0 = static_cast<int64_t>(blockIdx.x) * (kDropThreads * kU) + threadIdx.x; g0 < groups;
       g0 += step) {
    Vec8<F32 && BWD> xq[kU];
    Vec8<F32> rq[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t g = g0 + u * kDropThreads;
      if (g < groups) {
        xq[u].load(x, 8 * g);
        if (!BWD && residual) rq[u].load(residual, 8 * g);
      }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int64_t g = g0 + u * kDropThreads;
      if (g >= groups) continue;
      uint32_t dr[4], b[8];
      if (d.rng) philox8(ds, static_cast<uint64_t>(g), dr);
      xq[u].bits(b);
      if (d.rng) drop_bits(b, d, dr);
      Pair v[4], r[4];
      if (!BWD && residual) {
        rq[u].get(r);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) r[k] = pair_of(0x80000000u, 0x80000000u);  // -0: v + -0 is v
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = fma2(pair_of(b[2 * k], b[2 * k + 1]), scale, r[k]);
      Vec8<F32 && !BWD>::store(out, 8 * g, v);
    }
  }
}

bool norm_shape_ok(const mok_norm_shape* s) {
  return s && s->T >= 0 && s->H >= 8 && s->H % 8 == 0 && s->H <= kNormMaxH &&
         (s->stream_type == MOK_DT_BF16 || s->stream_type == MOK_DT_FP32) && std::isfinite(s->eps) && s->eps >= 0.0f &&
         s->T <= (int64_t{1} << 40) / s->H;
}

// Threads per row (a power of two of lanes up to a warp, then whole warps), vectors of 8 per thread, rows per
// block of 256 threads or one row of more.  More values per thread mean fewer threads to reduce over and more
// loads in flight each, as long as the registers hold them: forward, bf16, H = 2048 with dropout, 4096
// rows: 13.0 us with one vector per thread, 10.0 with two; H = 7168, MXFP8, 16384 rows: 158 with two, 140 with
// four; H = 4096, 8192 rows: 40.4 with two, 41.1 with four; fp32 stream, H = 7168: 204 with two, 253 with four.
struct RowPlan {
  int tpr, v, rows;
  RowPlan(int H, bool four) {  // four: four vectors already from H > 4096 on
    v = H <= 1024 ? 1 : H <= (four ? 4096 : 16 * kNormThreads) ? 2 : 4;
    const int need = (H / 8 + v - 1) / v;
    tpr = (need + 31) / 32 * 32;
    if (need <= 16) tpr = need > 8 ? 16 : need > 4 ? 8 : 4;
    rows = tpr >= 256 ? 1 : 256 / tpr;
  }
  // Every thread of every block has v vectors of an existing row.
  bool full(const mok_norm_shape& s) const { return tpr * v * 8 == s.H && s.T % rows == 0; }
};

// Blocks of the backward, and partial rows of dweight: at most two blocks of 256 threads, or one of more, per SM of 152 (a
// function of the shape alone, which the workspace is sized by).
int norm_bwd_blocks(const mok_norm_shape& s) {
  const RowPlan p(s.H, false);
  const int64_t need = (s.T + p.rows - 1) / p.rows;
  const int64_t cap = p.tpr > 256 ? kNormParts / 2 : kNormParts;
  return static_cast<int>(need < cap ? need : cap);
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }

template <class F>
int with_row_kernel(const RowPlan& p, int32_t f32, F&& f) {
  auto typed = [&](auto v) { return f32 ? f(v, std::true_type{}) : f(v, std::false_type{}); };
  if (p.v == 1) return typed(std::integral_constant<int, 1>{});
  if (p.v == 2) return typed(std::integral_constant<int, 2>{});
  return typed(std::integral_constant<int, 4>{});
}

template <bool F32, bool BWD>
mok_status launch_dropout(const void* x, const void* residual, void* out, int64_t groups, const DropArgs& d,
                          void* stream) {
  const int sms = sm_count();
  if (sms <= 0) return MOK_ERR_CUDA;
  constexpr int kPer = kDropThreads * drop_unroll<F32, BWD>(), kBlocks = drop_blocks<F32, BWD>();
  const int64_t need = (groups + kPer - 1) / kPer;
  const int64_t cap = kBlocks ? static_cast<int64_t>(sms) * kBlocks : (int64_t{1} << 31) - 1;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  trace_begin(st, BWD ? K_DROPOUT_BWD : K_DROPOUT_FWD);
  const cudaError_t e = launch_pdl(dropout_kernel<F32, BWD>, dim3(static_cast<unsigned>(need < cap ? need : cap)),
                                   dim3(kDropThreads), 0, st, x, residual, out, groups, d);
  trace_end(st);
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}

template <bool BWD>
mok_status dropout_call(int64_t n, int32_t stream_type, const mok_dropout* drop, const void* x, const void* residual,
                        void* out, void* stream) {
  DropArgs d;
  if (n < 0 || n % 8 != 0 || (stream_type != MOK_DT_BF16 && stream_type != MOK_DT_FP32) || !drop ||
      !make_drop(drop, &d))
    return MOK_ERR_INVALID_ARG;
  if (n == 0) return MOK_OK;
  if (!x || !out || off16(x) || off16(out) || off16(residual)) return MOK_ERR_INVALID_ARG;
  return stream_type == MOK_DT_FP32 ? launch_dropout<true, BWD>(x, residual, out, n / 8, d, stream)
                                    : launch_dropout<false, BWD>(x, residual, out, n / 8, d, stream);
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

mok_status mok_dropout_forward(int64_t n, int32_t stream_type, const mok_dropout* drop, const void* x,
                               const void* residual, void* out, void* stream) {
  return dropout_call<false>(n, stream_type, drop, x, residual, out, stream);
}

mok_status mok_dropout_backward(int64_t n, int32_t stream_type, const mok_dropout* drop, const void* dout, void* dx,
                                void* stream) {
  return dropout_call<true>(n, stream_type, drop, dout, nullptr, dx, stream);
}

mok_status mok_rmsnorm_forward(const mok_norm_shape* s, const void* x, const void* residual, const mok_dropout* drop,
                               const void* weight, void* h, void* y, uint8_t* yq, uint8_t* ys, float* rstd,
                               void* stream) {
  NormFwdArgs a{};
  if (!norm_shape_ok(s) || !make_drop(drop, &a.drop)) return MOK_ERR_INVALID_ARG;
  if (s->T == 0) return MOK_OK;
  if ((!y && !yq) || (yq == nullptr) != (ys == nullptr) || (yq && s->H % 32 != 0)) return MOK_ERR_INVALID_ARG;
  if (!h && (residual || drop || s->stream_type != MOK_DT_BF16)) return MOK_ERR_INVALID_ARG;
  if (!x || !weight || off16(x) || off16(residual) || off16(weight) || off16(h) || off16(y) || off16(yq) ||
      (reinterpret_cast<uintptr_t>(rstd) & 3u))
    return MOK_ERR_INVALID_ARG;
  a.x = x;
  a.residual = residual;
  a.w = static_cast<const uint16_t*>(weight);
  a.h = h;
  a.y = static_cast<uint16_t*>(y);
  a.yq = yq;
  a.ys = ys;
  a.rstd = rstd;
  a.T = s->T;
  a.H = s->H;
  a.eps = s->eps;
  const RowPlan p(s->H, s->stream_type == MOK_DT_BF16);
  a.tpr = p.tpr;
  const int64_t blocks = (s->T + p.rows - 1) / p.rows;
  if (blocks >= (int64_t{1} << 31)) return MOK_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  trace_begin(st, K_RMSNORM_FWD);
  const int e = with_row_kernel(p, s->stream_type == MOK_DT_FP32, [&](auto v, auto f32) {
    constexpr int kV = decltype(v)::value;
    constexpr bool kF32 = decltype(f32)::value;
    auto run = [&](auto known) {
      constexpr int kBlocks = kV == 4 ? 4 : 5;  // blocks of 256 threads per SM: as many as its registers hold
      constexpr int kKnown = decltype(known)::value;
      const dim3 grid(static_cast<unsigned>(blocks)), block(p.tpr * p.rows);
      return static_cast<int>(p.tpr <= 256
                                  ? launch_pdl(rmsnorm_fwd_kernel<kV, kF32, 256, kBlocks, kKnown>, grid, block, 0, st, a)
                                  : launch_pdl(rmsnorm_fwd_kernel<kV, kF32, 512, 2, kKnown>, grid, block, 0, st, a));
    };
    const bool stream_there = residual && h;
    if (!p.full(*s)) return a.drop.rng ? run(Known<kDrop>{}) : run(Known<0>{});
    if (!stream_there) return a.drop.rng ? run(Known<kFull | kDrop>{}) : run(Known<kFull>{});
    return a.drop.rng ? run(Known<kFull | kStream | kDrop>{}) : run(Known<kFull | kStream>{});
  });
  trace_end(st);
  return e ? MOK_ERR_CUDA : MOK_OK;
}

size_t mok_rmsnorm_workspace_bytes(const mok_norm_shape* s) {
  if (!norm_shape_ok(s)) return 0;
  const size_t n = static_cast<size_t>(norm_bwd_blocks(*s)) * s->H * sizeof(float);
  return n < 256 ? 256 : (n + 255) / 256 * 256;
}

mok_status mok_rmsnorm_backward(const mok_norm_shape* s, const void* h, const float* rstd, const void* weight,
                                const void* dy, const void* dres, const mok_dropout* drop, void* dh, void* dx,
                                float* dweight, void* ws, size_t ws_bytes, void* stream) {
  NormBwdArgs a{};
  if (!norm_shape_ok(s) || !make_drop(drop, &a.drop) || !dweight || (reinterpret_cast<uintptr_t>(dweight) & 15u))
    return MOK_ERR_INVALID_ARG;
  if (!ws || (reinterpret_cast<uintptr_t>(ws) & 255u)) return MOK_ERR_INVALID_ARG;
  if (ws_bytes < mok_rmsnorm_workspace_bytes(s)) return MOK_ERR_WORKSPACE_TOO_SMALL;
  if (s->T > 0 && (!h || !rstd || !weight || !dy || off16(h) || (reinterpret_cast<uintptr_t>(rstd) & 3u) ||
                   off16(weight) || off16(dy) || off16(dres) || off16(dh) || off16(dx)))
    return MOK_ERR_INVALID_ARG;
  a.h = h;
  a.rstd = rstd;
  a.w = static_cast<const uint16_t*>(weight);
  a.dy = static_cast<const uint16_t*>(dy);
  a.dres = dres;
  a.dh = dh;
  a.dx = static_cast<uint16_t*>(dx);
  a.part = static_cast<float*>(ws);
  a.T = s->T;
  a.H = s->H;
  const RowPlan p(s->H, false);
  a.tpr = p.tpr;
  const int blocks = norm_bwd_blocks(*s);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (blocks > 0) {
    trace_begin(st, K_RMSNORM_BWD);
    const int e = with_row_kernel(p, s->stream_type == MOK_DT_FP32, [&](auto v, auto f32) {
      constexpr int kV = decltype(v)::value;
      constexpr bool kF32 = decltype(f32)::value;
      const dim3 grid(blocks), block(p.tpr * p.rows);
      const size_t smem = p.rows > 1 ? static_cast<size_t>(p.rows) * s->H * sizeof(float) : 0;
      auto run = [&](auto known) {
        constexpr int kKnown = decltype(known)::value;
        return static_cast<int>(
            p.tpr <= 256 ? launch_pdl(rmsnorm_bwd_kernel<kV, kF32, 256, 2, kKnown>, grid, block, smem, st, a)
                         : launch_pdl(rmsnorm_bwd_kernel<kV, kF32, 512, 1, kKnown>, grid, block, smem, st, a));
      };
      if constexpr (!kF32 && kV <= 2) {
        if (p.full(*s) && dres && dh && dx) return run(Known<kFull | kStream>{});
      }
      return run(Known<0>{});
    });
    trace_end(st);
    if (e) return MOK_ERR_CUDA;
  }
  trace_begin(st, K_RMSNORM_DW);
  const cudaError_t e = launch_pdl(rmsnorm_dw_kernel, dim3((s->H + 31) / 32), dim3(32, 32), 0, st,
                                   static_cast<const float*>(a.part), blocks, static_cast<int>(s->H), dweight);
  trace_end(st);
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}

}  // extern "C"
