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
#include <cmath>
#include <type_traits>

#include "mok_internal.cuh"
#include "mok_philox.cuh"
#include "mok_ptx.cuh"

namespace mok {
namespace {

constexpr int kNormMaxH = 16384;
constexpr int kNormThreads = 512;  // most threads of a block
constexpr int kNormParts = 608;  // most partial dweight rows: four CTAs on each of 152 SMs

__device__ __forceinline__ void unpack_bf16x8(uint4 q, float (&v)[8]) {
  v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
  v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
}
__device__ __forceinline__ uint4 pack_bf16x8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
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
  __device__ __forceinline__ void get(float (&v)[8]) const { unpack_bf16x8(q, v); }
  // stores v and leaves in v what the stored values read back as
  static __device__ __forceinline__ void store(void* p, int64_t i, float (&v)[8]) {
    const uint4 q = pack_bf16x8(v);
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i) = q;
    unpack_bf16x8(q, v);
  }
  static __device__ __forceinline__ void rounded(float (&v)[8]) { unpack_bf16x8(pack_bf16x8(v), v); }
};
template <>
struct Vec8<true> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
    a = __ldcs(s);
    b = __ldcs(s + 1);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  static __device__ __forceinline__ void store(void* p, int64_t i, float (&v)[8]) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
    d[0] = make_float4(v[0], v[1], v[2], v[3]);
    d[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
  static __device__ __forceinline__ void rounded(float (&)[8]) {}
};

// Sum over the threads of one row (tpr of them, whole warps; a block holds blockDim.x / tpr rows), in
// a fixed order: a butterfly within each warp, then the warps' sums in ascending order.  Every thread
// gets it.  All threads of the block call it; `buf` (32 words) may be used again after the next call's
// first barrier, so two calls in a row need two buffers.
__device__ __forceinline__ float row_sum(float v, int tpr, float* buf) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
  if (tpr == 32) return v;  // the same for the whole grid
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

// MXFP8 of the 32 values held by four neighbouring lanes (8 each): shared = floor(log2 max) - 8,
// clamped at -127; codes E4M3 of v 2^-shared, saturating; a block with an Inf or a NaN gets scale 0xFF
// and codes 0x7F.
__device__ __forceinline__ void mx_store8(const float (&v)[8], uint8_t* q, uint8_t* s, int64_t row, int H, int c) {
  float m = fmax_abs_nan(fmax_abs_nan(fmax_abs_nan(v[0], v[1]), fmax_abs_nan(v[2], v[3])),
                         fmax_abs_nan(fmax_abs_nan(v[4], v[5]), fmax_abs_nan(v[6], v[7])));
  m = fmax_abs_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = fmax_abs_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const uint32_t amax = __float_as_uint(m) & 0x7FFFFFFFu;
  if (c >= H) return;  // after the shuffles
  const bool bad = amax > 0x7F7FFFFFu;
  int shared = static_cast<int>(amax >> 23) - 127 - 8;
  shared = shared < -127 ? -127 : shared;
  const float dn = pow2f(bad ? 0 : -shared);
  uint16_t e[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(e[j]) : "f"(v[2 * j + 1] * dn), "f"(v[2 * j] * dn));
  uint2 o = make_uint2(e[0] | static_cast<uint32_t>(e[1]) << 16, e[2] | static_cast<uint32_t>(e[3]) << 16);
  if (bad) o = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  *reinterpret_cast<uint2*>(q + row * H + c) = o;
  if ((c & 31) == 0) s[row * (H / 32) + c / 32] = static_cast<uint8_t>(bad ? 0xFF : shared + 127);
}

// Block = blockDim.x / tpr rows of tpr threads; thread t of a row holds vectors t, t + tpr, ...
template <int V, bool F32>
__global__ void __launch_bounds__(kNormThreads) rmsnorm_fwd_kernel(const NormFwdArgs a) {
  pdl_wait();
  __shared__ float buf[32];
  const int rl = static_cast<int>(threadIdx.x) / a.tpr, t = static_cast<int>(threadIdx.x) - rl * a.tpr;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (blockDim.x / a.tpr) + rl;
  const bool live = row < a.T;
  const int64_t base = row * a.H;
  float v[V][8];
  uint4 xq[V];
  Vec8<F32> rq[V];
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * a.tpr + t) * 8;
    if (live && c < a.H) {
      xq[j] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + base + c));
      if (a.residual) rq[j].load(a.residual, base + c);
    }
  }
  uint64_t seed = 0, offset = 0;
  if (a.drop.rng) seed = a.drop.rng[0], offset = a.drop.rng[1];
  float ss = 0.0f;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * a.tpr + t) * 8;
#pragma unroll
    for (int k = 0; k < 8; ++k) v[j][k] = 0.0f;
    if (live && c < a.H) {
      unpack_bf16x8(xq[j], v[j]);
      if (a.drop.rng) drop8(v[j], a.drop, seed, offset, static_cast<uint64_t>(base + c) >> 3);
      if (a.residual) {
        float r[8];
        rq[j].get(r);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] += r[k];
      }
      if (a.h) Vec8<F32>::store(a.h, base + c, v[j]);
#pragma unroll
      for (int k = 0; k < 8; ++k) ss = fmaf(v[j][k], v[j][k], ss);
    }
  }
  ss = row_sum(ss, a.tpr, buf);
  const float r = rsqrtf(ss / static_cast<float>(a.H) + a.eps);
  if (live && t == 0 && a.rstd) a.rstd[row] = r;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * a.tpr + t) * 8;
    const bool in = live && c < a.H;
    if (in) {
      float w[8];
      unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(a.w + c)), w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] = v[j][k] * r * w[k];
      if (a.y) *reinterpret_cast<uint4*>(a.y + base + c) = pack_bf16x8(v[j]);
    }
    if (a.yq) mx_store8(v[j], a.yq, a.ys, row, a.H, in ? c : a.H);
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
  float* part;  // [parts, H]
  int64_t T;
  int32_t H, tpr;
  DropArgs drop;
};

// The same layout; the grid strides over the rows and every thread sums dy xh of its columns over its
// rows in ascending order: one partial row of dweight per row group (blockIdx, rl).
template <int V, bool F32>
__global__ void __launch_bounds__(kNormThreads) rmsnorm_bwd_kernel(const NormBwdArgs a) {
  pdl_wait();
  __shared__ float buf[2][32];
  const int rows = static_cast<int>(blockDim.x) / a.tpr;
  const int rl = static_cast<int>(threadIdx.x) / a.tpr, t = static_cast<int>(threadIdx.x) - rl * a.tpr;
  float dw[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[j][k] = 0.0f;
  uint64_t seed = 0, offset = 0;
  if (a.drop.rng) seed = a.drop.rng[0], offset = a.drop.rng[1];
  int ph = 0;
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * rows; r0 < a.T;
       r0 += static_cast<int64_t>(gridDim.x) * rows, ph ^= 1) {
    const int64_t row = r0 + rl;
    const bool live = row < a.T;
    const int64_t base = row * a.H;
    const float rs = live ? a.rstd[row] : 0.0f;
    float g[V][8], xh[V][8];
    uint4 dyq[V];
    Vec8<F32> hq[V], dq[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * a.tpr + t) * 8;
      if (live && c < a.H) {
        hq[j].load(a.h, base + c);
        dyq[j] = __ldcs(reinterpret_cast<const uint4*>(a.dy + base + c));
        if (a.dres) dq[j].load(a.dres, base + c);
      }
    }
    float s = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * a.tpr + t) * 8;
      if (live && c < a.H) {
        float w[8];
        unpack_bf16x8(__ldg(reinterpret_cast<const uint4*>(a.w + c)), w);
        hq[j].get(xh[j]);
        unpack_bf16x8(dyq[j], g[j]);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          xh[j][k] *= rs;
          dw[j][k] = fmaf(g[j][k], xh[j][k], dw[j][k]);
          g[j][k] *= w[k];
          s = fmaf(g[j][k], xh[j][k], s);
        }
      }
    }
    s = row_sum(s, a.tpr, buf[ph]) / static_cast<float>(a.H);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * a.tpr + t) * 8;
      if (live && c < a.H) {
        float d[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) d[k] = rs * fmaf(-xh[j][k], s, g[j][k]);
        if (a.dres) {
          float e[8];
          dq[j].get(e);
#pragma unroll
          for (int k = 0; k < 8; ++k) d[k] += e[k];
        }
        if (a.dx) {
          float e[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) e[k] = d[k];
          if (a.drop.rng) drop8(e, a.drop, seed, offset, static_cast<uint64_t>(base + c) >> 3);
          *reinterpret_cast<uint4*>(a.dx + base + c) = pack_bf16x8(e);
        }
        if (a.dh) Vec8<F32>::store(a.dh, base + c, d);
      }
    }
  }
  float* p = a.part + (static_cast<int64_t>(blockIdx.x) * rows + rl) * a.H;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * a.tpr + t) * 8;
    if (c < a.H) {
      float4* d = reinterpret_cast<float4*>(p + c);
      d[0] = make_float4(dw[j][0], dw[j][1], dw[j][2], dw[j][3]);
      d[1] = make_float4(dw[j][4], dw[j][5], dw[j][6], dw[j][7]);
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
#pragma unroll 4
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

constexpr int kDropThreads = 256, kDropUnroll = 2;

// Forward (BWD = false): out = residual + dropout(x).  Backward: out (bf16) = factors * x, x of the
// stream's type.
template <bool F32, bool BWD>
__global__ void __launch_bounds__(kDropThreads) dropout_kernel(const void* x, const void* residual, void* out,
                                                               int64_t groups, DropArgs d) {
  pdl_wait();
  const uint64_t seed = d.rng[0], offset = d.rng[1];
  const int64_t step = static_cast<int64_t>(gridDim.x) * (kDropThreads * kDropUnroll);
  for (int64_t g0 = static_cast<int64_t>(blockIdx.x) * (kDropThreads * kDropUnroll) + threadIdx.x; g0 < groups;
       g0 += step) {
    Vec8<F32 && BWD> xq[kDropUnroll];
    Vec8<F32> rq[kDropUnroll];
#pragma unroll
    for (int u = 0; u < kDropUnroll; ++u) {
      const int64_t g = g0 + u * kDropThreads;
      if (g < groups) {
        xq[u].load(x, 8 * g);
        if (!BWD && residual) rq[u].load(residual, 8 * g);
      }
    }
#pragma unroll
    for (int u = 0; u < kDropUnroll; ++u) {
      const int64_t g = g0 + u * kDropThreads;
      if (g >= groups) continue;
      float v[8];
      xq[u].get(v);
      drop8(v, d, seed, offset, static_cast<uint64_t>(g));
      if (!BWD && residual) {
        float r[8];
        rq[u].get(r);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += r[k];
      }
      Vec8<F32 && !BWD>::store(out, 8 * g, v);
    }
  }
}

bool norm_shape_ok(const mok_norm_shape* s) {
  return s && s->T >= 0 && s->H >= 8 && s->H % 8 == 0 && s->H <= kNormMaxH &&
         (s->stream_type == MOK_DT_BF16 || s->stream_type == MOK_DT_FP32) && std::isfinite(s->eps) && s->eps >= 0.0f &&
         s->T <= (int64_t{1} << 40) / s->H;
}

// Threads per row (whole warps), vectors of 8 per thread, rows per block.
struct RowPlan {
  int tpr, v, rows;
  RowPlan(int H) {
    v = H <= 2048 ? 1 : H <= 16 * kNormThreads ? 2 : 4;
    tpr = ((H / 8 + v - 1) / v + 31) / 32 * 32;
    rows = tpr >= 256 ? 1 : 256 / tpr;
  }
};

int norm_bwd_blocks(const mok_norm_shape& s) {
  const RowPlan p(s.H);
  const int64_t need = (s.T + p.rows - 1) / p.rows;
  const int64_t cap = kNormParts / p.rows > 0 ? kNormParts / p.rows : 1;
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

template <bool BWD>
mok_status dropout_call(int64_t n, int32_t stream_type, const mok_dropout* drop, const void* x, const void* residual,
                        void* out, void* stream) {
  DropArgs d;
  if (n < 0 || n % 8 != 0 || (stream_type != MOK_DT_BF16 && stream_type != MOK_DT_FP32) || !drop ||
      !make_drop(drop, &d))
    return MOK_ERR_INVALID_ARG;
  if (n == 0) return MOK_OK;
  if (!x || !out || off16(x) || off16(out) || off16(residual)) return MOK_ERR_INVALID_ARG;
  const int sms = sm_count();
  if (sms <= 0) return MOK_ERR_CUDA;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t groups = n / 8, per = kDropThreads * kDropUnroll, need = (groups + per - 1) / per;
  const int64_t cap = static_cast<int64_t>(sms) * 8;
  const dim3 grid(static_cast<unsigned>(need < cap ? need : cap));
  trace_begin(st, BWD ? K_DROPOUT_BWD : K_DROPOUT_FWD);
  const cudaError_t e =
      stream_type == MOK_DT_FP32
          ? launch_pdl(dropout_kernel<true, BWD>, grid, dim3(kDropThreads), 0, st, x, residual, out, groups, d)
          : launch_pdl(dropout_kernel<false, BWD>, grid, dim3(kDropThreads), 0, st, x, residual, out, groups, d);
  trace_end(st);
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
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
  const RowPlan p(s->H);
  a.tpr = p.tpr;
  const int64_t blocks = (s->T + p.rows - 1) / p.rows;
  if (blocks >= (int64_t{1} << 31)) return MOK_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  trace_begin(st, K_RMSNORM_FWD);
  const int e = with_row_kernel(p, s->stream_type == MOK_DT_FP32, [&](auto v, auto f32) {
    return static_cast<int>(launch_pdl(rmsnorm_fwd_kernel<decltype(v)::value, decltype(f32)::value>,
                                       dim3(static_cast<unsigned>(blocks)), dim3(p.tpr * p.rows), 0, st, a));
  });
  trace_end(st);
  return e ? MOK_ERR_CUDA : MOK_OK;
}

size_t mok_rmsnorm_workspace_bytes(const mok_norm_shape* s) {
  if (!norm_shape_ok(s)) return 0;
  const size_t n = static_cast<size_t>(norm_bwd_blocks(*s)) * RowPlan(s->H).rows * s->H * sizeof(float);
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
  const RowPlan p(s->H);
  a.tpr = p.tpr;
  const int blocks = norm_bwd_blocks(*s);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (blocks > 0) {
    trace_begin(st, K_RMSNORM_BWD);
    const int e = with_row_kernel(p, s->stream_type == MOK_DT_FP32, [&](auto v, auto f32) {
      return static_cast<int>(launch_pdl(rmsnorm_bwd_kernel<decltype(v)::value, decltype(f32)::value>, dim3(blocks),
                                         dim3(p.tpr * p.rows), 0, st, a));
    });
    trace_end(st);
    if (e) return MOK_ERR_CUDA;
  }
  trace_begin(st, K_RMSNORM_DW);
  const cudaError_t e = launch_pdl(rmsnorm_dw_kernel, dim3((s->H + 31) / 32), dim3(32, 32), 0, st,
                                   static_cast<const float*>(a.part), blocks * p.rows, static_cast<int>(s->H), dweight);
  trace_end(st);
  return e == cudaSuccess ? MOK_OK : MOK_ERR_CUDA;
}

}  // extern "C"
