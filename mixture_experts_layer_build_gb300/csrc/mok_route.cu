// mok_route.cu -- routed rows as calls of their own: dispatch, combine and their gradients.
//
//   dispatch            rows[r] = x[token(r)], 0 on padding                   (the layer's gather kernel)
//   dispatch, backward  dx[t] = sum_k drows[inv[t,k]]                         (the layer's dX reduction)
//   combine             out[t] = sum_k s[t,k] rows[inv[t,k]]                  (the layer's combine kernel)
//   combine, backward   drows[inv[t,k]] = s[t,k] dout[t], 0 on padding; ds[t,k] = <dout[t], rows[inv[t,k]]>
//
// All of them move each row once: bound by HBM.  Measured at T = 8192, K = 8, E = 128, width 4096: combine 101 us (5,950 GB/s),
// its backward 202 (1.14 GB that it cannot do without, and 67 MB of zeroed padding: 5,980 GB/s); combine of 4096 tokens, K = 6,
// width 2048 20.9 us (5,640).
#include "mok_internal.cuh"
#include "mok_ptx.cuh"
#include "mok_route.cuh"

namespace mok {
namespace {

constexpr int kRouteThreads = 256;

// The gradient of combine.  A CTA takes a token: its threads hold that row of dout (read once, VECS 16-byte vectors each),
// and for each of the token's slots read the expert's row, write the gradient's, and add up the dot product -- each
// thread its own columns in ascending order, then a tree over the CTA: one fixed order.  Padding rows are dealt out
// over all CTAs and zeroed, as in the layer's gather.  With drows in rows' own buffer a thread has read a vector
// before it writes that vector.  `parts` CTAs share a token's slots: with few tokens one by one they are a chain of
// latencies (16 tokens, K = 8, E = 128, width 4096 31.8 us with one part).
template <int VECS>
__global__ void __launch_bounds__(kRouteThreads) combine_backward_kernel(
    const uint4* rows, const uint4* __restrict__ dout, const int32_t* __restrict__ inv, const float* __restrict__ s,
    const int32_t* __restrict__ row_token, const int32_t* __restrict__ meta, int64_t T, int K, int parts, int vecs,
    uint4* drows, float* __restrict__ ds) {
  pdl_wait();
  __shared__ float warp_dot[2][kRouteThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int buf = 0;
  for (int64_t i = blockIdx.x; i < T * parts; i += gridDim.x) {
    int64_t t = i;
    int k = 0, k_end = K;
    if (parts > 1) {  // (divisions that a token of its own need not wait for)
      t = i / parts;
      const int part = static_cast<int>(i - t * parts);
      k = K * part / parts;
      k_end = K * (part + 1) / parts;
    }
    uint4 d[VECS];
#pragma unroll
    for (int u = 0; u < VECS; ++u) {
      const int c = threadIdx.x + u * kRouteThreads;
      d[u] = c < vecs ? __ldcs(dout + t * vecs + c) : make_uint4(0, 0, 0, 0);
    }
    for (; k < k_end; ++k) {
      const int64_t j = t * K + k;
      const int row = __ldg(inv + j);
      const float w = __ldg(s + j);
      float dot = 0.0f;
      if (row >= 0) {
        const uint4* src = rows + static_cast<int64_t>(row) * vecs;
        uint4* dst = drows + static_cast<int64_t>(row) * vecs;
        uint4 v[VECS];
#pragma unroll
        for (int u = 0; u < VECS; ++u) {
          const int c = threadIdx.x + u * kRouteThreads;
          v[u] = c < vecs ? __ldcs(src + c) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < VECS; ++u) {
          const int c = threadIdx.x + u * kRouteThreads;
          const uint32_t a[4] = {v[u].x, v[u].y, v[u].z, v[u].w}, b[4] = {d[u].x, d[u].y, d[u].z, d[u].w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = bf16_lo(b[i]), hi = bf16_hi(b[i]);
            dot = fmaf(lo, bf16_lo(a[i]), dot);
            dot = fmaf(hi, bf16_hi(a[i]), dot);
            o[i] = pack_bf16x2(w * lo, w * hi);
          }
          if (c < vecs) __stcs(dst + c, make_uint4(o[0], o[1], o[2], o[3]));
        }
      }
#pragma unroll
      for (int x = 16; x >= 1; x >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, x);
      if (lane == 0) warp_dot[buf][warp] = dot;
      __syncthreads();  // (two buffers: a warp that is a slot ahead writes the other one)
      if (threadIdx.x == 0) {
        float sum = 0.0f;
#pragma unroll
        for (int w8 = 0; w8 < kRouteThreads / 32; ++w8) sum += warp_dot[buf][w8];
        ds[j] = sum;
      }
      buf ^= 1;
    }
  }
  const int64_t rpad = meta[0], nwarps = static_cast<int64_t>(gridDim.x) * (kRouteThreads / 32);
  const uint4 z = make_uint4(0, 0, 0, 0);
  for (int64_t r0 = static_cast<int64_t>(blockIdx.x) * (kRouteThreads / 32) + warp; r0 < rpad; r0 += 32 * nwarps) {
    const int64_t r = r0 + lane * nwarps;
    const bool pad = r < rpad && __ldg(row_token + r) < 0;
    for (unsigned m = __ballot_sync(0xffffffffu, pad); m; m &= m - 1) {
      uint4* q = drows + (r0 + static_cast<int64_t>(__ffs(m) - 1) * nwarps) * vecs;
      for (int c = lane; c < vecs; c += 32) __stcs(q + c, z);
    }
  }
}

constexpr int kMaxVecs = 8;  // 16-byte vectors of a row per thread: rows of up to 16384 values

int launch_combine_backward(const Sizes& z, const mok_schedule& s, const void* rows, const void* dout, int32_t width,
                            void* drows, float* ds, cudaStream_t stream) {
  const int vecs = width / 8, per = (vecs + kRouteThreads - 1) / kRouteThreads;
  const int sms = sm_count();
  if (sms <= 0) return static_cast<int>(cudaErrorInvalidDevice);
  // parts of a token: as many as it takes to have four CTAs per SM, and as it has slots
  const int64_t parts64 = z.T > 0 ? (4 * static_cast<int64_t>(sms) + z.T - 1) / z.T : 1;
  const int parts = static_cast<int>(parts64 < z.K ? (parts64 > 0 ? parts64 : 1) : z.K);
  const int64_t items = z.T * parts, pads = ((z.E < z.R ? z.E : z.R) * 127 + 7) / 8, zero = pads < 4 * sms ? pads : 4 * sms,
                want = items > zero ? items : zero;  // CTAs: a padding row per warp, up to four of them per SM
  const int grid = static_cast<int>(want < 8 * sms ? want : 8 * sms);
  if (grid <= 0) return 0;
  trace_begin(stream, K_COMBINE_BWD);
  cudaError_t e = cudaErrorInvalidValue;
  auto run = [&](auto kernel) {
    e = launch_pdl(kernel, dim3(grid), dim3(kRouteThreads), 0, stream, static_cast<const uint4*>(rows),
                   static_cast<const uint4*>(dout), static_cast<const int32_t*>(s.inv), s.topk_weights,
                   static_cast<const int32_t*>(s.row_token), static_cast<const int32_t*>(s.meta), z.T, z.K, parts, vecs,
                   static_cast<uint4*>(drows), ds);
  };
  if (per <= 1) run(combine_backward_kernel<1>);
  else if (per <= 2) run(combine_backward_kernel<2>);
  else if (per <= 4) run(combine_backward_kernel<4>);
  else if (per <= kMaxVecs) run(combine_backward_kernel<kMaxVecs>);
  trace_end(stream);
  return static_cast<int>(e);
}

}  // namespace

mok_status routed_sizes(const mok_schedule* s, Sizes* z) {
  if (!s || !make_sizes(&s->config, &s->shape, z)) return MOK_ERR_INVALID_ARG;
  if (!s->counts || !s->poff || !s->inv || !s->mblocks || !s->meta || !s->row_token || s->rpad_max != z->rpad_max ||
      s->mblocks_max != z->mblocks_max)
    return MOK_ERR_INVALID_ARG;
  return MOK_OK;
}

bool apart_from_tables(const mok_schedule& s, const Sizes& z, const void* out, int64_t n) {
  return apart(out, n, s.counts, 4 * static_cast<int64_t>(z.E)) && apart(out, n, s.poff, 4 * (static_cast<int64_t>(z.E) + 1)) &&
         apart(out, n, s.inv, 4 * z.R) && apart(out, n, s.mblocks, 16 * z.mblocks_max) && apart(out, n, s.meta, 4 * 16) &&
         apart(out, n, s.row_token, 4 * z.rpad_max);
}

namespace {
bool ok16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
mok_status from_cuda(int rc) { return rc == 0 ? MOK_OK : MOK_ERR_CUDA; }
constexpr int32_t kMaxWidth = kMaxVecs * kRouteThreads * 8;  // 16384
// Bytes of a bf16 tensor of tokens, and of routed rows.
int64_t token_bytes(const Sizes& z, int32_t w) { return z.T * w * 2; }
int64_t row_bytes(const Sizes& z, int32_t w) { return z.rpad_max * w * 2; }
bool width_ok(int32_t w) { return w >= 8 && w % 8 == 0 && w <= kMaxWidth; }
}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

mok_status mok_dispatch(const mok_schedule* sched, const void* x, int32_t width, void* rows, void* stream) {
  Sizes z;
  const mok_status rc = routed_sizes(sched, &z);
  if (rc != MOK_OK) return rc;
  if (!width_ok(width)) return MOK_ERR_INVALID_ARG;
  if (z.T == 0) return MOK_OK;
  if (!ok16(x) || !ok16(rows) || !apart(x, token_bytes(z, width), rows, row_bytes(z, width)) ||
      !apart_from_tables(*sched, z, rows, row_bytes(z, width)))
    return MOK_ERR_INVALID_ARG;
  return from_cuda(launch_gather_rows(plain_rows(x), sched->inv, sched->row_token, sched->meta, z.T, z.K, z.rpad_max, width,
                                      static_cast<uint16_t*>(rows), K_DISPATCH, static_cast<cudaStream_t>(stream)));
}

mok_status mok_dispatch_backward(const mok_schedule* sched, const void* drows, int32_t width, void* dx, void* stream) {
  Sizes z;
  const mok_status rc = routed_sizes(sched, &z);
  if (rc != MOK_OK) return rc;
  if (!width_ok(width)) return MOK_ERR_INVALID_ARG;
  if (z.T == 0) return MOK_OK;
  if (!ok16(drows) || !ok16(dx) || !apart(dx, token_bytes(z, width), drows, row_bytes(z, width)) ||
      !apart_from_tables(*sched, z, dx, token_bytes(z, width)))
    return MOK_ERR_INVALID_ARG;
  return from_cuda(launch_combine(static_cast<const uint16_t*>(drows), sched->inv, nullptr, z.T, z.K, width,
                                  static_cast<uint16_t*>(dx), K_DISPATCH_BWD, static_cast<cudaStream_t>(stream)));
}

mok_status mok_combine(const mok_schedule* sched, const void* rows, int32_t width, void* out, void* stream) {
  Sizes z;
  const mok_status rc = routed_sizes(sched, &z);
  if (rc != MOK_OK) return rc;
  if (!width_ok(width)) return MOK_ERR_INVALID_ARG;
  if (z.T == 0) return MOK_OK;
  if (!ok16(rows) || !ok16(out) || !sched->topk_weights) return MOK_ERR_INVALID_ARG;
  if (!apart(out, token_bytes(z, width), rows, row_bytes(z, width)) ||
      !apart(out, token_bytes(z, width), sched->topk_weights, z.R * 4) ||
      !apart_from_tables(*sched, z, out, token_bytes(z, width)))
    return MOK_ERR_INVALID_ARG;
  return from_cuda(launch_combine(static_cast<const uint16_t*>(rows), sched->inv, sched->topk_weights, z.T, z.K, width,
                                  static_cast<uint16_t*>(out), K_ROUTE_COMBINE, static_cast<cudaStream_t>(stream)));
}

mok_status mok_combine_backward(const mok_schedule* sched, const void* rows, const void* dout, int32_t width, void* drows,
                                float* d_topk_weights, void* stream) {
  Sizes z;
  const mok_status rc = routed_sizes(sched, &z);
  if (rc != MOK_OK) return rc;
  if (!width_ok(width)) return MOK_ERR_INVALID_ARG;
  if (z.T == 0) return MOK_OK;
  if (!ok16(rows) || !ok16(dout) || !ok16(drows) || !d_topk_weights || !sched->topk_weights) return MOK_ERR_INVALID_ARG;
  const int64_t nr = row_bytes(z, width), nt = token_bytes(z, width), nw = z.R * 4;
  if ((drows != rows && !apart(drows, nr, rows, nr)) || !apart(drows, nr, dout, nt) || !apart(d_topk_weights, nw, rows, nr) ||
      !apart(d_topk_weights, nw, dout, nt) || !apart(d_topk_weights, nw, drows, nr) ||
      !apart(d_topk_weights, nw, sched->topk_weights, nw) || !apart(drows, nr, sched->topk_weights, nw) ||
      !apart_from_tables(*sched, z, drows, nr) || !apart_from_tables(*sched, z, d_topk_weights, nw))
    return MOK_ERR_INVALID_ARG;
  return from_cuda(launch_combine_backward(z, *sched, rows, dout, width, drows, d_topk_weights,
                                           static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
