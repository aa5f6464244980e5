// mok_fp8_quant.cu -- quantisation to E4M3 with one fp32 scale per block of 128 (mok_fp8.cuh).
//
// One kernel makes every form from tiles of 128 x 128 bf16 values that stay in registers: 256 threads, each with
// 8 rows x 8 columns as packed pairs.  16 neighbouring lanes hold a row's 128 columns: its maximum is four shuffles.
// A column's maximum is a lane's own over its 8 rows, one shuffle, and one exchange over the warps in shared memory; a
// 128 x 128 block's comes from the row maxima.  Each form then converts from the same registers: row codes leave as 8
// bytes per lane, 128 contiguous ones per row; transposed codes go through shared memory (8 rows of a column are
// 8 bytes of a transposed row) and leave as 16-byte vectors.
//
// Bound by HBM: 2 bytes read, 1 written per value and form.  Measured: 8192 x 4096 rows alone 15.3 us (6,570 GB/s), transposed
// alone 16.7 (6,010), both 24.5 (5,470); 64 weights of 1024 x 2048 both ways 82 us (6,540); routed rows gathered from 4096 tokens (top-6,
// 64 experts, 2048 wide) both ways 36.6, where each token's row is read six times from L2.  (The transposed codes in
// rows padded by 16 bytes, whose stores met in one bank, 8192 x 4096 both ways took 34.7; a division per row, column and thread and
// four shuffles per row 40.)
#include "mok_ffn.cuh"  // pdl_trigger
#include "mok_fp8.cuh"

namespace mok {
namespace {

constexpr int kQThreads = 256;

enum QuantForm : int { Q_ROWS = 1, Q_COLS = 2, Q_BLOCKS = 4 };

struct QuantArgs {
  Fp8Source src;
  int64_t rows;
  int32_t cols;
  uint8_t* q;
  float* s;
  uint8_t* qt;
  float* st;
  int64_t ld, ldt, pitch, pitch_t;
  int64_t src_batch, q_batch, s_batch, qt_batch, st_batch;  // Q_BLOCKS: elements between matrices
};

__device__ __forceinline__ uint32_t absmax_word(uint32_t m) { return absmax2(m, m >> 16) & 0x7FFFu; }

// FORM: Q_ROWS | Q_COLS for 1 x 128 scales of rows and of columns, or Q_BLOCKS (q, qt as they are not null).
template <int FORM, bool GATHER>
__global__ void __launch_bounds__(kQThreads) fp8_quantize_kernel(const QuantArgs p) {
  pdl_wait();
  pdl_trigger();  // a product that follows sets itself up, and loads weights, meanwhile
  __shared__ uint32_t wmax[8][64];                                // per warp, packed column maxima
  __shared__ __align__(16) float col_up[FORM & Q_COLS ? 128 : 4];
  __shared__ __align__(16) uint8_t tile[FORM == Q_ROWS ? 16 : 128 * 128];
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, cg = t & 15, rg = t >> 4;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * 128;
  const int c0 = static_cast<int>(blockIdx.x) * 128, c = c0 + cg * 8;
  const bool routed = p.src.row_token != nullptr;
  if (routed && r0 >= p.src.meta[0]) return;  // (segments, and so the layout's end, are multiples of 128 rows)
  const uint16_t* x = p.src.x + (FORM == Q_BLOCKS ? blockIdx.z * p.src_batch : 0);
  uint4 v[8];
  uint32_t live = 0;  // rows that are there, and no padding
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int64_t r = r0 + rg * 8 + i;
    int64_t from = r;
    bool in = r < p.rows;
    if (routed && in) {
      const int token = __ldg(p.src.row_token + r);
      in = token >= 0;
      if (GATHER) from = token;
    }
    live |= in ? 1u << i : 0u;
    v[i] = in && c < p.cols ? *reinterpret_cast<const uint4*>(x + from * p.cols + c) : make_uint4(0, 0, 0, 0);
  }
  // The rows' maxima over the 16 lanes that hold a row, halving the rows that a lane keeps at each exchange: lanes 2 i and
  // 2 i + 1 of the 16 end with row i's.
  uint32_t rmax = 0;
  if constexpr (FORM != Q_COLS) {
    uint32_t m[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = absmax2(absmax2(v[i].x, v[i].y), absmax2(v[i].z, v[i].w));
#pragma unroll
    for (int d = 8, h = 4; d >= 2; d >>= 1, h >>= 1) {
      const bool hi = cg & d;
#pragma unroll
      for (int i = 0; i < h; ++i) m[i] = absmax2(hi ? m[i + h] : m[i], __shfl_xor_sync(0xffffffffu, hi ? m[i] : m[i + h], d));
    }
    rmax = absmax_word(absmax2(m[0], __shfl_xor_sync(0xffffffffu, m[0], 1)));
  }
  float up = 0.0f;
  bool bad = false;
  if constexpr (FORM == Q_BLOCKS) {
    uint32_t m = rmax;
#pragma unroll
    for (int d = 16; d >= 2; d >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, d));  // (magnitudes' bits order as they do)
    if (lane == 0) wmax[warp][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, wmax[w][0]);
    const float sc = fp8_scale(m, up);
    bad = m >= 0x7F80u;
    if (t == 0) {
      if (p.q) p.s[blockIdx.z * p.s_batch + static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x] = sc;
      if (p.qt) p.st[blockIdx.z * p.st_batch + static_cast<int64_t>(blockIdx.x) * gridDim.y + blockIdx.y] = sc;
    }
  }
  auto row_codes = [&](int i, float f, bool nan) {
    uint2 o = make_uint2(fp8_codes(v[i].x, f) | fp8_codes(v[i].y, f) << 16, fp8_codes(v[i].z, f) | fp8_codes(v[i].w, f) << 16);
    if (nan) o = make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    return o;
  };
  if ((FORM & Q_ROWS) || (FORM == Q_BLOCKS && p.q)) {
    uint8_t* q = p.q + (FORM == Q_BLOCKS ? blockIdx.z * p.q_batch : 0);
    float row_up = 0.0f;  // of row cg / 2, negative where the block is bad
    if constexpr (FORM != Q_BLOCKS) {
      const float sc = fp8_scale(rmax, row_up);
      if (rmax >= 0x7F80u) row_up = -1.0f;
      if (!(cg & 1) && (live >> (cg >> 1) & 1u)) p.s[static_cast<int64_t>(blockIdx.x) * p.pitch + r0 + rg * 8 + (cg >> 1)] = sc;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + rg * 8 + i;
      float f = up;
      bool nan = bad;
      if constexpr (FORM != Q_BLOCKS) {
        f = __shfl_sync(0xffffffffu, row_up, (lane & 16) | 2 * i);
        nan = f < 0.0f;
      }
      if (FORM == Q_BLOCKS ? r >= p.rows : !(live >> i & 1u)) continue;
      if (c < p.cols) *reinterpret_cast<uint2*>(q + r * p.ld + c) = row_codes(i, f, nan);
      else if (c < p.ld) *reinterpret_cast<uint2*>(q + r * p.ld + c) = make_uint2(0, 0);  // up to the pitch
    }
  }
  if constexpr (FORM != Q_ROWS) {
    if (FORM == Q_BLOCKS && !p.qt) return;
    float f[8];
    uint32_t nan = 0;
    if constexpr (FORM & Q_COLS) {
      uint32_t m[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = absmax2(m[j], w[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        m[j] = absmax2(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
        if (lane < 16) wmax[warp][cg * 4 + j] = m[j];
      }
      __syncthreads();
      if (t < 128) {  // a column each: its maximum over the warps, scale and multiplier (negative: a bad block)
        const uint16_t* halves = reinterpret_cast<const uint16_t*>(wmax);
        uint32_t a = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) a = max(a, halves[w * 128 + t] & 0x7FFFu);
        float m;
        const float sc = fp8_scale(a, m);
        col_up[t] = a >= 0x7F80u ? -1.0f : m;
        if (c0 + t < p.cols) p.st[static_cast<int64_t>(blockIdx.y) * p.pitch_t + c0 + t] = sc;
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const float4 x = *reinterpret_cast<const float4*>(col_up + cg * 8 + j);
        f[j] = x.x, f[j + 1] = x.y, f[j + 2] = x.z, f[j + 3] = x.w;
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) nan |= f[j] < 0.0f ? 1u << j : 0u;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = up;
      nan = bad ? 0xFFu : 0u;
    }
    // column j's codes over the thread's 8 rows: 8 bytes of a transposed row.  In a bad block they are NaN on the rows that
    // are there: bit i of `live` to byte i
    const uint32_t nan_codes[2] = {((live & 15u) * 0x00204081u & 0x01010101u) * 0x7Fu,
                                   ((live >> 4) * 0x00204081u & 0x01010101u) * 0x7Fu};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = j == 0 ? v[i].x : j == 1 ? v[i].y : j == 2 ? v[i].z : v[i].w;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t a = 0;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t w0 = w[4 * i + 2 * k], w1 = w[4 * i + 2 * k + 1];
            const uint32_t pair = h ? (w0 >> 16 | (w1 & 0xFFFF0000u)) : (w0 & 0xFFFFu) | w1 << 16;
            a |= fp8_codes(pair, f[2 * j + h]) << (16 * k);
          }
          o[i] = nan >> (2 * j + h) & 1u ? nan_codes[i] : a;
        }
        // (8-byte unit rg of the column at rg ^ cg: the lanes of a store fall into different banks)
        *reinterpret_cast<uint2*>(tile + (cg * 8 + 2 * j + h) * 128 + (rg ^ cg) * 8) = make_uint2(o[0], o[1]);
      }
    }
    __syncthreads();
    uint8_t* qt = p.qt + (FORM == Q_BLOCKS ? blockIdx.z * p.qt_batch : 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {  // 8 vectors of 16 rows per transposed row
      const int item = t + i * kQThreads, col = item >> 3, r16 = (item & 7) * 16;
      const int k = col >> 3;  // the column's swizzle: units 2 n and 2 n + 1 at 2 (n ^ k / 2), the other way round where k is odd
      uint4 o = *reinterpret_cast<const uint4*>(tile + col * 128 + (r16 ^ (k >> 1) * 16));
      if (k & 1) o = make_uint4(o.z, o.w, o.x, o.y);
      if (c0 + col < p.cols && r0 + r16 < p.ldt)
        *reinterpret_cast<uint4*>(qt + static_cast<int64_t>(c0 + col) * p.ldt + r0 + r16) = o;
    }
  }
}

// Rows alone, on the dispatch gather: in token order, each token's row read and quantised once and written to the rows of its K
// slots (the tile kernel above reads it K times).  A warp takes 1024 columns of a token, a lane 16 contiguous ones of
// each of two 512-column pieces: 8 lanes hold a block of 128, codes leave as 16 bytes per lane.  Measured at T = 8192, H =
// 4096, K = 8: 58 us (340 MB, 5,900 GB/s), 164 on the tile kernel.
__global__ void __launch_bounds__(kQThreads) fp8_dispatch_kernel(const uint16_t* __restrict__ x, const int32_t* __restrict__ inv,
                                                                 int64_t T, int K, int cols, int64_t ld, int64_t pitch,
                                                                 uint8_t* __restrict__ q, float* __restrict__ s) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kQThreads / 32) + (threadIdx.x >> 5);
  const int64_t nwarps = static_cast<int64_t>(gridDim.x) * (kQThreads / 32);
  const int64_t chunks = (cols + 1023) / 1024;
  for (int64_t item = warp; item < T * chunks; item += nwarps) {
    const int64_t t = item / chunks;
    const int c0 = static_cast<int>(item - t * chunks) * 1024 + lane * 16;
    int row = lane < K ? __ldg(inv + t * K + lane) : -1;  // of the first 32 slots, beside the loads of x
    uint4 v[2][2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = c0 + 512 * u + 8 * h;
        v[u][h] = c < cols ? __ldcs(reinterpret_cast<const uint4*>(x + t * cols + c)) : make_uint4(0, 0, 0, 0);
      }
    uint4 codes[2];
    float scale[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t m = absmax2(absmax2(absmax2(v[u][0].x, v[u][0].y), absmax2(v[u][0].z, v[u][0].w)),
                           absmax2(absmax2(v[u][1].x, v[u][1].y), absmax2(v[u][1].z, v[u][1].w)));
#pragma unroll
      for (int d = 4; d >= 1; d >>= 1) m = absmax2(m, __shfl_xor_sync(0xffffffffu, m, d));
      m = absmax_word(m);
      float up;
      scale[u] = fp8_scale(m, up);
      codes[u] = make_uint4(fp8_codes(v[u][0].x, up) | fp8_codes(v[u][0].y, up) << 16,
                            fp8_codes(v[u][0].z, up) | fp8_codes(v[u][0].w, up) << 16,
                            fp8_codes(v[u][1].x, up) | fp8_codes(v[u][1].y, up) << 16,
                            fp8_codes(v[u][1].z, up) | fp8_codes(v[u][1].w, up) << 16);
      if (m >= 0x7F80u) {
        const uint32_t second = c0 + 512 * u + 8 < cols ? 0x7F7F7F7Fu : 0u;  // (past the columns: zeros up to the pitch)
        codes[u] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, second, second);
      }
    }
    for (int k0 = 0; k0 < K; k0 += 32) {
      if (k0) row = k0 + lane < K ? __ldg(inv + t * K + k0 + lane) : -1;
      for (unsigned live = __ballot_sync(0xffffffffu, row >= 0); live; live &= live - 1) {
        const int64_t r = __shfl_sync(0xffffffffu, row, __ffs(live) - 1);
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int c = c0 + 512 * u;
          if (c >= cols) continue;
          __stcs(reinterpret_cast<uint4*>(q + r * ld + c), codes[u]);
          if ((lane & 7) == 0) s[(c >> 7) * pitch + r] = scale[u];
        }
      }
    }
  }
}

bool ok16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Row tiles are the grid's y.
template <int FORM, bool GATHER>
int launch_form(const QuantArgs& p, int batch, int kind, cudaStream_t stream) {
  const int64_t ty = fp8_blocks(p.rows), tx = fp8_blocks(p.cols);
  trace_begin(stream, kind);
  const cudaError_t e = launch_pdl(fp8_quantize_kernel<FORM, GATHER>, dim3(static_cast<unsigned>(tx), static_cast<unsigned>(ty), batch),
                                   dim3(kQThreads), 0, stream, p);
  trace_end(stream);
  return static_cast<int>(e);
}

}  // namespace

int launch_fp8_quantize(const Fp8Source& src, int64_t rows, int32_t cols, uint8_t* q, float* s, uint8_t* qt, float* st,
                        int kind, cudaStream_t stream) {
  QuantArgs p{};
  p.src = src;
  p.rows = rows;
  p.cols = cols;
  p.q = q;
  p.s = s;
  p.qt = qt;
  p.st = st;
  p.ld = fp8_ld(cols);
  p.ldt = fp8_ld(rows);
  p.pitch = fp8_pitch(rows);
  p.pitch_t = fp8_pitch(cols);
  if (src.gather && !qt) {
    const int64_t want = (src.tokens * ((cols + 1023) / 1024) + kQThreads / 32 - 1) / (kQThreads / 32);
    const int64_t most = static_cast<int64_t>(sm_count()) * 16;
    if (most <= 0) return static_cast<int>(cudaErrorInvalidDevice);
    trace_begin(stream, kind);
    const cudaError_t e = launch_pdl(fp8_dispatch_kernel, dim3(static_cast<unsigned>(want < most ? want : most)), dim3(kQThreads),
                                     0, stream, src.x, src.inv, src.tokens, src.K, static_cast<int>(cols), p.ld, p.pitch, q, s);
    trace_end(stream);
    return static_cast<int>(e);
  }
  auto run = [&](auto gather) {
    constexpr bool G = decltype(gather)::value;
    if (q && qt) return launch_form<Q_ROWS | Q_COLS, G>(p, 1, kind, stream);
    if constexpr (!G) {
      if (q) return launch_form<Q_ROWS, G>(p, 1, kind, stream);
    }
    return launch_form<Q_COLS, G>(p, 1, kind, stream);
  };
  return src.gather ? run(std::true_type{}) : run(std::false_type{});
}

}  // namespace mok

using namespace mok;

namespace {
mok_status outputs_ok(const void* q, const void* s, const void* qt, const void* st) {
  if ((!q && !qt) || (q != nullptr) != (s != nullptr) || (qt != nullptr) != (st != nullptr)) return MOK_ERR_INVALID_ARG;
  if ((q && (!ok16(q) || !ok16(s))) || (qt && (!ok16(qt) || !ok16(st)))) return MOK_ERR_INVALID_ARG;
  return MOK_OK;
}
// Whether codes and scales (of nscale and nscale_t floats) of `rows` x `cols` values (of each of `batch`) spare x's n bytes.
bool spare(const void* x, int64_t n, int64_t batch, int64_t rows, int64_t cols, const void* q, const void* s, int64_t nscale,
           const void* qt, const void* st, int64_t nscale_t) {
  return apart(x, n, q, batch * rows * fp8_ld(cols)) && apart(x, n, s, nscale * 4) && apart(x, n, qt, batch * cols * fp8_ld(rows)) &&
         apart(x, n, st, nscale_t * 4);
}
// The same with a scale per row and 128 columns.
bool spare_rows(const void* x, int64_t n, int64_t rows, int64_t cols, const void* q, const void* s, const void* qt, const void* st) {
  return spare(x, n, 1, rows, cols, q, s, fp8_blocks(cols) * fp8_pitch(rows), qt, st, fp8_blocks(rows) * fp8_pitch(cols));
}
}  // namespace

extern "C" {

mok_status mok_fp8_quantize(const void* x, int64_t rows, int32_t cols, uint8_t* q, float* s, uint8_t* qt, float* st,
                            void* stream) {
  if (rows < 0 || cols < 8 || cols % 8 != 0) return MOK_ERR_INVALID_ARG;
  if (rows > kFp8MaxRows) return MOK_ERR_UNSUPPORTED;
  if (rows == 0) return MOK_OK;
  if (!ok16(x)) return MOK_ERR_INVALID_ARG;
  const mok_status rc = outputs_ok(q, s, qt, st);
  if (rc != MOK_OK) return rc;
  if (!spare_rows(x, rows * cols * 2, rows, cols, q, s, qt, st)) return MOK_ERR_INVALID_ARG;
  const Fp8Source src{static_cast<const uint16_t*>(x), nullptr, nullptr, nullptr, rows, 1, 0};
  return launch_fp8_quantize(src, rows, cols, q, s, qt, st, K_FP8_QUANTIZE, static_cast<cudaStream_t>(stream)) ? MOK_ERR_CUDA
                                                                                                             : MOK_OK;
}

mok_status mok_fp8_quantize_routed(const mok_schedule* sched, int32_t gather, const void* x, int32_t cols, uint8_t* q,
                                   float* s, uint8_t* qt, float* st, void* stream) {
  Sizes z;
  mok_status rc = routed_sizes(sched, &z);
  if (rc != MOK_OK) return rc;
  if (cols < 8 || cols % 8 != 0 || (gather != 0 && gather != 1)) return MOK_ERR_INVALID_ARG;
  if (z.rpad_max > kFp8MaxRows) return MOK_ERR_UNSUPPORTED;
  if (z.T == 0) return MOK_OK;
  if (!ok16(x)) return MOK_ERR_INVALID_ARG;
  rc = outputs_ok(q, s, qt, st);
  if (rc != MOK_OK) return rc;
  if (!spare_rows(x, (gather ? z.T : z.rpad_max) * cols * 2, z.rpad_max, cols, q, s, qt, st)) return MOK_ERR_INVALID_ARG;
  if (!apart_from_tables(*sched, z, q, z.rpad_max * fp8_ld(cols)) || !apart_from_tables(*sched, z, qt, cols * fp8_ld(z.rpad_max)) ||
      !apart_from_tables(*sched, z, s, 4 * fp8_blocks(cols) * fp8_pitch(z.rpad_max)) ||
      !apart_from_tables(*sched, z, st, 4 * fp8_blocks(z.rpad_max) * fp8_pitch(cols)))
    return MOK_ERR_INVALID_ARG;
  const Fp8Source src{static_cast<const uint16_t*>(x), sched->row_token, sched->meta, sched->inv, z.T, z.K, gather};
  return launch_fp8_quantize(src, z.rpad_max, cols, q, s, qt, st, gather ? K_FP8_DISPATCH : K_FP8_QUANTIZE,
                             static_cast<cudaStream_t>(stream))
             ? MOK_ERR_CUDA
             : MOK_OK;
}

mok_status mok_fp8_quantize_blocks(const void* x, int32_t batch, int64_t rows, int32_t cols, uint8_t* q, float* s,
                                   uint8_t* qt, float* st, void* stream) {
  if (batch < 1 || rows < 8 || rows % 8 != 0 || cols < 8 || cols % 8 != 0) return MOK_ERR_INVALID_ARG;
  if (rows > kFp8MaxRows || batch > 65535) return MOK_ERR_UNSUPPORTED;
  if (!ok16(x)) return MOK_ERR_INVALID_ARG;
  const mok_status rc = outputs_ok(q, s, qt, st);
  if (rc != MOK_OK) return rc;
  const int64_t scales = batch * fp8_blocks(rows) * fp8_blocks(cols);
  if (!spare(x, batch * rows * cols * 2, batch, rows, cols, q, s, scales, qt, st, scales)) return MOK_ERR_INVALID_ARG;
  QuantArgs p{};
  p.src.x = static_cast<const uint16_t*>(x);
  p.rows = rows;
  p.cols = cols;
  p.q = q;
  p.s = s;
  p.qt = qt;
  p.st = st;
  p.ld = fp8_ld(cols);
  p.ldt = fp8_ld(rows);
  p.src_batch = rows * cols;
  p.q_batch = rows * p.ld;
  p.qt_batch = cols * p.ldt;
  p.s_batch = p.st_batch = fp8_blocks(rows) * fp8_blocks(cols);
  return launch_form<Q_BLOCKS, false>(p, batch, K_FP8_WEIGHT, static_cast<cudaStream_t>(stream)) ? MOK_ERR_CUDA : MOK_OK;
}

}  // extern "C"
