// mok_fp8.cu -- the C ABI of the 8-bit products: checks, and which kernel a product runs on.
#include "mok_fp8_gemm.cuh"

namespace mok {
namespace {

constexpr int64_t kMax = (int64_t{1} << 31) - 1024;  // rows and columns: indices of padded tiles stay within 31 bits

bool ok16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
mok_status from_cuda(int rc) { return rc == 0 ? MOK_OK : MOK_ERR_CUDA; }

// A matrix that a product can read (rows * cols may be 0: then nothing is).
bool matrix_ok(const mok_fp8_matrix* m, int32_t batch) {
  if (!m || m->rows < 0 || m->cols < 0 || m->rows > kMax || m->cols > kMax || m->batch != batch || batch < 1) return false;
  if (m->scaling != MOK_FP8_ROWS && m->scaling != MOK_FP8_BLOCKS) return false;
  if (m->ld < m->cols || m->ld % 16 != 0 || m->ld > kMax) return false;
  if (m->rows * static_cast<int64_t>(batch) > kMax) return false;  // TMA coordinates
  return m->rows == 0 || m->cols == 0 || (ok16(m->q) && ok16(m->s));
}

// Whether an output of n bytes overlaps neither codes nor scales of a matrix.
bool apart_from(const mok_fp8_matrix& m, const void* out, int64_t n) {
  const int64_t scales = m.scaling == MOK_FP8_ROWS ? fp8_blocks(m.cols) * fp8_pitch(m.rows)
                                                   : fp8_blocks(m.cols) * fp8_blocks(m.rows) * m.batch;
  return apart(m.q, m.rows * m.ld * m.batch, out, n) && apart(m.s, scales * 4, out, n);
}

Fp8Operand operand(const mok_fp8_matrix& m) {
  return {m.q, m.s, m.rows, m.cols, m.ld, m.batch, m.scaling == MOK_FP8_ROWS};
}

// out [M, N]: see mok_fp8_matmul.  x: a's values where the product quantises them itself, or null; early: b may be read before
// the previous kernel of the stream has ended.
mok_status product(const mok_fp8_matrix& a, const void* x, const mok_fp8_matrix& b, void* out, int32_t out_type, bool early,
                   uint32_t* status, cudaStream_t stream) {
  Fp8Problem g{};
  g.mode = FP8_DENSE;
  g.k_blocks = static_cast<int32_t>(fp8_blocks(a.cols));
  g.out = out;
  g.ldo = b.rows;
  g.out_f32 = out_type == MOK_DT_FP32;
  g.early_p = g.early_q = early;
  g.status = status;
  // Pairs from about a quarter of the SMs' worth of 128 x 128 tiles on, or where K is short; below, tiles, which can split K.
  // Measured, tiles and pairs: 129 x 2048 x 7168 12.3 and 20.2 us, 512 x 1536 x 4096 13.0 and 13.4, 1003 x 1000 x 2056 10.2 and 9.7,
  // 256 x 1024 x 1024 7.0 and 6.6, 1024 x 2048 x 2048 13.7 and 9.5; both row-scaled 512 x 512 x 2048 7.8 and 10.6.
  // The rule does not look at how long K is beyond that: over 7168, 300 x 2048 17.8 and 21.2, 512 x 1280 17.4 and 21.1 run on pairs
  // all the same (160 x 2432 21.9 and 21.1, 256 x 2432 22.6 and 21.2; 600 x 4096 over 4096 37.8 and 19.2).
  if (a.rows > 128 && (4 * fp8_blocks(a.rows) * fp8_blocks(b.rows) >= sm_count() || g.k_blocks <= 8))
    return from_cuda(launch_fp8_pair(operand(a), operand(b), g, 0, K_FP8_PAIR, stream));
  return from_cuda(launch_fp8_tile(operand(a), x, operand(b), g, a.rows, 0, K_FP8_TILE, stream));
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

mok_status mok_fp8_matmul(const mok_fp8_matrix* a, const mok_fp8_matrix* b, void* out, int32_t out_type,
                          uint32_t* status, void* stream) {
  if (!matrix_ok(a, 1) || !matrix_ok(b, 1) || a->scaling != MOK_FP8_ROWS || a->cols != b->cols) return MOK_ERR_INVALID_ARG;
  if (b->rows < 8 || b->rows % 8 != 0 || (out_type != MOK_DT_BF16 && out_type != MOK_DT_FP32)) return MOK_ERR_INVALID_ARG;
  if (a->rows == 0) return MOK_OK;
  const int64_t bytes = a->rows * b->rows * (out_type == MOK_DT_FP32 ? 4 : 2);
  if (!ok16(out) || !apart_from(*a, out, bytes) || !apart_from(*b, out, bytes)) return MOK_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (a->cols == 0)
    return from_cuda(static_cast<int>(cudaMemsetAsync(out, 0, static_cast<size_t>(bytes), s)));
  return product(*a, nullptr, *b, out, out_type, false, status, s);
}

size_t mok_fp8_linear_workspace_bytes(int64_t M, int64_t K) {
  if (M < 0 || M > kFp8MaxRows || K < 8 || K % 8 != 0 || K > kMax) return 0;
  if (M <= kFp8XqRows) return 256;  // none is used
  const int64_t codes = (M * fp8_ld(K) + 255) / 256 * 256, scales = fp8_blocks(K) * fp8_pitch(M) * 4;
  return static_cast<size_t>((codes + scales + 255) / 256 * 256 + 256);
}

mok_status mok_fp8_linear(const void* x, int64_t M, const mok_fp8_matrix* w, void* out, void* ws, size_t ws_bytes,
                          uint32_t* status, void* stream) {
  if (M < 0 || !matrix_ok(w, 1) || w->scaling != MOK_FP8_BLOCKS) return MOK_ERR_INVALID_ARG;
  if (w->rows < 8 || w->rows % 8 != 0 || w->cols < 8 || w->cols % 8 != 0) return MOK_ERR_INVALID_ARG;
  if (M > kFp8MaxRows) return MOK_ERR_UNSUPPORTED;
  if (M == 0) return MOK_OK;
  const int64_t bytes = M * w->rows * 2;
  if (!ok16(x) || !ok16(out) || !apart(x, M * w->cols * 2, out, bytes) || !apart_from(*w, out, bytes)) return MOK_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  mok_fp8_matrix a{};
  a.rows = M;
  a.cols = w->cols;
  a.ld = fp8_ld(w->cols);
  a.batch = 1;
  a.scaling = MOK_FP8_ROWS;
  // (w is read no earlier than the previous kernel's end: it may be what wrote it)
  if (M <= kFp8XqRows) return product(a, x, *w, out, MOK_DT_BF16, false, status, st);
  if (!ws || reinterpret_cast<uintptr_t>(ws) % 256 != 0) return MOK_ERR_INVALID_ARG;
  if (ws_bytes < mok_fp8_linear_workspace_bytes(M, w->cols)) return MOK_ERR_WORKSPACE_TOO_SMALL;
  const int64_t used = static_cast<int64_t>(mok_fp8_linear_workspace_bytes(M, w->cols));
  if (!apart(ws, used, out, bytes) || !apart_from(*w, ws, used)) return MOK_ERR_INVALID_ARG;
  uint8_t* q = static_cast<uint8_t*>(ws);
  float* s = reinterpret_cast<float*>(q + (M * fp8_ld(w->cols) + 255) / 256 * 256);
  const mok_status rc = mok_fp8_quantize(x, M, static_cast<int32_t>(w->cols), q, s, nullptr, nullptr, stream);
  if (rc != MOK_OK) return rc;
  a.q = q;
  a.s = s;
  // the quantisation has waited for all before it, and does not write w
  return product(a, nullptr, *w, out, MOK_DT_BF16, true, status, st);
}

mok_status mok_fp8_grouped_matmul(const mok_schedule* sched, const mok_fp8_matrix* a, const mok_fp8_matrix* w, void* out,
                                  void* stream) {
  Sizes z;
  const mok_status rc = routed_sizes(sched, &z);
  if (rc != MOK_OK) return rc;
  if (!matrix_ok(a, 1) || !matrix_ok(w, z.E) || a->scaling != MOK_FP8_ROWS || w->scaling != MOK_FP8_BLOCKS)
    return MOK_ERR_INVALID_ARG;
  if (a->rows != z.rpad_max || a->cols != w->cols || w->cols < 8 || w->rows < 8 || w->rows % 8 != 0)
    return MOK_ERR_INVALID_ARG;
  if (z.T == 0) return MOK_OK;
  const int64_t bytes = a->rows * w->rows * 2;
  if (!ok16(out) || !apart_from(*a, out, bytes) || !apart_from(*w, out, bytes) || !apart_from_tables(*sched, z, out, bytes))
    return MOK_ERR_INVALID_ARG;
  Fp8Problem g{};
  g.mode = FP8_GROUPED;
  g.k_blocks = static_cast<int32_t>(fp8_blocks(a->cols));
  g.out = out;
  g.ldo = w->rows;
  g.experts = z.E;
  g.mblocks = sched->mblocks;
  g.poff = sched->poff;
  g.counts = sched->counts;
  g.meta = sched->meta;
  g.status = sched->status;
  // an expert with rows has one block that is not full at most
  const int64_t blocks = (z.R < z.E ? z.R : z.E) + z.R / 128;
  // Pairs from about 48 rows per expert on.  Measured, tiles and pairs: 128 experts, K = 4096, N = 1536, 32 rows each 187 and 190
  // us, 64 rows 243 and 192; 64 experts, K = 2048, N = 1024, 24 rows 35.2 and 45.1, 48 rows 45.3 and 45.1; 8 experts, K = 4096, N =
  // 1536, 128 rows 21.5 and 20.6.  The rule does not look at how many units there are: 4 experts, K = 7168, N = 1024, 48 rows 18.2 and
  // 22.1, 192 rows 18.9 and 22.2.
  if (z.R >= 48 * static_cast<int64_t>(z.E))
    return from_cuda(launch_fp8_pair(operand(*a), operand(*w), g, (z.R < z.E ? z.R : z.E) + z.R / 256, K_FP8_GROUPED_PAIR,
                                     static_cast<cudaStream_t>(stream)));
  return from_cuda(launch_fp8_tile(operand(*a), nullptr, operand(*w), g, z.R, blocks < z.mblocks_max ? blocks : z.mblocks_max,
                                   K_FP8_GROUPED_TILE, static_cast<cudaStream_t>(stream)));
}

mok_status mok_fp8_grouped_wgrad(const mok_schedule* sched, const mok_fp8_matrix* a, const mok_fp8_matrix* b, void* dw,
                                 int32_t dw_type, void* stream) {
  Sizes z;
  const mok_status rc = routed_sizes(sched, &z);
  if (rc != MOK_OK) return rc;
  if (!matrix_ok(a, 1) || !matrix_ok(b, 1) || a->scaling != MOK_FP8_ROWS || b->scaling != MOK_FP8_ROWS)
    return MOK_ERR_INVALID_ARG;
  if (a->cols != z.rpad_max || b->cols != z.rpad_max || a->rows < 8 || b->rows < 8 || b->rows % 8 != 0)
    return MOK_ERR_INVALID_ARG;
  if ((dw_type != MOK_DT_BF16 && dw_type != MOK_DT_FP32) || !ok16(dw)) return MOK_ERR_INVALID_ARG;
  if (a->rows * z.E > kMax) return MOK_ERR_UNSUPPORTED;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int64_t bytes = static_cast<int64_t>(z.E) * a->rows * b->rows * (dw_type == MOK_DT_FP32 ? 4 : 2);
  if (!apart_from(*a, dw, bytes) || !apart_from(*b, dw, bytes) || !apart_from_tables(*sched, z, dw, bytes))
    return MOK_ERR_INVALID_ARG;
  if (z.T == 0) return from_cuda(static_cast<int>(cudaMemsetAsync(dw, 0, static_cast<size_t>(bytes), s)));
  Fp8Problem g{};
  g.mode = FP8_WGRAD;
  g.k_blocks = static_cast<int32_t>(fp8_blocks(z.rpad_max));
  g.out = dw;
  g.ldo = b->rows;
  g.out_f32 = dw_type == MOK_DT_FP32;
  g.experts = z.E;
  g.mblocks = sched->mblocks;
  g.poff = sched->poff;
  g.counts = sched->counts;
  g.meta = sched->meta;
  g.status = sched->status;
  return from_cuda(launch_fp8_pair(operand(*a), operand(*b), g, 0, K_FP8_WGRAD, s));
}

}  // extern "C"
