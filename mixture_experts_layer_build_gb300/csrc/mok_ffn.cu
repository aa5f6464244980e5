// mok_ffn.cu -- the C ABI of the dense gated feed-forward block: checks, buffers and the order of its
// contractions.
#include "mok_ffn.cuh"

namespace mok {
namespace {

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

bool ffn_shape_ok(const mok_ffn_shape* s) {
  return s && s->T >= 0 && s->T <= kFfnMaxTokens && s->H >= 8 && s->I >= 8 && s->H <= 65536 &&
         s->I <= 65536 && s->H % 8 == 0 && s->I % 8 == 0 && (s->act == MOK_ACT_SILU || s->act == MOK_ACT_GELU);
}

// The context: a [T, I] bf16, then (saved) the factors u act'(g) and act(g) in fp32, in the layout of ffn_saved_offset.
struct FfnCtx {
  uint16_t* a;
  float* kg;
  float* ku;
  size_t bytes;
  FfnCtx(const mok_ffn_shape& s, bool save, const void* p) {
    char* base = static_cast<char*>(const_cast<void*>(p));
    const size_t n = static_cast<size_t>(s.T) * s.I;
    const size_t ns = (static_cast<size_t>(s.T) + 31) / 32 * 32 * s.I;
    const size_t og = up256(2 * n), ou = og + up256(4 * ns);
    a = reinterpret_cast<uint16_t*>(base);
    kg = save ? reinterpret_cast<float*>(base + og) : nullptr;
    ku = save ? reinterpret_cast<float*>(base + ou) : nullptr;
    bytes = save ? ou + up256(4 * ns) : og;
    if (bytes < 256) bytes = 256;
  }
};

bool unaligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) != 0; }
bool overlap(const void* a, const void* b, size_t n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < n : x - y < n;
}
bool need16(const void* p) { return p && !unaligned(p, 16); }

bool on_pairs(int var, int64_t M, int64_t N) { return ffn_on_pairs(var, M, N, sm_count()); }

int launch_fwd(int var, int64_t M, int64_t N, int64_t K, const FfnOperands& o, const FfnArgs& a,
               cudaStream_t stream) {
  if (M <= kFfnRowTokens) return launch_ffn_row(var, M, N, K, o, a, stream);
  return on_pairs(var, M, N) ? launch_ffn_pair_fwd(var, M, N, K, o, a, stream)
                             : launch_ffn_tile(var, M, N, K, o, a, stream);
}

}  // namespace
}  // namespace mok

using namespace mok;

extern "C" {

size_t mok_ffn_ctx_bytes(const mok_ffn_shape* s, int32_t save) {
  return ffn_shape_ok(s) ? FfnCtx(*s, save != 0, nullptr).bytes : 0;
}

size_t mok_ffn_workspace_bytes(const mok_ffn_shape* s) {
  if (!ffn_shape_ok(s)) return 0;
  const size_t n = up256(static_cast<size_t>(s->T) * s->I * 2);
  return n ? 2 * n : 256;
}

mok_status mok_ffn_forward(const mok_ffn_shape* s, const void* x, const void* w_gate, const void* w_up,
                           const void* w_down, const void* residual, void* out, void* ctx, size_t ctx_bytes,
                           int32_t save, uint32_t* status, void* stream) {
  if (!ffn_shape_ok(s) || !ctx || unaligned(ctx, 256) || unaligned(status, 4)) return MOK_ERR_INVALID_ARG;
  const FfnCtx c(*s, save != 0, ctx);
  if (ctx_bytes < c.bytes) return MOK_ERR_WORKSPACE_TOO_SMALL;
  if (s->T == 0) return MOK_OK;
  if (!need16(x) || !need16(w_gate) || !need16(w_up) || !need16(w_down) || !need16(out) || unaligned(residual, 16))
    return MOK_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  FfnArgs a{};
  a.act = s->act;
  a.status = status;
  a.out0 = c.a;
  a.kg = c.kg;
  a.ku = c.ku;
  if (launch_fwd(F_GATEUP, s->T, s->I, s->H, {x, nullptr, w_gate, w_up}, a, st)) return MOK_ERR_CUDA;
  a.out0 = out;
  a.kg = a.ku = nullptr;
  a.residual = static_cast<const uint16_t*>(residual);
  return launch_fwd(F_DOWN, s->T, s->H, s->I, {c.a, nullptr, w_down, nullptr}, a, st) ? MOK_ERR_CUDA : MOK_OK;
}

mok_status mok_ffn_backward(const mok_ffn_shape* s, const void* x, const void* w_gate, const void* w_up,
                            const void* w_down, const void* ctx, size_t ctx_bytes, const void* dy,
                            const mok_ffn_grads* gr, void* ws, size_t ws_bytes, uint32_t* status, void* stream) {
  if (!ffn_shape_ok(s) || !gr || (gr->dw_type != MOK_DT_BF16 && gr->dw_type != MOK_DT_FP32) || unaligned(status, 4))
    return MOK_ERR_INVALID_ARG;
  if ((gr->dw_gate == nullptr) != (gr->dw_up == nullptr) || unaligned(gr->dx, 16) || unaligned(gr->dx_add, 16) ||
      unaligned(gr->dw_gate, 16) ||
      unaligned(gr->dw_up, 16) || unaligned(gr->dw_down, 16))
    return MOK_ERR_INVALID_ARG;
  if (!ctx || unaligned(ctx, 256) || !ws || unaligned(ws, 256)) return MOK_ERR_INVALID_ARG;
  const FfnCtx c(*s, true, ctx);
  if (ctx_bytes < c.bytes || ws_bytes < mok_ffn_workspace_bytes(s)) return MOK_ERR_WORKSPACE_TOO_SMALL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (s->T == 0) {  // sums over no tokens
    const size_t n = static_cast<size_t>(s->H) * s->I * (gr->dw_type == MOK_DT_FP32 ? 4 : 2);
    for (void* p : {gr->dw_gate, gr->dw_up, gr->dw_down})
      if (p && cudaMemsetAsync(p, 0, n, st) != cudaSuccess) return MOK_ERR_CUDA;
    return MOK_OK;
  }
  if (!need16(x) || !need16(w_gate) || !need16(w_up) || !need16(w_down) || !need16(dy)) return MOK_ERR_INVALID_ARG;
  // dx is written while the weight gradients read x and dy
  const size_t tokens = static_cast<size_t>(s->T) * s->H * 2;
  if (gr->dx && ((gr->dw_down && overlap(gr->dx, dy, tokens)) || (gr->dw_gate && overlap(gr->dx, x, tokens))))
    return MOK_ERR_INVALID_ARG;
  uint16_t* dg = static_cast<uint16_t*>(ws);
  uint16_t* du = reinterpret_cast<uint16_t*>(static_cast<char*>(ws) + up256(static_cast<size_t>(s->T) * s->I * 2));
  FfnBackward b{};
  b.T = s->T;
  b.H = s->H;
  b.I = s->I;
  b.act = s->act;
  b.dw_f32 = gr->dw_type == MOK_DT_FP32;
  b.x = x;
  b.w_gate = w_gate;
  b.w_up = w_up;
  b.w_down = w_down;
  b.a = c.a;
  b.kg = c.kg;
  b.ku = c.ku;
  b.dy = dy;
  b.dg = dg;
  b.du = du;
  b.dx = gr->dx;
  b.dx_add = gr->dx_add;
  b.dw_gate = gr->dw_gate;
  b.dw_up = gr->dw_up;
  b.dw_down = gr->dw_down;
  b.status = status;
  FfnArgs a{};
  a.act = s->act;
  a.status = status;
  // DACT, then DX: each in its phase's launch with weight gradients, or before it on the tile kernel
  const bool dact = gr->dx || gr->dw_gate;
  b.dact = dact && on_pairs(F_DACT, s->T, s->I);
  b.dx_rows = gr->dx && on_pairs(F_DX, s->T, s->H);
  if (dact && !b.dact) {
    a.out0 = dg;
    a.out1 = du;
    a.kg = c.kg;
    a.ku = c.ku;
    if (launch_ffn_tile(F_DACT, s->T, s->I, s->H, {dy, nullptr, w_down, nullptr}, a, st)) return MOK_ERR_CUDA;
    a.kg = a.ku = nullptr;
  }
  if (launch_ffn_pair_bwd(1, b, st)) return MOK_ERR_CUDA;
  if (gr->dx && !b.dx_rows) {
    a.out0 = gr->dx;
    a.out1 = nullptr;
    a.residual = static_cast<const uint16_t*>(gr->dx_add);
    if (launch_ffn_tile(F_DX, s->T, s->H, s->I, {dg, du, w_gate, w_up}, a, st)) return MOK_ERR_CUDA;
  }
  if (launch_ffn_pair_bwd(2, b, st)) return MOK_ERR_CUDA;
  return MOK_OK;
}

}  // extern "C"
