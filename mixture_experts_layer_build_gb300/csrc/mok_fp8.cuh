// mok_fp8.cuh -- 8-bit products with one fp32 scale per block of 128: what the quantisers and the products share.
//
//   t = max(amax, 2^-50), scale = t / 448, code = E4M3(v * (448 / t))
//   C[m, n] = sum over K blocks b, ascending, of sa[b][m] sb[b][n] * (sum over k in b of a[m, k] b[n, k])
//
// The product of two codes is exact; a block's 128 of them are added in the tensor core's fp32 accumulator, which cannot hold
// every such sum (they span 2^-18 to 2^25): the tests allow 127 additions of 2^-24 of the magnitudes.  The outer sum is fp32
// fused multiply-adds.
#pragma once
#include <cuda.h>

#include "mok_internal.cuh"
#include "mok_once.h"
#include "mok_ptx.cuh"
#include "mok_route.cuh"

namespace mok {

constexpr int kFp8Block = 128;        // values per scale: a K block of the products
constexpr float kFp8Max = 448.0f;
constexpr float kFp8Least = 0x1p-50f;  // of a block's largest magnitude
constexpr int64_t kFp8MaxRows = int64_t{65535} * kFp8Block;  // that a quantisation takes: row tiles in a grid's y

inline int64_t fp8_ld(int64_t cols) { return (cols + 15) / 16 * 16; }       // bytes between rows of codes
inline int64_t fp8_pitch(int64_t rows) { return (rows + 3) / 4 * 4; }       // floats between K blocks of row scales
inline int64_t fp8_blocks(int64_t n) { return (n + kFp8Block - 1) / kFp8Block; }

#ifdef __CUDACC__
// Scale and multiplier of a block whose largest bf16 magnitude is `amax` (15 bits); a NaN scale for an infinity or NaN.
__device__ __forceinline__ float fp8_scale(uint32_t amax, float& up) {
  const float t = fmaxf(__uint_as_float(amax << 16), kFp8Least);
  up = __fdiv_rn(kFp8Max, t);
  return amax >= 0x7F80u ? __uint_as_float(0x7FC00000u) : __fdiv_rn(t, kFp8Max);
}
// E4M3 codes of the two bf16 halves of a word, times `up`; NaN codes where the block is bad.
__device__ __forceinline__ uint32_t fp8_codes(uint32_t w, float up) {
  uint16_t q;
  float lo, hi;
  mul_f32x2(lo, hi, bf16_lo(w), bf16_hi(w), up, up);
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(q) : "f"(hi), "f"(lo));
  return q;
}
// Per half the larger magnitude, NaN if either is NaN (sign bits mean nothing).
__device__ __forceinline__ uint32_t absmax2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
#endif

// x: plain rows, tokens that the rows of a schedule gather, or a schedule's rows.
struct Fp8Source {
  const uint16_t* x;
  const int32_t* row_token;  // null: plain rows
  const int32_t* meta;
  const int32_t* inv;        // the row of each token's slots
  int64_t tokens;
  int32_t K;
  int32_t gather;
};
int launch_fp8_quantize(const Fp8Source& src, int64_t rows, int32_t cols, uint8_t* q, float* s, uint8_t* qt, float* st,
                        int kind, cudaStream_t stream);

bool make_tmap_fp8(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint64_t pitch, uint32_t box_outer);

}  // namespace mok
