// mok_fp8_gemm.cuh -- what the kernels of the 8-bit products are given (mok_fp8.cuh has the mathematics).
#pragma once
#include "mok_fp8.cuh"

namespace mok {

enum Fp8Mode : int32_t {
  FP8_DENSE = 0,
  FP8_GROUPED,  // a's rows are a schedule's, b is one matrix per expert
  FP8_WGRAD     // the summed index is a schedule's rows: one output per expert
};

struct Fp8Operand {
  const uint8_t* q;
  const float* s;
  int64_t rows, cols, ld;
  int32_t batch;
  bool row_scales;
};

// P: the operand whose rows are an accumulator's lanes, Q: its columns (the tile kernel has P = b, the pairs P = a).  Scales
// of K block kb: a scale per row at s[kb * pitch + row], one per 128 rows at s[matrix * batch + row / 128 * k_blocks + kb].
struct Fp8Problem {
  int32_t mode;
  int32_t p_rows, q_rows;    // of one matrix
  int32_t p_tiles, q_tiles;
  int32_t k_blocks;
  const float* sp;
  const float* sq;
  int64_t p_pitch, q_pitch;
  int64_t p_batch, q_batch;
  void* out;
  int64_t ldo;
  int32_t out_f32;
  int32_t early_p, early_q;  // P or Q (weights) may be read before the previous kernel of the stream ends
  int32_t experts;
  const int32_t* mblocks;    // of the schedule
  const int32_t* poff;
  const int32_t* counts;
  const int32_t* meta;
  uint32_t* status;
};

// out [rows of a, rows of b].  x: a's bf16 values, quantised on the way (dense, at most kFp8XqRows rows; a's codes and scales
// are not read then), or null.  rows: of a that hold values; row_blocks: (FP8_GROUPED) 128-row blocks of the layout at most.
constexpr int kFp8XqRows = 8;
int launch_fp8_tile(const Fp8Operand& a, const void* x, const Fp8Operand& b, Fp8Problem g, int64_t rows, int64_t row_blocks,
                    int kind, cudaStream_t stream);

bool make_tmap_f32(CUtensorMap* m, const void* base, uint64_t inner, uint64_t outer, uint32_t box_inner,
                   uint32_t box_outer);

// p: rows of the output, with a scale per row; q: its columns.  row_units: (FP8_GROUPED) 256-row units at most.
int launch_fp8_pair(const Fp8Operand& p, const Fp8Operand& q, Fp8Problem g, int64_t row_units, int kind, cudaStream_t stream);

}  // namespace mok
