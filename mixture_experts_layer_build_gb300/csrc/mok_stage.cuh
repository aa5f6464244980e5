// mok_stage.cuh -- what the epilogue warps of the CTA-pair kernels share: reading a TMEM accumulator, and staging
// output rows for TMA stores.
#pragma once
#include "mok_ptx.cuh"

namespace mok {

// One epilogue warp's output staging: two shared tiles of 32 rows x 64 bytes in the 64-byte TMA swizzle
// (chunk j of row r at j ^ ((r >> 1) & 3)), each stored by one TMA store that clips at the tensor's
// edges; a tile is refilled once its previous store has read it.
struct WarpStage {
  uint32_t base;
  int cur, lane;
  __device__ __forceinline__ void put(const uint4 (&ch)[4], const CUtensorMap* tm, int c0, int r0) {
    if (lane == 0) bulk_wait_read<1>();
    __syncwarp();
    const uint32_t b = base + static_cast<uint32_t>(cur) * 2048u;
    cur ^= 1;
    const uint32_t row = b + static_cast<uint32_t>(lane) * 64u;
#pragma unroll
    for (int j = 0; j < 4; ++j) st_shared_v4(row + (static_cast<uint32_t>(j ^ ((lane >> 1) & 3)) << 4), ch[j]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(tm, b, c0, r0);
      bulk_commit();
    }
  }
  __device__ __forceinline__ void put_bf16(const float (&v)[32], const CUtensorMap* tm, int c0, int r0) {
    uint4 ch[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      ch[j] = make_uint4(pack_bf16x2(v[8 * j], v[8 * j + 1]), pack_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                         pack_bf16x2(v[8 * j + 4], v[8 * j + 5]), pack_bf16x2(v[8 * j + 6], v[8 * j + 7]));
    put(ch, tm, c0, r0);
  }
};

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  tmem_ld_32x32b_x32(taddr, r);
  tmem_ld_wait();
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

// Waits for this warp's TMEM loads.  r, the registers of the one that is needed now, passes through: nothing that
// uses them can be moved before the wait.
__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_ld_wait_for(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

}  // namespace mok
