// Shared by the kernels of the 8-bit KV cache: block sizes, table lookup, and the
// conversions between codes and 16-bit floating point.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace grok {

constexpr int kKv8Block = GROK_KV8_BLOCK;             // tokens per block
constexpr int kKv8Bytes = kKv8Block * kD;             // codes of one K or V block
constexpr int kKv8MaxBlocks = GROK_MAX_POSITION / kKv8Block;

// Blocks of a sequence of `len` rows; 0 when the length is outside [1, max_blocks * 64].
__device__ __forceinline__ int kv8_blocks(int len, int max_blocks) {
  return len < 1 || len > max_blocks * kKv8Block ? 0 : (len + kKv8Block - 1) / kKv8Block;
}

// A table entry; -1, reported, when it lies outside the pool.
__device__ __forceinline__ int kv8_block_id(const int32_t* table, size_t at, int n_blocks, int32_t* status) {
  const int id = table[at];
  if (id < 0 || id >= n_blocks) {
    report(status, GROK_DEV_BAD_PAGE);
    return -1;
  }
  return id;
}

// Four codes (one 32-bit word, first code in the low byte) to two fp16 pairs,
// exactly. int8: byte c with its sign bit flipped is c + 128; behind the byte
// 0x64 it is the fp16 number 1024 + (c + 128), from which 1152 is taken.
// e4m3: the hardware conversion.
template <int kKind>
__device__ __forceinline__ void kv8_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (kKind == GROK_KV8_INT8) {
    const uint32_t u = w ^ 0x80808080u;
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    constexpr uint32_t k1152 = 0x64806480u;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(a), "r"(k1152));
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(b), "r"(k1152));
  } else {
    asm("{\n\t.reg .b16 l, h;\n\t"
        "mov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
  }
}

// D[16 x 8] += A[16 x 16] B[16 x 8], fp16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held two to a lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 16-byte-multiple copy from global to shared memory, counted on an mbarrier.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

}  // namespace grok
