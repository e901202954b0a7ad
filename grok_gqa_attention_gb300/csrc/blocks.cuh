// Shared by the calls that read part of a paged cache: blocks of 64 tokens (two to
// a page), the 8-bit scale of the block bounds and the queries.
#pragma once

#include "common.cuh"

namespace grok {

constexpr int kBlk = GROK_SPARSE_BLOCK;                       // tokens per block
constexpr int kBlkPerPage = GROK_PAGE_TOKENS / kBlk;
constexpr int kBlkMax = GROK_MAX_POSITION / kBlk;             // blocks of a sequence at most
static_assert(GROK_PAGE_TOKENS % kBlk == 0, "a page is whole blocks");

// Blocks of a sequence of `len` rows; 0 when the length is outside [1, cap].
__device__ __forceinline__ int blk_count(int len, int cap) { return len < 1 || len > cap ? 0 : (len + kBlk - 1) / kBlk; }

// The page that holds block `blk` of sequence b; -1, reported, when the table's entry lies outside the pool.
__device__ __forceinline__ int blk_page(const PageMap& pm, int b, int blk, int32_t* status) {
  const int pg = pm.table[(size_t)b * pm.max_pages + blk / kBlkPerPage];
  if (pg < 0 || pg >= pm.n_pages) {
    report(status, GROK_DEV_BAD_PAGE);
    return -1;
  }
  return pg;
}

// Scale 2^e of 8-bit codes of values up to `a` (the bits of a bf16 magnitude): the least e with a <= 127 * 2^e, kept
// within [-32, 16] (above it no bf16 times 2^-e leaves fp32's range downwards; codes saturate at 127). With a = 1.m *
// 2^E, 127 * 2^(E - 6) = 1.984375 * 2^E is below a only where m is the largest, 127 / 128.
__device__ __forceinline__ int scale_exponent(uint32_t a) {
  const int e = int(a >> 7) - 127 - ((a & 127u) == 127u ? 5 : 6);
  return a >= 0x7F80u ? 16 : max(-32, min(16, e));
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(e + 127) << 23); }

// A NaN counts as the infinity of its sign.
__device__ __forceinline__ float no_nan(float x) {
  return x != x ? __uint_as_float((__float_as_uint(x) & 0x80000000u) | 0x7F800000u) : x;
}
__device__ __forceinline__ float clamp127(float x) { return fminf(fmaxf(x, -127.f), 127.f); }

}  // namespace grok
