// Bounds of the keys of each 64-token block, and the blocks that a query reads.
//
// A decode step over a long cache (code-reading guide ch. 4 §4.4.1, §4.5.2) needs
// the keys with large logits; the others' softmax weights are next to nothing. For
// every block and KV head the cache's owner keeps, per feature d, the largest and
// the smallest key in 8 bits with one power of two as scale:
//   u_d = ceil(max_j k_jd / 2^e), l_d = floor(min_j k_jd / 2^e)
// and a query head in 8 bits, q_d = c_d 2^f, is bounded over the whole block by
//   max_j q . k_j <= 2^(e + f) sum_d max(c_d u_d, c_d l_d)
//                  = 2^(e + f) (sum_d max(c_d, 0) u_d + sum_d min(c_d, 0) l_d).
// The sum is of whole numbers below 2^21 and the scales are powers of two, so a
// score is exact in any order of summation: which blocks are chosen is a function
// of the cache and the query alone.
#include "block_decode.cuh"

namespace grok {

// ----------------------------------------------------------------------------
// Bounds of the blocks that rows [start, start + valid) touch, from their rows so
// far. A CTA takes two KV heads of a block (32 KB of keys): warp w reads rows w,
// w + 8, ..., 512 contiguous bytes each, all loads in flight at once. bf16 bits
// order as 16-bit integers once the lower bits of negative numbers are flipped, so
// a maximum is one packed instruction for two features; NaNs order beyond the
// infinities of their sign.
constexpr int kBdThreads = 256;
constexpr int kBdRows = kBlk / (kBdThreads / 32);  // rows per warp

__device__ __forceinline__ uint32_t order16(uint32_t x) { return x ^ (((x >> 15) & 0x00010001u) * 0x7FFFu); }

__global__ void __launch_bounds__(kBdThreads) kv_bounds_kernel(const uint4* __restrict__ k_pool, PageMap pm,
                                                               const int32_t* __restrict__ start_pos,
                                                               const int32_t* __restrict__ valid_len, int T,
                                                               uint16_t* __restrict__ codes, float* __restrict__ scale,
                                                               int32_t* status) {
  __shared__ uint4 part[2][kBdThreads / 32][32];  // [upper, lower][warp][lane]
  __shared__ uint32_t top[kBdThreads / 32];
  const int b = blockIdx.y, pair = blockIdx.x % (kKVHeads / 2), nth = blockIdx.x / (kKVHeads / 2);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int s = start_pos[b], n = valid_len ? valid_len[b] : T;
  const int bad = (s < 0 || (long long)s + T > (long long)pm.max_pages * GROK_PAGE_TOKENS ? GROK_DEV_BAD_START : 0) |
                  (n < 1 || n > T ? GROK_DEV_BAD_VALID : 0);
  if (bad) {
    if (blockIdx.x == 0 && tid == 0) report(status, bad);
    return;
  }
  const int blk = s / kBlk + nth, end = s + n;
  if (blk * kBlk >= end) return;
  const int pg = pm.table[(size_t)b * pm.max_pages + blk / kBlkPerPage];
  if (pg < 0 || pg >= pm.n_pages) {
    if (tid == 0) report(status, GROK_DEV_BAD_PAGE);
    return;
  }
  const int rows = min(kBlk, end - blk * kBlk);
  const size_t at = (size_t)pg * kBlkPerPage + blk % kBlkPerPage;  // of the pool's blocks

  uint32_t hi[4], lo[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) hi[q] = 0x80008000u, lo[q] = 0x7FFF7FFFu;
  const uint4* src = k_pool + (at * kBlk * kKVHeads + pair * 2) * (kD / 8) + lane;
  uint4 x[kBdRows];
#pragma unroll
  for (int i = 0; i < kBdRows; ++i) {
    const int r = warp + i * (kBdThreads / 32);
    if (r < rows) x[i] = __ldg(src + r * (kKVHeads * kD / 8));
  }
#pragma unroll
  for (int i = 0; i < kBdRows; ++i)
    if (warp + i * (kBdThreads / 32) < rows) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        hi[q] = __vmaxs2(hi[q], order16(w[q]));
        lo[q] = __vmins2(lo[q], order16(w[q]));
      }
    }
  part[0][warp][lane] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  part[1][warp][lane] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  __syncthreads();
  // Thread (which, word): the upper or the lower bound of two features.
  const int which = tid >> 7, word = tid & 127;
  uint32_t m = reinterpret_cast<const uint32_t*>(part[which][0])[word];
#pragma unroll
  for (int w = 1; w < kBdThreads / 32; ++w) {
    const uint32_t v = reinterpret_cast<const uint32_t*>(part[which][w])[word];
    m = which ? __vmins2(m, v) : __vmaxs2(m, v);
  }
  m = order16(m);  // bf16 bits again
  const uint32_t mag = __reduce_max_sync(0xffffffffu, max(m & 0x7FFFu, (m >> 16) & 0x7FFFu));
  if (lane == 0) top[warp] = mag;
  __syncthreads();
  const int head = word >> 6;  // of the pair: words 0..63, 64..127, warps 0, 1, 4, 5 and 2, 3, 6, 7
  const int e = scale_exponent(max(max(top[2 * head], top[2 * head + 1]), max(top[2 * head + 4], top[2 * head + 5])));
  const float inv = pow2(-e);
  const float x0 = no_nan(bf16lo_to_f32(m)) * inv, x1 = no_nan(bf16hi_to_f32(m)) * inv;
  const int c0 = int(clamp127(which ? floorf(x0) : ceilf(x0))), c1 = int(clamp127(which ? floorf(x1) : ceilf(x1)));
  const size_t row = at * kKVHeads + pair * 2 + head;  // of (block, head)
  codes[(row * 2 + which) * (kD / 2) + (word & 63)] = uint16_t((c0 & 0xFF) | ((c1 & 0xFF) << 8));
  if (which == 0 && (word & 63) == 0) scale[row] = pow2(e);
}

// ----------------------------------------------------------------------------
// Scores of a sequence's blocks for one KV head, and the choice. A CTA per (KV head,
// sequence); four threads share a block: two take the upper bounds with the query's
// positive codes, two the lower bounds with the negative ones.
constexpr int kSlThreads = 256;
constexpr int kSlPer = kBlkMax / kSlThreads;  // blocks per thread in the choice

struct SlParams {
  const uint32_t* q;  // [B, 48, 64] pairs of bf16
  const uint4* codes;
  const float* scale;
  PageMap pm;
  const int32_t* kv_len;
  int budget, sink, recent;
  float* score;
  int32_t* sel;
  int32_t* status;
};

__global__ void __launch_bounds__(kSlThreads) select_kernel(const SlParams p) {
  __shared__ uint32_t sq[kGroup][2][kD / 4];  // [head][positive, negative][4 codes]
  __shared__ float sf[kGroup];
  __shared__ float scores[kBlkMax];
  __shared__ int sums[2][kSlThreads / 32];
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = p.pm.max_pages * GROK_PAGE_TOKENS, n = blk_count(p.kv_len[b], cap);
  if (n == 0) {
    if (g == 0 && tid == 0) report(p.status, GROK_DEV_BAD_KV_LEN);
    return;
  }
  if (warp < kGroup) {  // head `warp` in 8 bits, four features a lane
    const uint2 x = reinterpret_cast<const uint2*>(p.q)[((size_t)b * kQHeads + g * kGroup + warp) * (kD / 4) + lane];
    const uint32_t a = max(max(x.x & 0x7FFFu, (x.x >> 16) & 0x7FFFu), max(x.y & 0x7FFFu, (x.y >> 16) & 0x7FFFu));
    const int f = scale_exponent(__reduce_max_sync(0xffffffffu, a));
    const float inv = pow2(-f), v[4] = {bf16lo_to_f32(x.x), bf16hi_to_f32(x.x), bf16lo_to_f32(x.y), bf16hi_to_f32(x.y)};
    uint32_t pos = 0, neg = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = int(clamp127(rintf(no_nan(v[i]) * inv)));
      pos |= uint32_t(max(c, 0) & 0xFF) << (8 * i);
      neg |= uint32_t(min(c, 0) & 0xFF) << (8 * i);
    }
    sq[warp][0][lane] = pos;
    sq[warp][1][lane] = neg;
    if (lane == 0) sf[warp] = pow2(f);
  }
  __syncthreads();
  const int part = tid & 3;
  uint32_t qw[kGroup][16];
#pragma unroll
  for (int h = 0; h < kGroup; ++h)
#pragma unroll
    for (int w = 0; w < 16; ++w) qw[h][w] = sq[h][part >> 1][(part & 1) * 16 + w];
  float* out = p.score + ((size_t)b * kKVHeads + g) * (p.pm.max_pages * kBlkPerPage);
  for (int i0 = 0; i0 < n; i0 += kSlThreads / 4) {
    const int i = i0 + (tid >> 2), blk = min(i, n - 1);
    const int pg = max(0, blk_page(p.pm, b, blk, p.status));  // (a bad page: reported, page 0's bounds)
    const size_t row = ((size_t)pg * kBlkPerPage + blk % kBlkPerPage) * kKVHeads + g;
    const uint4* src = p.codes + row * (2 * kD / 16) + part * 4;
    uint4 x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = __ldg(src + c);
    const float sc = __ldg(p.scale + row);
    int acc[kGroup] = {};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
#pragma unroll
        for (int h = 0; h < kGroup; ++h) acc[h] = __dp4a(int(w[k]), int(qw[h][c * 4 + k]), acc[h]);
    }
    float best = -INFINITY;
#pragma unroll
    for (int h = 0; h < kGroup; ++h) {
      acc[h] += __shfl_xor_sync(0xffffffffu, acc[h], 1);
      acc[h] += __shfl_xor_sync(0xffffffffu, acc[h], 2);
      best = fmaxf(best, float(acc[h]) * sf[h]);
    }
    if (part == 0 && i < n) out[i] = scores[i] = best * sc;
  }
  __syncthreads();

  // The choice. Keys order as the scores do; blocks that are always chosen come first.
  int32_t* sel = p.sel + ((size_t)b * kKVHeads + g) * p.budget;
  const int take = min(n, p.budget);
  uint32_t key[kSlPer];
#pragma unroll
  for (int e = 0; e < kSlPer; ++e) {
    const int i = tid * kSlPer + e;
    key[e] = 0u;
    if (i < n) {
      const uint32_t x = __float_as_uint(scores[i] + 0.f);
      key[e] = i < p.sink || i >= n - p.recent ? 0xFFFFFFFFu : x ^ (x >> 31 ? 0xFFFFFFFFu : 0x80000000u);
    }
  }
  // The largest `edge` with at least `take` keys at or above it.
  uint32_t edge = 0;
  if (n > take) {
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t trial = edge | (1u << bit);
      int c = 0;
#pragma unroll
      for (int e = 0; e < kSlPer; ++e) c += key[e] >= trial;
      c = __reduce_add_sync(0xffffffffu, c);
      if (lane == 0) sums[bit & 1][warp] = c;
      __syncthreads();
      int total = 0;
#pragma unroll
      for (int w = 0; w < kSlThreads / 32; ++w) total += sums[bit & 1][w];
      if (total >= take) edge = trial;
      if (total == take) break;
    }
    __syncthreads();
  }
  // Blocks above the edge, and of those at it the first ones (counts packed: above in the low half).
  uint32_t mine = 0;
#pragma unroll
  for (int e = 0; e < kSlPer; ++e)
    if (tid * kSlPer + e < n) mine += key[e] > edge ? 1u : key[e] == edge ? 0x10000u : 0u;
  uint32_t before = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += up;
  }
  if (lane == 31) sums[0][warp] = int(before);
  __syncthreads();
  uint32_t all = 0, base = 0;
#pragma unroll
  for (int w = 0; w < kSlThreads / 32; ++w) {
    if (w < warp) base += uint32_t(sums[0][w]);
    all += uint32_t(sums[0][w]);
  }
  before += base - mine;
  const int ties = take - int(all & 0xFFFFu);  // of those at the edge
  int above = int(before & 0xFFFFu), equal = int(before >> 16);
#pragma unroll
  for (int e = 0; e < kSlPer; ++e) {
    const int i = tid * kSlPer + e;
    if (i >= n) break;
    const int at = above + min(equal, ties);
    if (key[e] > edge) {
      sel[at] = i;
      ++above;
    } else if (key[e] == edge) {
      if (equal < ties) sel[at] = i;
      ++equal;
    }
  }
  for (int i = take + tid; i < p.budget; i += kSlThreads) sel[i] = -1;
}

}  // namespace grok

using namespace grok;

extern "C" grok_status grok_kv_bounds_paged(const grok_bf16* k_pool, int n_pages, const int32_t* block_table,
                                            int max_pages, const int32_t* start_pos, const int32_t* valid_len, int B,
                                            int T, int8_t* codes, float* scale, int32_t* dev_status, void* stream) {
  if (!k_pool || !block_table || !start_pos || !codes || !scale)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv_bounds_paged: null pointer");
  if (!aligned16(k_pool) || !aligned16(codes))
    return fail(GROK_ERR_INVALID_ARG, "grok_kv_bounds_paged: k_pool and codes must be 16-byte aligned");
  grok_status st = page_args(n_pages, max_pages, B, "grok_kv_bounds_paged");
  if (st != GROK_OK) return st;
  if (T < 1 || T > max_pages * GROK_PAGE_TOKENS)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv_bounds_paged: need 1 <= T <= max_pages * %d (T=%d max_pages=%d)",
                GROK_PAGE_TOKENS, T, max_pages);
  int sms = 0;
  if ((st = device_sm_count(&sms)) != GROK_OK) return st;
  const int touched = (T + 2 * kBlk - 2) / kBlk;  // blocks that T rows can touch
  kv_bounds_kernel<<<dim3(touched * (kKVHeads / 2), B), kBdThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      reinterpret_cast<const uint4*>(k_pool), PageMap{block_table, max_pages, n_pages}, start_pos, valid_len, T,
      reinterpret_cast<uint16_t*>(codes), scale, dev_status);
  return check_launch("kv_bounds");
}

extern "C" grok_status grok_attn_select_paged(const grok_bf16* q_rot, const int8_t* codes, const float* scale,
                                              int n_pages, const int32_t* block_table, int max_pages,
                                              const int32_t* kv_len, int B, int budget, int sink, int recent,
                                              float* score, int32_t* sel, int32_t* dev_status, void* stream) {
  if (!q_rot || !codes || !scale || !block_table || !kv_len || !score || !sel)
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_select_paged: null pointer");
  if (!aligned16(q_rot) || !aligned16(codes))
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_select_paged: q_rot and codes must be 16-byte aligned");
  grok_status st = page_args(n_pages, max_pages, B, "grok_attn_select_paged");
  if (st != GROK_OK) return st;
  if (budget < 1 || budget > kBlkMax || sink < 0 || recent < 0 || (long long)sink + recent > budget)
    return fail(GROK_ERR_INVALID_ARG,
                "grok_attn_select_paged: need 1 <= budget <= %d, sink, recent >= 0, sink + recent <= budget "
                "(budget=%d sink=%d recent=%d)",
                kBlkMax, budget, sink, recent);
  int sms = 0;
  if ((st = device_sm_count(&sms)) != GROK_OK) return st;
  SlParams p;
  p.q = reinterpret_cast<const uint32_t*>(q_rot);
  p.codes = reinterpret_cast<const uint4*>(codes);
  p.scale = scale;
  p.pm = PageMap{block_table, max_pages, n_pages};
  p.kv_len = kv_len;
  p.budget = budget;
  p.sink = sink;
  p.recent = recent;
  p.score = score;
  p.sel = sel;
  p.status = dev_status;
  select_kernel<<<dim3(kKVHeads, B), kSlThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return check_launch("select");
}
