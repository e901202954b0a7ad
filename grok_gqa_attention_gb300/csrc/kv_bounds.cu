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
// infinities of their sign. Measured (graph replays): 8192 rows of a prompt, 16.8 MB, 5.5
// us, which is the launch, the table's and the keys' latency and 2.5 us of HBM; the blocks
// of a decode step, 32 sequences, 4.0 us.
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
// sequence). The products run on tensor-core instructions: 8-bit codes are exact in
// fp16, and so are sums of whole numbers below 2^24 in fp32:
//   [16 blocks x 8 heads] += codes [16 x 16] . query codes [16 x 8]  (6 of 8 columns used)
// over 256 codes of a block, the upper bounds against the query's positive codes and
// the lower ones against its negative. A lane loads 16-byte words of two blocks; the order
// of the contracted index is chosen to fit them. A warp has the next 16 blocks' codes
// under way while it multiplies. Measured: 32 sequences of 65536 rows (68 MB of codes) 20.2
// us, 3.4 TB/s, of which 3 us are the start, 13 the codes (SMs with two of the 256 CTAs
// read 0.5 MB each, at 40 bytes a clock), 3 the choice; one of 8192 rows 5.5 us. With
// integer products (mma s8) 22.3 us, with dp4a 32.7; with two to four CTAs to a pair,
// in a cluster, 28 and 34: each pays the start again.
constexpr int kSlThreads = 256;
constexpr int kSlWarps = kSlThreads / 32;
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

// D[16 x 8] += A[16 x 16] B[16 x 8], fp16 operands, fp32 sums.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four codes, first in the low byte, as two pairs of fp16: a byte c with its sign bit flipped is c + 128, behind the byte
// 0x64 the fp16 number 1024 + (c + 128), from which 1152 is taken.
__device__ __forceinline__ void codes_to_half(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(lo) : "r"(__byte_perm(u, 0x64646464u, 0x4140)), "r"(0x64806480u));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(hi) : "r"(__byte_perm(u, 0x64646464u, 0x4342)), "r"(0x64806480u));
}

__device__ __forceinline__ uint32_t word_of(const uint4& x, int w) { return w == 0 ? x.x : w == 1 ? x.y : w == 2 ? x.z : x.w; }

__global__ void __launch_bounds__(kSlThreads, 2) select_kernel(const SlParams p) {
  __shared__ __align__(16) uint32_t sq[8][kD + 4];  // [head][2 codes in fp16: positive, negative] (rows apart in the banks)
  __shared__ float sf[8];
  __shared__ int pages[GROK_MAX_POSITION / GROK_PAGE_TOKENS];
  __shared__ float scores[kBlkMax];
  __shared__ uint2 sums[kSlWarps];
  __shared__ uint32_t bins[256];
  __shared__ uint2 found;
  const int g = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cap = p.pm.max_pages * GROK_PAGE_TOKENS;
  const int len = p.kv_len[b];
  // (the whole row of the table: entries behind the sequence's last are not looked at)
  for (int i = tid; i < p.pm.max_pages; i += kSlThreads) pages[i] = p.pm.table[(size_t)b * p.pm.max_pages + i];
  if (warp < kGroup) {  // head `warp` in 8 bits, four features a lane
    const uint2 x = reinterpret_cast<const uint2*>(p.q)[((size_t)b * kQHeads + g * kGroup + warp) * (kD / 4) + lane];
    const uint32_t a = max(max(x.x & 0x7FFFu, (x.x >> 16) & 0x7FFFu), max(x.y & 0x7FFFu, (x.y >> 16) & 0x7FFFu));
    const int f = scale_exponent(__reduce_max_sync(0xffffffffu, a));
    const float inv = pow2(-f), v[4] = {bf16lo_to_f32(x.x), bf16hi_to_f32(x.x), bf16lo_to_f32(x.y), bf16hi_to_f32(x.y)};
    float c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = clamp127(rintf(no_nan(v[i]) * inv));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      sq[warp][2 * lane + i] = pack_f16x2(fmaxf(c[2 * i], 0.f), fmaxf(c[2 * i + 1], 0.f));
      sq[warp][kD / 2 + 2 * lane + i] = pack_f16x2(fminf(c[2 * i], 0.f), fminf(c[2 * i + 1], 0.f));
    }
    if (lane == 0) sf[warp] = pow2(f);
  } else {  // columns 6 and 7 are not used
    if (lane == 0) sf[warp] = 0.f;
    *reinterpret_cast<uint4*>(&sq[warp][4 * lane]) = make_uint4(0u, 0u, 0u, 0u);
  }
  const int n = blk_count(len, cap);
  if (n == 0) {
    if (g == 0 && tid == 0) report(p.status, GROK_DEV_BAD_KV_LEN);
    return;
  }
  __syncthreads();
  {
    const int row = lane >> 2, t = lane & 3;
    uint32_t qb[16][2];  // k-step: the four codes of word s % 4 of 64-byte group s / 4
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      const uint2 w = *reinterpret_cast<const uint2*>(&sq[row][(s >> 2) * 32 + t * 8 + (s & 3) * 2]);
      qb[s][0] = w.x;
      qb[s][1] = w.y;
    }
    const float f0 = sf[2 * t], f1 = sf[2 * t + 1];
    uint4 x[2][4];
    float sc[2];
    // Codes and scales of blocks i0 + row and i0 + 8 + row.
    auto load = [&](int i0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int blk = min(i0 + 8 * h + row, n - 1);
        int pg = pages[blk / kBlkPerPage];
        if (pg < 0 || pg >= p.pm.n_pages) {  // (page 0's bounds in its place)
          report(p.status, GROK_DEV_BAD_PAGE);
          pg = 0;
        }
        const size_t at = ((size_t)pg * kBlkPerPage + blk % kBlkPerPage) * kKVHeads + g;
        const uint4* src = p.codes + at * (2 * kD / 16) + t;
#pragma unroll
        for (int c = 0; c < 4; ++c) x[h][c] = __ldg(src + 4 * c);
        sc[h] = __ldg(p.scale + at);
      }
    };
    float* out = p.score + ((size_t)b * kKVHeads + g) * (p.pm.max_pages * kBlkPerPage);
    int i0 = warp * 16;
    if (i0 < n) load(i0);
    while (i0 < n) {
      uint4 y[2][4];
      float ysc[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        ysc[h] = sc[h];
#pragma unroll
        for (int c = 0; c < 4; ++c) y[h][c] = x[h][c];
      }
      const int next = i0 + kSlWarps * 16;
      if (next < n) load(next);
      float d[2][4] = {};
#pragma unroll
      for (int s = 0; s < 16; ++s) {
        uint32_t a[4];
        codes_to_half(word_of(y[0][s >> 2], s & 3), a[0], a[2]);
        codes_to_half(word_of(y[1][s >> 2], s & 3), a[1], a[3]);
        mma_f16_16816(d[s & 1], a[0], a[1], a[2], a[3], qb[s][0], qb[s][1]);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float best = t < kGroup / 2 ? fmaxf((d[0][2 * h] + d[1][2 * h]) * f0, (d[0][2 * h + 1] + d[1][2 * h + 1]) * f1)
                                    : -INFINITY;
        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 1));
        best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, 2));
        const int i = i0 + 8 * h + row;
        if (t == 0 && i < n) out[i] = scores[i] = best * ysc[h];
      }
      i0 = next;
    }
  }
  __syncthreads();

  // The choice. The first `sink` and the last `recent` blocks are in; the others' keys order as their scores do, and of
  // them the `want` largest are in: all above `edge`, and of those at it the first ones.
  int32_t* sel = p.sel + ((size_t)b * kKVHeads + g) * p.budget;
  const int take = min(n, p.budget), tail = max(p.sink, n - p.recent);  // (blocks from `tail` on are in)
  const int want = take - min(n, p.sink) - max(0, n - tail);
  uint32_t key[kSlPer], top = 0u, low = 0xFFFFFFFFu;
#pragma unroll
  for (int e = 0; e < kSlPer; ++e) {
    const int i = tid * kSlPer + e;
    key[e] = 0u;  // (no score has this key)
    if (i >= p.sink && i < tail && i < n) {
      const uint32_t x = __float_as_uint(scores[i] + 0.f);
      key[e] = max(1u, x ^ (x >> 31 ? 0xFFFFFFFFu : 0x80000000u));  // (a scale that nobody wrote may be any NaN)
      top = max(top, key[e]);
      low = min(low, key[e]);
    }
  }
  uint32_t edge = 0u;
  if (want == 0) {
    edge = 0xFFFFFFFFu;
  } else if (n > take) {
    // (One bit at a time, a sum over the CTA for each, takes 4400 clocks of 128 blocks; this way 1500.)
    // The key of rank `want`, eight bits at a time from the first that any two keys differ in: keys that agree with it so
    // far are counted by their next eight bits.
    top = __reduce_max_sync(0xffffffffu, top);
    low = __reduce_min_sync(0xffffffffu, low);
    if (lane == 0) sums[warp] = make_uint2(top, low);
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSlWarps; ++w) {
      top = max(top, sums[w].x);
      low = min(low, sums[w].y);
    }
    const int differ = 32 - __clz(top ^ low);
    int rank = want;
    edge = differ == 32 ? 0u : top >> differ << differ;
    for (int bits = differ; bits > 0;) {
      const int shift = max(0, bits - 8);
      static_assert(kSlThreads == 256, "a bin a thread");
      bins[tid] = 0u;
      __syncthreads();
#pragma unroll
      for (int e = 0; e < kSlPer; ++e)
        if (key[e] && (bits == 32 || (key[e] ^ edge) >> bits == 0)) atomicAdd(&bins[key[e] >> shift & 255u & ((1u << (bits - shift)) - 1u)], 1u);
      __syncthreads();
      const uint32_t bin = 255u - tid, mine = bins[bin];  // (the largest first)
      uint32_t upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += up;
      }
      if (lane == 31) sums[warp].x = upto;
      __syncthreads();
      for (int w = 0; w < warp; ++w) upto += sums[w].x;
      if (upto >= uint32_t(rank) && upto - mine < uint32_t(rank)) found = make_uint2(bin, (upto - mine) << 16 | mine);
      __syncthreads();
      edge |= found.x << shift;
      rank -= int(found.y >> 16);
      bits = shift;
      if (rank == int(found.y & 0xFFFFu)) break;  // all of them are in: those at or above `edge` as it stands
    }
    __syncthreads();
  }
  // In, and in order: the blocks that are always in count as above the edge (counts packed: above in the low half).
  uint32_t kind[kSlPer], mine = 0;
#pragma unroll
  for (int e = 0; e < kSlPer; ++e) {
    const int i = tid * kSlPer + e;
    kind[e] = i >= n ? 0u : i < p.sink || i >= tail || key[e] > edge ? 1u : key[e] == edge ? 0x10000u : 0u;
    mine += kind[e];
  }
  uint32_t before = mine;
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const uint32_t up = __shfl_up_sync(0xffffffffu, before, d);
    if (lane >= d) before += up;
  }
  if (lane == 31) sums[warp].x = before;
  __syncthreads();
  uint32_t all = 0, base = 0;
#pragma unroll
  for (int w = 0; w < kSlWarps; ++w) {
    if (w < warp) base += sums[w].x;
    all += sums[w].x;
  }
  before += base - mine;
  const int ties = take - int(all & 0xFFFFu);  // of those at the edge
  int above = int(before & 0xFFFFu), equal = int(before >> 16);
#pragma unroll
  for (int e = 0; e < kSlPer; ++e) {
    const int at = above + min(equal, ties);
    if (kind[e] == 1u) {
      sel[at] = tid * kSlPer + e;
      ++above;
    } else if (kind[e]) {
      if (equal < ties) sel[at] = tid * kSlPer + e;
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
