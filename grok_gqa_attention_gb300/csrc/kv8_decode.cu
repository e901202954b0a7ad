// Single-token attention over the 8-bit KV cache, and the blocks' weights.
//
// Code-reading guide ch. 4 §4.4.1, §4.5.2-§4.5.4 (decode over the cache, GQA
// logits, cap, softmax, weighted sum), over codes with a scale per 64-token
// block and KV head:
//   x_j = (q . kcode_j) ks / sqrt(128),  z_j = log2(e) (30 tanh(x_j / 30) - 30),
//   out = sum_j 2^(z_j - m) vs vcode_j / sum_j 2^(z_j - m).
//
// Memory-bound: 16 KB of codes per block of 64 tokens and KV head are read once.
// Every warp is a worker of its own: the blocks of all (sequence, head) pairs, in
// order, are dealt out in equal contiguous shares, so the load is even for any
// lengths and no barrier joins warps. A worker streams its blocks through a
// private K and a private V buffer in shared memory (one bulk copy each, of 8 KB),
// and writes one partial result (m, l, O) per pair that it touches; a second
// kernel, launched as a dependent, joins a pair's partials. Which blocks make a
// partial follows from the lengths alone, so the bits do too. Calls of a few tokens
// run here as well (kFew).
//
// Measured (graph replays, one GB300): 32 sequences of up to 8192 rows (274 MB of
// codes) 52.1 us, 5.26 TB/s, 0.78 of the copy rate; 16 of up to 65536 (1.14 GB) 179 us,
// 6.38 TB/s, 0.94; one of 300 rows 6.2 us. Of the 52 us about 3 are the join, 45 the
// loads alone, the rest what the products do not hide. Ten warps with two buffers
// read as fast as any other split of the shared memory tried (14 x 2, 12 x 2, 9 x 3,
// 8 x 3, 7 x 4, within 3 %).
//
// Per block, on fp16 tensor-core products (codes convert to fp16 exactly, q is
// scaled to fp16 by a power of two per head):
//   S^T [64 keys x 8 heads] = K q^T   (4 tiles of 16 keys; 6 of the 8 columns used)
//   O^T [128 x 8] += V^T P^T          (8 tiles of 16 features)
// The transposed form wastes 2 of 8 columns where rows of heads would waste 10 of
// 16. S^T leaves the accumulators as P^T needs it but for one 8 x 8 transpose per
// register (movmatrix). K rows and V columns are both contiguous bytes in a
// block, so a thread reads operands as 16-byte words and the order of the
// contracted index is chosen to fit them: thread t of a row's four holds
// features (keys) 16 t .. 16 t + 15.
// kFew: four tokens of a sequence are 24 columns, three tiles without waste, over
// one pass: their codes are loaded and converted once. A column has the keys that
// its token sees. Two more tiles' outputs and scores leave registers for four warps
// per CTA (255 each) and put the queries in shared memory. Four tokens of 8
// sequences behind 8000 rows 41.6 us (72 as four single ones), 32 tokens behind
// 16000 rows 66 us; without four tokens to fill it a pass costs more than a single
// token's (1 token, 300 rows: 9.8 us against 6.3).
// P is rounded once to fp16 against a running reference: the maximum puts P at 2^7
// and may outgrow that by 2^8 before the reference follows it. A weight is off by
// 2^-11 of itself, or where it is below 2^-21 of the largest by 2^-32 of that (2^-16
// for 65536 of them). l, the weights and O stay in fp32.
#include <algorithm>
#include <cfloat>

#include "host.cuh"
#include "kv8.cuh"

namespace grok {

constexpr int kDqWarps = 5;
constexpr int kDqCtas = 2;  // CTAs resident on an SM
constexpr int kDqBufs = 2;  // a warp's ring: K and V of its blocks in turn
constexpr int kDqThreads = kDqWarps * 32;
constexpr int kDqRing = kDqBufs * kKv8Bytes;
constexpr int kDqSmem = kDqWarps * kDqRing + kDqWarps * kDqBufs * 8 + 16;
static_assert(kDqCtas * (kDqSmem + 1024) <= 233472, "shared memory per SM");
// A call of few tokens: this many share a pass over the codes, 24 columns, three tiles of 8.
constexpr int kDqTok = 4;
constexpr int kDqFewCols = kDqTok * kGroup;
constexpr int kDqFewQ = 8 * (kDqFewCols / 8) * 32 * 8;  // a warp's queries as operands, in shared memory
constexpr int kDqFewWarps = 4;  // two warps on a scheduler, up to 255 registers each
constexpr int kDqFewThreads = kDqFewWarps * 32;
constexpr int kDqFewSmem = kDqFewWarps * (kDqRing + kDqFewQ) + kDqFewWarps * kDqBufs * 8 + 16;
static_assert(kDqCtas * (kDqFewSmem + 1024) <= 233472, "shared memory per SM");
constexpr float kDqNone = -1.0e4f;  // reference of a column that has seen no key
constexpr int kDqLong = 24;  // blocks per worker from which a second wave of small shares pays
constexpr float kDqTop = 7.f;  // log2 of the weight of the maximum that sets the reference
constexpr float kDqLag = 15.f;  // log2 units that a weight may reach before the reference follows

struct DqParams {
  grok_kv8_cache c;
  const uint4* q;
  const int32_t* kv_len;     // rows that a query sees; kFew: rows before the call's tokens
  const int32_t* valid_len;  // kFew: valid tokens of a sequence, or null (all)
  int few_tokens;  // kFew: tokens per sequence
  int n_seq;       // what a pair is one KV head of: sequences, or (kFew) groups of kDqTok tokens of a sequence
  float* part_o;    // [slot][6][128] (kFew: 24 for 6)
  float2* part_ml;  // [slot][6]: reference (log2), sum
  int2* pair_parts; // [n_seq * 8]: a pair's first slot and number of slots
  float* block_w;   // [n_seq * 8][max_blocks][8]: a block's weights per head on the fixed reference 30
  uint2* out;
  const float* weight_in;
  float* weight_out;
  int wave, second;  // workers of the CTAs resident at a time, and of those behind them
  int32_t* status;
};

// How `total` blocks are dealt out. The SMs do not all read at the same rate (with
// equal shares the mean SM is done at 0.82 of the slowest's time). Where shares are
// long, 7/8 of the blocks are dealt to the `wave` workers that start at once and the
// rest, in small shares, to a second wave of CTAs that take SMs as they come free
// (128 sequences of up to 8192 rows: 184.6 -> 178.7 us; 16 of 65536: 185.1 -> 179.1).
// With short shares the second wave's start costs more than it evens out (32
// sequences: 52.2 us without, 56.2 with).
struct Deal {
  int first, big, small;
  __device__ __forceinline__ Deal(int total, int wave, int second) {
    big = second && total >= kDqLong * wave ? int((long long)total * 7 / 8 / wave) : 0;
    first = big > 0 ? wave : 0;
    const int slots = first ? second : wave;
    small = max(1, (total - big * first + slots - 1) / slots);
  }
  __device__ __forceinline__ int start(int item) const {
    return item < first ? item * big : first * big + (item - first) * small;
  }
  __device__ __forceinline__ int item_of(int block) const {
    return block < first * big ? block / big : first + (block - first * big) / small;
  }
};

__device__ __forceinline__ uint32_t word_of(const uint4& x, int w) {
  return w == 0 ? x.x : w == 1 ? x.y : w == 2 ? x.z : x.w;
}

__host__ __device__ __forceinline__ int groups_of(int tokens) { return (tokens + kDqTok - 1) / kDqTok; }

// (This kernel starts beside the one before it, which may write any of its inputs: they are loaded behind the wait, and
// not by the read-only path, which supposes that they stay as they are while the kernel runs.)
// Rows that v's queries see: 0 when its sequence's integers are bad. kFew: those of
// the group's last token (token i sees the rows before the call and the valid
// tokens' up to its own). (A template: the choice at run time costs a call over
// 300 rows 0.3 of its 6.2 us.)
template <bool kFew>
__device__ __forceinline__ int rows_of(const DqParams& p, int v) {
  if (!kFew) return p.kv_len[v];
  const int groups = groups_of(p.few_tokens), b = v / groups, first = v % groups * kDqTok;
  const int s = p.kv_len[b], n = p.valid_len ? p.valid_len[b] : p.few_tokens;
  if (s < 0 || n < 1 || n > p.few_tokens || (long long)s + n > (long long)p.c.max_blocks * kKv8Block) return 0;
  return s + min(first + kDqTok, n);
}
template <bool kFew>
__device__ __forceinline__ int blocks_of(const DqParams& p, int v) {
  return kv8_blocks(rows_of<kFew>(p, v), p.c.max_blocks);
}

// Bits for a query whose sequence's integers are bad (as the many-token kernel reports them).
template <bool kFew>
__device__ __forceinline__ int bad_bits(const DqParams& p, int v) {
  if (!kFew) return GROK_DEV_BAD_KV_LEN;
  const int b = v / groups_of(p.few_tokens);
  const int s = p.kv_len[b], n = p.valid_len ? p.valid_len[b] : p.few_tokens;
  return (n < 1 || n > p.few_tokens ? GROK_DEV_BAD_VALID : 0) |
         (s < 0 || (long long)s + max(n, 0) > (long long)p.c.max_blocks * kKv8Block ? GROK_DEV_BAD_KV_LEN : 0);
}

// The queries' blocks: total over the batch of ceil(rows / 64), by one warp.
template <bool kFew>
__device__ __forceinline__ int count_blocks(const DqParams& p, int lane) {
  int total = 0;
  for (int c = 0; c < p.n_seq; c += 32)
    total += __reduce_add_sync(0xffffffffu, c + lane < p.n_seq ? blocks_of<kFew>(p, c + lane) : 0);
  return total;
}

template <int kKind, bool kWeights, bool kFew>
__global__ void __launch_bounds__(kFew ? kDqFewThreads : kDqThreads, kDqCtas) kv8_decode_kernel(const DqParams p) {
  constexpr int kWarps = kFew ? kDqFewWarps : kDqWarps;
  constexpr int kTiles = kFew ? kDqFewCols / 8 : 1;  // of 8 columns: a column is a query head of a token
  constexpr int kCols = kFew ? kDqFewCols : kGroup;
  extern __shared__ __align__(128) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = lane >> 2, t = lane & 3;
  constexpr int kData = kWarps * (kDqRing + (kFew ? kDqFewQ : 0));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kData);
  int* abort_flag = reinterpret_cast<int*>(bars + kDqBufs * kWarps);
  volatile int* abort = abort_flag;
  bars += kDqBufs * warp;
  uint8_t* ring = smem + warp * kDqRing;
  if (lane == 0) {
    for (int i = 0; i < kDqBufs; ++i) mbar_init(&bars[i], 1);
    if (warp == 0) *abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int n_total = kKVHeads * count_blocks<kFew>(p, lane);
  const Deal deal(n_total, p.wave, p.second);
  const int n_first = p.wave / kWarps, cta = blockIdx.x;
  const int item = cta < n_first ? warp * n_first + cta : cta * kWarps + warp;  // (few blocks: over the SMs first)
  if (item == 0)
    for (int v = lane; v < p.n_seq; v += 32)
      if (blocks_of<kFew>(p, v) == 0) report(p.status, bad_bits<kFew>(p, v));
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // (item * small passes n_total by less than a wave of shares: no overflow below 2^31)
  const int lo = min(deal.start(item), n_total), hi = min(deal.start(item + 1), n_total);
  if (lo >= hi) return;

  uint32_t qb[8][2];  // (kFew: in shared memory)
  uint2* sq = reinterpret_cast<uint2*>(smem + kWarps * kDqRing + warp * kDqFewQ) + lane;
  // of columns 8 nt + 2 t, 8 nt + 2 t + 1
  float q_scale[kTiles][2], o[kTiles][8][4], m[kTiles][2], l[kTiles][2];
  int seen = 0;  // kFew: tokens of the group up to the last valid one
  int pair = -1;
  int buf = 0, next_buf = 0;         // buffers of the next piece to read and to load (a piece: a block's K or V)
  uint32_t phase = 0;                // of buffer `buf`
  int due = 0;                       // pieces loaded and not yet waited for
  bool ok = true;

  // One partial result: this item's share of a pair.
  auto flush = [&]() {
    const size_t slot = (size_t)item + pair;
#pragma unroll
    for (int nt = 0; nt < kTiles; ++nt) {
#pragma unroll
      for (int d = 4; d < 32; d *= 2) {
        l[nt][0] += __shfl_xor_sync(0xffffffffu, l[nt][0], d);
        l[nt][1] += __shfl_xor_sync(0xffffffffu, l[nt][1], d);
      }
      if (kFew || t < kGroup / 2) {
        const int c = 8 * nt + 2 * t;
        float* po = p.part_o + (slot * kCols + c) * kD + row;
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          po[16 * mt] = o[nt][mt][0];
          po[16 * mt + kD] = o[nt][mt][1];
          po[16 * mt + 8] = o[nt][mt][2];
          po[16 * mt + 8 + kD] = o[nt][mt][3];
        }
        if (row == 0) {
          p.part_ml[slot * kCols + c] = make_float2(m[nt][0], l[nt][0]);
          p.part_ml[slot * kCols + c + 1] = make_float2(m[nt][1], l[nt][1]);
        }
      }
    }
  };

  for (int base = lo; base < hi && ok; base += 32) {
    const int cnt = min(32, hi - base);
    // Each lane finds one block of the batch: its pair, number, scales and visible keys.
    int my_pair = 0, my_blk = 0, my_keys = 0;
    {
      const int idx = base + lane;
      bool found = lane >= cnt;
      int cum = 0;
      for (int c = 0; c < p.n_seq; c += 32) {
        const int len = c + lane < p.n_seq ? rows_of<kFew>(p, c + lane) : 0;
        const int n = kv8_blocks(len, p.c.max_blocks);
        int incl = n;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int up = __shfl_up_sync(0xffffffffu, incl, d);
          if (lane >= d) incl += up;
        }
        const int rest = idx - kKVHeads * cum;
        int s = 0;  // the sequence of this chunk that holds block `rest`
#pragma unroll
        for (int step = 16; step; step /= 2)
          if (kKVHeads * __shfl_sync(0xffffffffu, incl, s + step - 1) <= rest) s += step;
        s = min(s, 31);
        const int sn = __shfl_sync(0xffffffffu, n, s), si = __shfl_sync(0xffffffffu, incl, s);
        const int sl = __shfl_sync(0xffffffffu, len, s);
        const int chunk = __shfl_sync(0xffffffffu, incl, 31);
        if (!found && rest < kKVHeads * chunk) {
          const int in = rest - kKVHeads * (si - sn);
          my_pair = (c + s) * kKVHeads + in / sn;
          my_blk = in % sn;
          my_keys = min(2 * kKv8Block, sl - my_blk * kKv8Block);  // (up to the last row)
          found = true;
          if (my_blk == 0) p.pair_parts[my_pair] = make_int2(item + my_pair, deal.item_of(idx + sn - 1) - item + 1);
        }
        cum += chunk;
        if (__all_sync(0xffffffffu, found)) break;
      }
    }
    int my_id = 0;
    float my_ks = 0.f, my_vs = 0.f;
    if (lane < cnt) {
      size_t row_of = my_pair;  // of the table
      if (kFew) row_of = (size_t)(my_pair / kKVHeads / groups_of(p.few_tokens)) * kKVHeads + my_pair % kKVHeads;
      my_id = max(0, kv8_block_id(p.c.table, row_of * p.c.max_blocks + my_blk, p.c.n_blocks, p.status));
      my_ks = p.c.k_scale[my_id];
      my_vs = p.c.v_scale[my_id];
      // (a token that does not see the block meets its V scale: what is not finite shows in the logits)
      if (kFew && my_vs != my_vs) my_ks = my_vs, my_vs = 0.f;
    }
    int loaded = 0;  // pieces of this batch
    auto load = [&]() {
      const bool v = loaded & 1;
      const int id = __shfl_sync(0xffffffffu, my_id, loaded >> 1);
      if (lane == 0) {
        mbar_arrive_expect_tx(&bars[next_buf], kKv8Bytes);
        bulk_load(ring + next_buf * kKv8Bytes,
                  static_cast<const uint8_t*>(v ? p.c.v_pool : p.c.k_pool) + (size_t)id * kKv8Bytes, kKv8Bytes,
                  &bars[next_buf]);
      }
      next_buf = next_buf + 1 == kDqBufs ? 0 : next_buf + 1;
      ++loaded;
      ++due;
    };
    auto wait = [&]() {
      ok = __all_sync(0xffffffffu, mbar_wait(&bars[buf], phase, abort, p.status));
      return ok;
    };
    // The piece in `buf` is read by every lane: its place takes the next one.
    auto release = [&]() {
      __syncwarp();
      --due;
      if (buf + 1 == kDqBufs) {
        buf = 0;
        phase ^= 1;
      } else {
        ++buf;
      }
      if (loaded < 2 * cnt) load();
    };
    for (int i = 0; i < kDqBufs && i < 2 * cnt; ++i) load();
    for (int j = 0; j < cnt; ++j) {
      const int jp = __shfl_sync(0xffffffffu, my_pair, j);
      if (jp != pair) {  // the next pair: its partial starts empty, its six queries come in
        if (pair >= 0) flush();
        pair = jp;
        int b = 0, first = 0;
        if (kFew) {
          const int groups = groups_of(p.few_tokens), v = pair / kKVHeads;
          b = v / groups, first = v % groups * kDqTok;
          seen = min(kDqTok, (p.valid_len ? p.valid_len[b] : p.few_tokens) - first);
        }
        uint4 xs[kTiles][4];
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) {  // the query row of this lane's column
          const int c = 8 * nt + row, tok = first + c / kGroup;
          const bool live = kFew ? tok < p.few_tokens : row < kGroup;
          const size_t at =
              kFew ? (((size_t)b * p.few_tokens + tok) * kKVHeads + pair % kKVHeads) * kGroup + c % kGroup
                   : (size_t)pair * kGroup + row;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            xs[nt][i] = make_uint4(0, 0, 0, 0);
            if (live) xs[nt][i] = p.q[at * 16 + (i >> 1) * 8 + 2 * t + (i & 1)];
          }
        }
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) {
          m[nt][0] = m[nt][1] = kDqNone;
          l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) o[nt][mt][0] = o[nt][mt][1] = o[nt][mt][2] = o[nt][mt][3] = 0.f;
          const uint4 (&x)[4] = xs[nt];
          uint32_t top = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            top = __vmaxu2(top, __vmaxu2(__vmaxu2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu),
                                         __vmaxu2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu)));
          top = max(top & 0xFFFFu, top >> 16);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // q / 2^e with the largest element in [1, 2): what falls below fp16's normal range is off by 2^-25 at most
          const uint32_t e = min(max(top >> 7, 1u), 253u);
          const float down = __uint_as_float((254u - e) << 23), up = __uint_as_float(e << 23);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int c4 = 0; c4 < 4; c4 += 2) {
              const int u = (i >> 1) * 4 + (i & 1) * 2 + (c4 >> 1);  // product of the 16 features 64 (i >> 1) + 16 t + ..
              const uint32_t y0 = pack_f16x2(bf16lo_to_f32(w[c4]) * down, bf16hi_to_f32(w[c4]) * down);
              const uint32_t y1 = pack_f16x2(bf16lo_to_f32(w[c4 + 1]) * down, bf16hi_to_f32(w[c4 + 1]) * down);
              if (kFew) {
                sq[(nt * 8 + u) * 32] = make_uint2(y0, y1);  // (read by this lane alone)
              } else {
                qb[u][0] = y0, qb[u][1] = y1;
              }
            }
          }
          q_scale[nt][0] = __shfl_sync(0xffffffffu, up, 8 * t) * (2.f * kY * kLog2e);
          q_scale[nt][1] = __shfl_sync(0xffffffffu, up, 8 * t + 4) * (2.f * kY * kLog2e);
        }
      }
      const float ks = __shfl_sync(0xffffffffu, my_ks, j), vs = __shfl_sync(0xffffffffu, my_vs, j);
      const int keys = __shfl_sync(0xffffffffu, my_keys, j), blk = __shfl_sync(0xffffffffu, my_blk, j);

      if (!wait()) break;
      const uint8_t* k_buf = ring + buf * kKv8Bytes;
      float s[kTiles][4][4];
#pragma unroll
      for (int st = 0; st < 4; ++st) {
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) s[nt][st][0] = s[nt][st][1] = s[nt][st][2] = s[nt][st][3] = 0.f;
        // row r of the tile is key 16 (r >> 1) + 4 st + (r & 1), row r + 8 two keys on: the order P^T is read in below
        const uint8_t* k0 = k_buf + (16 * (row >> 1) + 4 * st + (row & 1)) * 64 + 16 * t;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 a = *reinterpret_cast<const uint4*>(k0 + h * (kKv8Bytes / 2));
          const uint4 b = *reinterpret_cast<const uint4*>(k0 + h * (kKv8Bytes / 2) + 128);
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            uint32_t a0, a1, a2, a3;
            kv8_to_half<kKind>(word_of(a, w), a0, a2);
            kv8_to_half<kKind>(word_of(b, w), a1, a3);
#pragma unroll
            for (int nt = 0; nt < kTiles; ++nt) {
              const uint2 q = kFew ? sq[(nt * 8 + 4 * h + w) * 32] : make_uint2(qb[4 * h + w][0], qb[4 * h + w][1]);
              mma_f16_16816(s[nt][st], a0, a1, a2, a3, q.x, q.y);
            }
          }
        }
      }
      release();

      uint32_t pb[kTiles][4][2];
#pragma unroll
      for (int nt = 0; nt < kTiles; ++nt) {
        float (&z)[4][4] = s[nt];
        // z = log2 of the weight against the fixed reference 30: -2 kT / (1 + e^(2 x / 30))
        // (a product beyond fp32 counts as its largest number: a score of zero stays zero, others are at the cap all the
        // same; a NaN scale stays NaN)
        float f0 = ks * q_scale[nt][0], f1 = ks * q_scale[nt][1];
        f0 = f0 > FLT_MAX ? FLT_MAX : f0, f1 = f1 > FLT_MAX ? FLT_MAX : f1;
        // keys seen: a group's earlier tokens see fewer than its last
        const int keys0 = kFew ? keys - max(0, seen - 1 - (8 * nt + 2 * t) / kGroup) : keys;
        const int keys1 = kFew ? keys - max(0, seen - 1 - (8 * nt + 2 * t + 1) / kGroup) : keys;
        float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
        for (int st = 0; st < 4; ++st)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = (-2.f * kT) * rcp_approx(1.f + ex2_approx(z[st][e] * (e & 1 ? f1 : f0)));
            if (keys < kKv8Block + (kFew ? kDqTok - 1 : 0) &&
                16 * (row >> 1) + 4 * st + (row & 1) + (e & 2) >= (e & 1 ? keys1 : keys0))
              x = -INFINITY;
            z[st][e] = x;
            if (e & 1) top1 = fmaxf(top1, x); else top0 = fmaxf(top0, x);
          }
#pragma unroll
        for (int d = 4; d < 32; d *= 2) {
          top0 = fmaxf(top0, __shfl_xor_sync(0xffffffffu, top0, d));
          top1 = fmaxf(top1, __shfl_xor_sync(0xffffffffu, top1, d));
        }
        float &m0 = m[nt][0], &m1 = m[nt][1];
        if (__any_sync(0xffffffffu, top0 > m0 + kDqLag || top1 > m1 + kDqLag)) {
          const float n0 = fmaxf(m0, top0 - kDqTop), n1 = fmaxf(m1, top1 - kDqTop);
          const float c0 = ex2_approx(m0 - n0), c1 = ex2_approx(m1 - n1);
          m0 = n0, m1 = n1;
          l[nt][0] *= c0, l[nt][1] *= c1;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt)
            o[nt][mt][0] *= c0, o[nt][mt][1] *= c1, o[nt][mt][2] *= c0, o[nt][mt][3] *= c1;
        }
        float b0 = 0.f, b1 = 0.f;
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          const float p0 = ex2_approx(z[st][0] - m0), p1 = ex2_approx(z[st][1] - m1);
          const float p2 = ex2_approx(z[st][2] - m0), p3 = ex2_approx(z[st][3] - m1);
          b0 += p0 + p2, b1 += p1 + p3;
          pb[nt][st][0] = movmatrix_trans(pack_f16x2(p0, p1));
          pb[nt][st][1] = movmatrix_trans(pack_f16x2(p2, p3));
        }
        l[nt][0] += b0, l[nt][1] += b1;
        if (kWeights) {
#pragma unroll
          for (int d = 4; d < 32; d *= 2) {
            b0 += __shfl_xor_sync(0xffffffffu, b0, d);
            b1 += __shfl_xor_sync(0xffffffffu, b1, d);
          }
          if (row == 0 && t < kGroup / 2)
            *reinterpret_cast<float2*>(p.block_w + ((size_t)pair * p.c.max_blocks + blk) * 8 + 2 * t) =
                make_float2(b0 * ex2_approx(m0), b1 * ex2_approx(m1));
        }
      }

      if (!wait()) break;
      const uint8_t* v_buf = ring + buf * kKv8Bytes;
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        uint4 a = *reinterpret_cast<const uint4*>(v_buf + (16 * mt + row) * 64 + 16 * t);
        uint4 b = *reinterpret_cast<const uint4*>(v_buf + (16 * mt + row + 8) * 64 + 16 * t);
        if (kKind == GROK_KV8_E4M3 && keys < kKv8Block) {  // codes behind the last row may be NaN
#pragma unroll
          for (int st = 0; st < 4; ++st) {
            const int left = keys - (16 * t + 4 * st);
            const uint32_t mask = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
            reinterpret_cast<uint32_t*>(&a)[st] &= mask;
            reinterpret_cast<uint32_t*>(&b)[st] &= mask;
          }
        }
        float acc[kTiles][4];
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
        for (int st = 0; st < 4; ++st) {
          uint32_t a0, a1, a2, a3;
          kv8_to_half<kKind>(word_of(a, st), a0, a2);
          kv8_to_half<kKind>(word_of(b, st), a1, a3);
#pragma unroll
          for (int nt = 0; nt < kTiles; ++nt) mma_f16_16816(acc[nt], a0, a1, a2, a3, pb[nt][st][0], pb[nt][st][1]);
        }
#pragma unroll
        for (int nt = 0; nt < kTiles; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[nt][mt][e] = fmaf(acc[nt][e], vs, o[nt][mt][e]);
      }
      release();
    }
  }
  if (ok) {
    flush();
    return;
  }
  // A wait gave up: copies in flight land before the shared memory is released.
  volatile int never = 0;
  for (; due > 0; --due) {
    mbar_wait(&bars[buf], phase, &never, p.status);
    if (++buf == kDqBufs) {
      buf = 0;
      phase ^= 1;
    }
  }
}

// Joins a pair's partials. A CTA takes kHeads of the pair's six query heads,
// kSplit warps to a head; the blocks' weights are done by the pair's CTA (kHeads 6)
// or by one CTA more (kHeads 1).
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d; d /= 2) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d /= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}

template <int kHeads, int kSplit, bool kFew>
__global__ void __launch_bounds__(kHeads * kSplit * 32) kv8_join_kernel(const DqParams p) {
  constexpr int kThreads = kHeads * kSplit * 32;
  constexpr int kBatch = 12;  // partial outputs in flight per warp
  __shared__ float4 s_o[kHeads * kSplit][32];
  __shared__ float s_inv[8];
  constexpr int kCols = kFew ? kDqFewCols : kGroup;
  const int pair = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // The column of head 0: kFew has its tokens' heads along y.
  const int col0 = kFew ? blockIdx.y / (kGroup / kHeads) * kGroup : 0;
  const int head0 = (kFew ? blockIdx.y % (kGroup / kHeads) : kHeads == 1 ? blockIdx.y : 0) * kHeads;
  const int blocks = blocks_of<kFew>(p, pair / kKVHeads);
  const bool weights = p.weight_out && (kHeads > 1 || blockIdx.y == kGroup);
  int few_b = 0, few_tok = 0;
  if (kFew) {
    const int groups = groups_of(p.few_tokens), v = pair / kKVHeads;
    few_b = v / groups, few_tok = v % groups * kDqTok + col0 / kGroup;
  }
  // The first blocks' old weights do not depend on the first kernel.
  const size_t at0 = (size_t)pair * p.c.max_blocks + threadIdx.x;
  float w_in = 0.f;
  if (weights && p.weight_in && threadIdx.x < p.c.max_blocks) w_in = p.weight_in[at0];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (blocks == 0) return;                // reported by the first kernel
  if (kFew && few_tok >= p.few_tokens) return;
  const int2 parts = p.pair_parts[pair];  // first slot, number
  const int n_parts = parts.y;
  const float2* ml = p.part_ml + (size_t)parts.x * kCols + col0;
  float4 wa = make_float4(0.f, 0.f, 0.f, 0.f);
  float2 wb = make_float2(0.f, 0.f);
  if (weights && threadIdx.x < blocks) {
    wa = *reinterpret_cast<const float4*>(p.block_w + at0 * 8);
    wb = *reinterpret_cast<const float2*>(p.block_w + at0 * 8 + 4);
  }

  if (kFew || kHeads > 1 || blockIdx.y < kGroup) {
    // Everything is loaded before anything is used: the partials' sums, a lane to each, and this warp's first outputs.
    const int head = head0 + warp / kSplit, sub = warp % kSplit;
    const float* po = p.part_o + ((size_t)parts.x * kCols + col0 + head) * kD + 4 * lane;
    const float2 mine = lane < n_parts ? ml[lane * kCols + head] : make_float2(-INFINITY, 0.f);
    float4 v[kBatch];
    float vm[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int k = sub + u * kSplit;
      v[u] = make_float4(0.f, 0.f, 0.f, 0.f);
      vm[u] = -INFINITY;
      if (k < n_parts) {
        v[u] = *reinterpret_cast<const float4*>(po + (size_t)k * (kCols * kD));
        vm[u] = ml[k * kCols + head].x;
      }
    }
    float m = mine.x;
    for (int k = lane + 32; k < n_parts; k += 32) m = fmaxf(m, ml[k * kCols + head].x);
    m = warp_max(m);
    float l = mine.y * ex2_approx(mine.x - m);
    for (int k = lane + 32; k < n_parts; k += 32) {
      const float2 x = ml[k * kCols + head];
      l = fmaf(x.y, ex2_approx(x.x - m), l);
    }
    l = warp_sum(l);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const float f = ex2_approx(vm[u] - m);
      acc.x = fmaf(v[u].x, f, acc.x);
      acc.y = fmaf(v[u].y, f, acc.y);
      acc.z = fmaf(v[u].z, f, acc.z);
      acc.w = fmaf(v[u].w, f, acc.w);
    }
#pragma unroll 8
    for (int k = sub + kBatch * kSplit; k < n_parts; k += kSplit) {
      const float4 x = *reinterpret_cast<const float4*>(po + (size_t)k * (kCols * kD));
      const float f = ex2_approx(ml[k * kCols + head].x - m);
      acc.x = fmaf(x.x, f, acc.x);
      acc.y = fmaf(x.y, f, acc.y);
      acc.z = fmaf(x.z, f, acc.z);
      acc.w = fmaf(x.w, f, acc.w);
    }
    if (kSplit > 1) {
      s_o[warp][lane] = acc;
      __syncthreads();
      if (sub == 0) {
#pragma unroll
        for (int w = 1; w < kSplit; ++w) {
          const float4 x = s_o[warp + w][lane];
          acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
        }
      }
    }
    if (sub == 0) {
      const float inv = 1.f / l;
      size_t at = (size_t)pair * kGroup + head;
      if (kFew)
        at = (((size_t)few_b * p.few_tokens + few_tok) * kKVHeads + pair % kKVHeads) * kGroup + head;
      p.out[at * (kD / 4) + lane] =
          make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
      if (kHeads > 1 && lane == 0) s_inv[head] = 1.f / (l * ex2_approx(m));  // on the fixed reference 30
    }
  } else {
    for (int h = warp; h < kGroup; h += kSplit) {
      float l = 0.f;
      for (int k = lane; k < n_parts; k += 32) l = fmaf(ml[k * kGroup + h].y, ex2_approx(ml[k * kGroup + h].x), l);
      l = warp_sum(l);
      if (lane == 0) s_inv[h] = 1.f / l;
    }
  }
  if (!weights) return;
  __syncthreads();
  for (int i = threadIdx.x; i < p.c.max_blocks; i += kThreads) {
    const size_t at = (size_t)pair * p.c.max_blocks + i;
    if (i >= kThreads) {
      w_in = p.weight_in ? p.weight_in[at] : 0.f;
      if (i < blocks) {
        wa = *reinterpret_cast<const float4*>(p.block_w + at * 8);
        wb = *reinterpret_cast<const float2*>(p.block_w + at * 8 + 4);
      }
    }
    float w = 0.f;
    if (i < blocks)
      w = wa.x * s_inv[0] + wa.y * s_inv[1] + wa.z * s_inv[2] + wa.w * s_inv[3] + wb.x * s_inv[4] + wb.y * s_inv[5];
    p.weight_out[at] = w_in + w;
  }
}

}  // namespace grok

using namespace grok;

namespace {

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }
int wave_of(int sms, int warps = kDqWarps) { return sms * kDqCtas * warps; }  // workers resident at a time
// A share touches a run of pairs, so (share, pair) runs through fewer than shares + pairs values of their sum.
size_t part_slots(int B, int sms) { return size_t(2) * wave_of(sms) + size_t(B) * kKVHeads; }
size_t part_o_bytes(int B, int sms, int cols) { return part_slots(B, sms) * cols * kD * sizeof(float); }
size_t part_ml_bytes(int B, int sms, int cols) { return up256(part_slots(B, sms) * cols * sizeof(float2)); }
size_t pairs_bytes(int B) { return up256(size_t(B) * kKVHeads * sizeof(int2)); }
size_t block_w_bytes(int B, int max_blocks) { return size_t(B) * kKVHeads * max_blocks * 8 * sizeof(float); }

}  // namespace

size_t grok::kv8_decode_bytes(int B, int few_tokens, int max_blocks, bool weights, int sms) {
  const int n_seq = few_tokens ? B * groups_of(few_tokens) : B, cols = few_tokens ? kDqFewCols : kGroup;
  return part_o_bytes(n_seq, sms, cols) + part_ml_bytes(n_seq, sms, cols) + pairs_bytes(n_seq) +
         (weights ? block_w_bytes(n_seq, max_blocks) : 0);
}

grok_status grok::kv8_decode_run(const grok_kv8_cache& cache, const grok_bf16* q_rot, const int32_t* len,
                                 const int32_t* valid_len, int few_tokens, char* ws, grok_bf16* out,
                                 const float* weight_in, float* weight_out, int sms, int32_t* dev_status,
                                 cudaStream_t stream) {
  int dev = 0;
  grok_status st = device_index(&dev);
  if (st != GROK_OK) return st;
  const int n_seq = few_tokens ? cache.B * groups_of(few_tokens) : cache.B, cols = few_tokens ? kDqFewCols : kGroup;
  const size_t o_bytes = part_o_bytes(n_seq, sms, cols), ml_bytes = part_ml_bytes(n_seq, sms, cols);
  const int warps = few_tokens ? kDqFewWarps : kDqWarps, wave = wave_of(sms, warps);
  const int second = (long long)n_seq * kKVHeads * cache.max_blocks >= (long long)kDqLong * wave ? wave : 0;
  const DqParams p{cache,
                   reinterpret_cast<const uint4*>(q_rot),
                   len,
                   valid_len,
                   few_tokens,
                   n_seq,
                   reinterpret_cast<float*>(ws),
                   reinterpret_cast<float2*>(ws + o_bytes),
                   reinterpret_cast<int2*>(ws + o_bytes + ml_bytes),
                   weight_out ? reinterpret_cast<float*>(ws + o_bytes + ml_bytes + pairs_bytes(n_seq)) : nullptr,
                   reinterpret_cast<uint2*>(out),
                   weight_in,
                   weight_out,
                   wave,
                   second,
                   dev_status};
  const bool i8 = cache.kind == GROK_KV8_INT8;
  const int which = few_tokens ? 2 : weight_out ? 1 : 0;
  decltype(&kv8_decode_kernel<GROK_KV8_INT8, false, false>) kernels[2][3] = {
      {kv8_decode_kernel<GROK_KV8_INT8, false, false>, kv8_decode_kernel<GROK_KV8_INT8, true, false>,
       kv8_decode_kernel<GROK_KV8_INT8, false, true>},
      {kv8_decode_kernel<GROK_KV8_E4M3, false, false>, kv8_decode_kernel<GROK_KV8_E4M3, true, false>,
       kv8_decode_kernel<GROK_KV8_E4M3, false, true>}};
  auto kernel = kernels[i8 ? 0 : 1][which];
  // Per device and kernel; idempotent: every thread would set the same value.
  static bool attr_set[kMaxDevices][2][3] = {};
  const int smem = few_tokens ? kDqFewSmem : kDqSmem;
  bool& set = attr_set[dev][i8 ? 0 : 1][which];
  if (!set) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return fail(cuda_status(e), "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    set = true;
  }
  // Both kernels are launched as dependents of the one before them: each begins with a wait for all of it.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((p.wave + p.second) / warps);
  cfg.blockDim = dim3(32 * warps);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e != cudaSuccess) return fail(cuda_status(e), "kv8_decode launch: %s", cudaGetErrorString(e));
  if ((st = check_launch("kv8_decode")) != GROK_OK) return st;
  // Many pairs have few partials each: a CTA per pair, a warp per head. Few pairs have many (workers / pairs and
  // two more at most): a CTA per pair and head, where all of them run at once (two on an SM). Whole calls, us, CTA per
  // pair and head against CTA per pair: 2 sequences of 5120 rows 9.8 against 15.0, 4 14.9 against 18.0, 8 22.4 against
  // 21.9; of 300 rows 1 6.9 against 6.9, 8 9.0 against 7.6, 16 11.0 against 8.3.
  // (With or without weights the same join adds the outputs, in the same order.)
  const int pairs = n_seq * kKVHeads;
  const int toks = few_tokens ? kDqTok : 1;  // (a group's tokens are joined apart)
  const bool few = pairs * toks * (kGroup + 1) <= 2 * sms;
  auto join = few ? kv8_join_kernel<1, 8, false> : kv8_join_kernel<kGroup, 1, false>;
  int split = few ? kGroup : 1, threads = few ? 256 : kGroup * 32;  // CTAs per pair and token
  if (few_tokens) {
    join = few ? kv8_join_kernel<1, 8, true> : kv8_join_kernel<kGroup, 1, true>;
    // Between the two, two warps per head, three CTAs on an SM: 1 sequence behind 16000 rows, 8 / 12 tokens 28.1 / 34.7
    // against 29.6 / 36.1 with a warp per head; 4 behind 3000, 2 tokens 16.5 against 18.1, 16 tokens 35.1 against 33.3.
    if (!few && pairs * toks * 2 <= 3 * sms) join = kv8_join_kernel<3, 2, true>, split = 2;
  }
  cfg.gridDim = dim3(pairs, toks * split + (weight_out && few ? 1 : 0));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = 0;
  e = cudaLaunchKernelEx(&cfg, join, p);
  if (e != cudaSuccess) return fail(cuda_status(e), "kv8_join launch: %s", cudaGetErrorString(e));
  return check_launch("kv8_join");
}

extern "C" grok_status grok_kv8_decode_workspace(int B, int max_blocks, int weights, size_t* bytes) {
  if (!bytes) return fail(GROK_ERR_INVALID_ARG, "grok_kv8_decode_workspace: null pointer");
  if (B < 1 || B > 65535 || max_blocks < 1 || max_blocks > kKv8MaxBlocks)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_decode_workspace: need 1 <= B <= 65535, 1 <= max_blocks <= %d",
                kKv8MaxBlocks);
  int sms = 0;
  grok_status st = device_sm_count(&sms);
  if (st != GROK_OK) return st;
  *bytes = kv8_decode_bytes(B, 0, max_blocks, weights != 0, sms);
  return GROK_OK;
}

extern "C" grok_status grok_kv8_decode(const grok_kv8_cache* cache, const grok_bf16* q_rot, const int32_t* kv_len,
                                       void* workspace, size_t workspace_bytes, grok_bf16* out,
                                       const float* weight_in, float* weight_out, int32_t* dev_status, void* stream) {
  grok_status st = kv8_check(cache, "grok_kv8_decode");
  if (st != GROK_OK) return st;
  if (!q_rot || !kv_len || !workspace || !out) return fail(GROK_ERR_INVALID_ARG, "grok_kv8_decode: null pointer");
  if (weight_in && !weight_out) return fail(GROK_ERR_INVALID_ARG, "grok_kv8_decode: weight_in without weight_out");
  if (!aligned16(q_rot) || !aligned16(out))
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_decode: bf16 tensors must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_decode: workspace must be 256-byte aligned");
  int sms = 0;
  if ((st = device_sm_count(&sms)) != GROK_OK) return st;
  const size_t need = kv8_decode_bytes(cache->B, 0, cache->max_blocks, weight_out != nullptr, sms);
  if (workspace_bytes < need)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_decode: workspace of %zu bytes is smaller than the %zu needed",
                workspace_bytes, need);
  return kv8_decode_run(*cache, q_rot, kv_len, nullptr, 0, static_cast<char*>(workspace), out, weight_in, weight_out, sms,
                        dev_status, static_cast<cudaStream_t>(stream));
}
