// Decode over blocks of a paged cache: a list of blocks per KV head, or a sequence's
// rows behind a prefix that it shares.
//
// Code-reading guide ch. 4 §4.4.1, §4.5.2-§4.5.4: out = sum_j w_j v_j / sum_j w_j,
// w_j = exp(30 tanh(q . k_j / (30 sqrt(128))) - 30). Every capped logit is below 30,
// so weights need no running maximum and partial sums simply add.
//
// Memory-bound: 32 KB of keys and values per block of 64 tokens and KV head are read
// once. The blocks of all (sequence, KV head) pairs, in order, are dealt out to the
// CTAs in equal contiguous shares whatever the lengths. A producer warp finds the
// blocks (32 at a time, one a lane) and streams them through a ring of 16 KB tiles, K
// and V in turn, by TMA, with the pair's six queries beside its first block; four warps
// take 16 keys of each block. On mma.sync (bf16 operands, fp32 accumulators):
//   S^T [16 keys x 8 heads] = K q^T, O^T [128 x 8] += V^T P^T
// (6 of 8 columns used; rows of heads would use 6 of 16). P is split into two bf16
// halves, so a weight is off by 2^-16. S^T leaves the accumulators as P^T needs it but
// for an 8 x 8 transpose per register. Where a CTA's share of a pair ends, its warps add
// their sums through shared memory (handed over by barriers whose waits are bounded, as
// all are) and write one part; a second kernel, launched as a dependent, adds a pair's
// parts in their order.
//
// Measured (graph replays): 8 sequences x 128 blocks per head (268 MB) in equal shares
// 50.4 us, 5.3 TB/s, 0.79 of the copy rate: 2 us launch, 4 us to the first keys (lengths, list,
// table, keys: four round trips), 40 us at 6.6 TB/s, 3 us the join. A second wave of small shares,
// which evens out the SMs in the 8-bit decode, starts too late to pay here (54 us). Short lists of
// few pairs go to clusters of CTAs, one to a pair (kPairs), which need neither plan nor join:
// one sequence, 16 blocks, 6.8 us, 9.2 with a plan and a join.
#include <algorithm>

#include "block_decode.cuh"

namespace grok {

constexpr int kBkThreads = (kBkWarps + 1) * 32;
constexpr int kBkBox = kBlk * 128;           // [64 rows][64 bf16]
constexpr int kBkTile = 2 * kBkBox;          // the K or the V of a block
// Tiles of the ring, K and V of the blocks in turn. Over lists two CTAs share an SM; over the rows behind prefixes one runs
// beside a CTA of the prefix kernel.
__host__ __device__ constexpr int bk_ring(bool list) { return list ? 5 : 4; }
constexpr int kBkQ = kGroup * kD * 2;        // a pair's queries
constexpr int kBkPlan = 512;                 // entries of the table of block counts
constexpr int kBkCtas = 2;                   // CTAs resident on an SM
constexpr int kBkPairMost = 8;               // blocks of a list that a CTA of its pair's cluster may get
// Beside the prefix kernel: blocks per CTA up to which half of the CTAs take them all; key tiles of the prefix in whose time a CTA
// gets through a block; blocks in the time that a CTA behind the prefix takes to start.
constexpr int kBkFew = 8, kBkBeside = 10, kBkStart = 6;

template <int kRing>
struct BkShared {
  float4 sum_o[kBkWarps][6 * 32];  // the warps' sums but those of the quarter of the features that each adds itself
  float2 sum_l[kBkWarps][4];
  uint64_t full[kRing], empty[kRing], sum_full, sum_empty;
  int2 token[kRing];      // pair and visible keys of the block whose K is in a place of the ring; pair -1: the end
  int cum[kBkPlan + 1];   // blocks per KV head of the sequences before each entry's
  int seq[kBkPlan];       // length | pages left out << 17, where an entry is a sequence
  GroupTable groups;
  int warp_sum[kBkWarps + 1];
  int3 deal;              // CTAs of the first kind, blocks to each, blocks to each of the others
  int abort;
};
template <bool kList>
constexpr int kBkSmem = 1024 + bk_ring(kList) * (kBkTile + kBkQ) + int(sizeof(BkShared<bk_ring(kList)>));
static_assert(kBkCtas * (kBkSmem<true> + 1024) <= 233472, "shared memory per SM");
static_assert(kBkSmem<false> + 1024 + kPxSmemMax + 1024 <= 233472, "shared memory beside the prefix kernel");

struct BkParams {
  const uint8_t* q;
  PageMap pm;
  const int32_t* kv_len;
  int B;
  const int32_t* sel;
  int budget;
  Groups groups;
  BlockParts parts;
  grok_bf16* out;     // kPairs
  int4* prefix_pair;  // entries of sequences without a prefix are cleared here
  int32_t* status;
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Blocks that a sequence of `len` rows reads per KV head, `share` of its pages left out; -1 when its length is bad.
__device__ __forceinline__ int bk_blocks(const BkParams& p, int len, int share) {
  if (len < 1 || len > p.pm.max_pages * GROK_PAGE_TOKENS || len < share * GROK_PAGE_TOKENS) return -1;
  return min((len + kBlk - 1) / kBlk - share * kBlkPerPage, p.budget);
}

// How `total` blocks behind prefixes are dealt to the CTAs: (CTAs of the first kind, blocks to each, blocks to each of the others).
// Beside the prefix kernel an SM has room for one CTA, which is slowed by it (its few warps wait for issue slots beside sixteen);
// the second half of the CTAs starts behind the prefix. Little work is dealt to the first half (32 sequences behind 8192 rows, 5
// blocks to a CTA: 30.6 us, 39 over all of them), of more work as much as lets both halves end together: 256 behind 16384 rows,
// 20 blocks to a CTA of the first half and none to the others, 130 us (145 in equal shares); 128 behind 4096, 31 and 23, 75.3
// (78.6). (kBkBeside and kBkStart were measured on those two, whose query tiles are full.) Where no group shares a page the
// prefix kernel has nothing to do, and all CTAs take equal shares (64 sequences of up to 300 rows: 19.9 us, 24.2 over half of
// them). A function that is not inlined: with the same lines in the kernel the code of its loop comes out slower (140 and 77).
__device__ __noinline__ int3 bk_deal(int total, int ctas, const GroupTable* groups, int n_groups) {
  int early = ctas, late = 0, tiles = 0;  // (key tiles of the prefix kernel)
  for (int i = threadIdx.x % 32; i < n_groups; i += 32)
    tiles += (groups->start[i + 1] - groups->start[i] + kPxSeqs - 1) / kPxSeqs * groups->pages[i] * (kBlkPerPage * kKVHeads);
  tiles = __reduce_add_sync(0xffffffffu, tiles);
  if (tiles) {
    early /= kBkCtas;
    if (total > kBkFew * ctas) {
      const int both = (total + early - 1) / early;  // blocks of a CTA of each half
      late = max(0, both - tiles / early / kBkBeside - kBkStart) / 2;
    }
  }
  return make_int3(early, max(1, (total - early * late + early - 1) / early), late);
}

// kOwn: the rows behind prefixes. (Registers: 112 a thread at most, for the same reason as in the prefix kernel.)
// kLists: lists of blocks, dealt out to the CTAs in equal shares. kPairs: the same for short lists of few pairs: a cluster of CTAs takes a
// pair's list and joins its parts itself, so that there is neither a plan nor a second kernel.
enum BkMode { kOwn, kLists, kPairs };
template <int kMode>
__global__ void __launch_bounds__(kMode != kOwn ? kBkThreads : 576, kMode != kOwn ? kBkCtas : 1)
    block_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_k16, const __grid_constant__ CUtensorMap tm_v16,
                        const BkParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  constexpr bool kList = kMode != kOwn, kPair = kMode == kPairs;
  constexpr int kBkRing = bk_ring(kList);
  uint8_t* sq = smem + kBkRing * kBkTile;
  BkShared<kBkRing>* sh = reinterpret_cast<BkShared<kBkRing>*>(sq + kBkRing * kBkQ);
  volatile int* abort = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // The kernel that joins the partial results may be scheduled as soon as every CTA has started.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    for (int s = 0; s < kBkRing; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], kBkWarps);
    }
    mbar_init(&sh->sum_full, kBkWarps);
    mbar_init(&sh->sum_empty, kBkWarps);
    sh->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // The lists and the tables come closer while the plan is made, a line a thread of the grid.
  {
    const size_t line = (size_t)blockIdx.x * kBkThreads + tid, lines = (size_t)p.B * p.pm.max_pages / 32;
    if (line < lines) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.pm.table + line * 32));
    if (kList && line < (size_t)p.B * kKVHeads * p.budget / 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.sel + line * 32));
  }
  const int cta = blockIdx.x;
  int lo, hi, share_of = 1;                    // this CTA's blocks; blocks per CTA
  int pair0 = 0, len0 = 0, n0 = 0, rank = 0, ctas = 1;  // kPairs: the pair, its sequence's rows, its blocks, the CTA's place
  int step = 1, entries = 0, n_groups = 0;
  if (kPair) {
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
    pair0 = cta / ctas;
    rank = cta % ctas;
    len0 = p.kv_len[pair0 / kKVHeads];
    n0 = bk_blocks(p, len0, 0);
    if (n0 < 0) {
      if (rank == 0 && pair0 % kKVHeads == 0 && tid == 0) report(p.status, GROK_DEV_BAD_KV_LEN);
      return;  // (the whole cluster)
    }
    share_of = (n0 + ctas - 1) / ctas;
    lo = min(rank * share_of, n0);
    hi = min(lo + share_of, n0);
    __syncthreads();
  } else {
    // The plan: blocks per KV head before each sequence (or each `step` sequences, where there are many).
    step = (p.B + kBkPlan - 1) / kBkPlan;
    entries = (p.B + step - 1) / step;
    constexpr int kPer = (kBkPlan + kBkThreads - 1) / kBkThreads;  // contiguous entries per thread
    const int per = (entries + kBkThreads - 1) / kBkThreads, e0 = tid * per;
    int lens[kPer];  // (loaded beside the groups)
#pragma unroll
    for (int i = 0; i < kPer; ++i) lens[i] = i < per && e0 + i < entries ? p.kv_len[(e0 + i) * step] : 0;
    if (!kList) {
      bool fine = true;
      for (int i = tid; i < p.groups.n; i += kBkThreads) fine &= load_groups(p.groups, p.B, p.pm.max_pages, &sh->groups, i);
      if (__syncthreads_and(fine))
        n_groups = p.groups.n;
      else if (blockIdx.x == 0 && tid == 0)
        report(p.status, GROK_DEV_BAD_GROUP);
    }
    {
      int n_of[kPer], mine = 0;
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        n_of[i] = 0;
        const int e = e0 + i;
        if (i < per && e < entries)
          for (int b = e * step; b < min((e + 1) * step, p.B); ++b) {
            const int len = b == e * step ? lens[i] : p.kv_len[b], share = n_groups ? sh->groups.of_seq(n_groups, b) : 0;
            const int n = bk_blocks(p, len, share);
            if (step == 1) sh->seq[e] = len | share << 17;
            if (blockIdx.x == 0) {
              if (n < 0) report(p.status, GROK_DEV_BAD_KV_LEN);
              if (n <= 0)
                for (int g = 0; g < kKVHeads; ++g) p.parts.pair[b * kKVHeads + g] = make_int2(0, n);
              if (!kList && share == 0)
                for (int g = 0; g < kKVHeads; ++g) p.prefix_pair[b * kKVHeads + g] = make_int4(0, 0, 0, 0);
            }
            n_of[i] += max(n, 0);
          }
        mine += n_of[i];
      }
      int incl = mine;
#pragma unroll
      for (int d = 1; d < 32; d *= 2) {
        const int up = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += up;
      }
      if (lane == 31) sh->warp_sum[warp] = incl;
      __syncthreads();
      int at = incl - mine;
      for (int w = 0; w < warp; ++w) at += sh->warp_sum[w];
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        if (i < per && e0 + i < entries) {
          sh->cum[e0 + i] = at;
          at += n_of[i];
          if (e0 + i == entries - 1) sh->cum[entries] = at;
        }
    }
    __syncthreads();
    const int total = kKVHeads * sh->cum[entries];
    if (kList) {
      share_of = max(1, (total + int(gridDim.x) - 1) / int(gridDim.x));
      lo = int(min((long long)cta * share_of, (long long)total));
      hi = min(lo + share_of, total);
    } else {
      const int3 d = bk_deal(total, int(gridDim.x), &sh->groups, n_groups);
      if (tid == kBkWarps * 32) sh->deal = d;
      lo = min(cta < d.x ? cta * d.y : d.x * d.y + (cta - d.x) * d.z, total);
      hi = min(lo + (cta < d.x ? d.y : d.z), total);
    }
  }
  if (lo < hi) {
    if (warp == kBkWarps) {
      // ------------------------------------------------------------ producer
      __syncwarp();
      int st = 0, turn = 1, loads = 0;  // the ring's next place, the parity that frees it, places taken so far
      int cur = -1;        // the pair of the last block looked at
      bool sent = true;    // a token of that pair is out
      bool ok = true;
      auto acquire = [&]() {  // (false when a bounded wait gave up)
        ok = ok && __all_sync(0xffffffffu, mbar_wait(&sh->empty[st], turn, abort, p.status));
        return ok;
      };
      auto next = [&]() {
        ++loads;
        if (++st == kBkRing) st = 0, turn ^= 1;
      };
      // A block's K or V into the ring, with `more` bytes that come beside it: in one copy, or of a sequence's last block
      // the rows that there are, 16 at a time (two copies of half of the features each, one a lane).
      auto load = [&](const CUtensorMap* tm, const CUtensorMap* tm16, int row, int g, int keys, int more) {
        const int groups = (keys + 15) / 16;
        if (lane == 0) mbar_arrive_expect_tx(&sh->full[st], groups * 16 * kD * 2 + more);
        uint8_t* to = smem + st * kBkTile;
        if (groups == 4) {
          if (lane == 0) tma_load_4d(to, tm, &sh->full[st], 0, row, 0, g);
        } else if (lane < 2 * groups) {
          tma_load_4d(to + (lane & 1) * kBkBox + (lane >> 1) * 16 * 128, tm16, &sh->full[st], 0, row + (lane >> 1) * 16,
                      lane & 1, g);
        }
        next();
      };
      auto send_empty = [&](int pair) {  // a token without a block
        if (!acquire()) return;
        if (lane == 0) {
          sh->token[st] = make_int2(pair, 0);
          mbar_arrive(&sh->full[st]);
        }
        next();
      };
      // (The lookups go on after a wait that gave up: every pair's entry is written, and the join reads in bounds.)
      for (int base = lo; base < hi; base += 32) {
        const int cnt = min(32, hi - base), idx = base + lane;
        int my_pair = 0, my_row = -1, my_keys = 0;  // (row of the pools; -1: no block here)
        if (lane < cnt) {
          int b = pair0 / kKVHeads, len = len0, share = 0, k = idx;
          my_pair = pair0;
          if (!kPair) {
            int e = 0, n;
            for (int d = kBkPlan / 2; d; d /= 2)
              if (e + d < entries && kKVHeads * sh->cum[e + d] <= idx) e += d;
            int rest = idx - kKVHeads * sh->cum[e];
            b = e * step;
            while (true) {
              len = step == 1 ? sh->seq[e] & 0x1FFFF : p.kv_len[b];
              share = step == 1 ? sh->seq[e] >> 17 : n_groups ? sh->groups.of_seq(n_groups, b) : 0;
              n = max(bk_blocks(p, len, share), 0);
              if (step == 1 || rest < kKVHeads * n) break;
              rest -= kKVHeads * n;
              ++b;
            }
            my_pair = b * kKVHeads + rest / n;
            k = rest % n;
            if (k == 0) {  // the pair's parts: one of each CTA from this one on that takes some of its blocks
              int last = 0, end = idx + n - 1, each = share_of;
              if (!kList && end >= sh->deal.x * sh->deal.y) {
                last = sh->deal.x;
                end -= last * sh->deal.y;
                each = sh->deal.z;
              } else if (!kList) {
                each = sh->deal.y;
              }
              last += end / each;
              p.parts.pair[my_pair] = make_int2(cta + my_pair, last - cta + 1);
            }
          }
          const int blocks = (len + kBlk - 1) / kBlk;
          int blk = share * kBlkPerPage + k;
          if (kList) blk = p.sel[(size_t)my_pair * p.budget + k];
          if (blk >= blocks) {
            report(p.status, GROK_DEV_BAD_BLOCK);
          } else if (blk >= 0) {
            my_row = max(0, blk_page(p.pm, b, blk, p.status)) * GROK_PAGE_TOKENS + blk % kBlkPerPage * kBlk;
            my_keys = min(kBlk, len - blk * kBlk);
          }
        }
        for (int j = 0; j < cnt && ok; ++j) {
          const int pair = __shfl_sync(0xffffffffu, my_pair, j), row = __shfl_sync(0xffffffffu, my_row, j);
          const int keys = __shfl_sync(0xffffffffu, my_keys, j);
          if (pair != cur) {
            if (!sent) send_empty(cur);  // nothing of the last pair's list here: its part is zero
            cur = pair;
            sent = false;
          }
          if (row < 0 || !acquire()) continue;
          const int g = pair % kKVHeads;
          if (lane == 0) {
            sh->token[st] = make_int2(pair, keys);
            if (!sent) bulk_load(sq + st * kBkQ, p.q + (size_t)pair * kBkQ, kBkQ, &sh->full[st]);
          }
          load(&tm_k, &tm_k16, row, g, keys, sent ? 0 : kBkQ);
          sent = true;
          if (!acquire()) continue;
          load(&tm_v, &tm_v16, row, g, keys, 0);
        }
      }
      if (ok && !sent) send_empty(cur);
      if (ok) send_empty(-1);
      // Copies in flight (only after an abort) land before the CTA exits.
      volatile int never = 0;
      if (lane == 0)
        for (int t = max(0, loads - kBkRing); t < loads; ++t)
          mbar_wait(&sh->full[t % kBkRing], (t / kBkRing) & 1, &never, p.status);
    } else {
      // ------------------------------------------------------------ 16 keys of each block
      const int row = lane >> 2, t = lane & 3, mi = lane >> 3, mr = lane & 7;
      const uint32_t sbase = smem_u32(smem);
      uint32_t qb[8][2];
      float o[8][4], l0 = 0.f, l1 = 0.f;  // columns 2 t, 2 t + 1
      int cur = -1, st = 0, turn = 0, sums = 0;
      auto release = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->empty[st]);
        if (++st == kBkRing) st = 0, turn ^= 1;
      };
      while (true) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sh->full[st], turn, abort, p.status))) break;
        const int2 tok = sh->token[st];
        if (tok.x != cur) {
          if (cur >= 0) {  // the sums of this CTA's share of the pair: each warp adds and writes a quarter of the features
#pragma unroll
            for (int d = 4; d < 32; d *= 2) {
              l0 += __shfl_xor_sync(0xffffffffu, l0, d);
              l1 += __shfl_xor_sync(0xffffffffu, l1, d);
            }
            const uint32_t odd = sums++ & 1;
            if (!__all_sync(0xffffffffu, mbar_wait(&sh->sum_empty, odd ^ 1, abort, p.status))) break;
            float4 own[2];
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              const float4 x = make_float4(o[mt][0], o[mt][1], o[mt][2], o[mt][3]);
              if (mt / 2 == warp)
                own[mt & 1] = x;
              else
                sh->sum_o[warp][(mt - (mt / 2 > warp ? 2 : 0)) * 32 + lane] = x;
            }
            if (row == 0) sh->sum_l[warp][t] = make_float2(l0, l1);
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->sum_full);
            if (!__all_sync(0xffffffffu, mbar_wait(&sh->sum_full, odd, abort, p.status))) break;
            const size_t slot = kPair ? (size_t)cta : (size_t)cta + cur;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float4 v = own[i];
#pragma unroll
              for (int j = 1; j < kBkWarps; ++j) {
                const int w = (warp + j) % kBkWarps;
                const float4 x = sh->sum_o[w][(2 * warp + i - (warp > w ? 2 : 0)) * 32 + lane];
                v.x += x.x;
                v.y += x.y;
                v.z += x.z;
                v.w += x.w;
              }
              p.parts.o[slot * kBkPartO + (2 * warp + i) * 32 + lane] = v;
            }
            if (warp == 0 && lane < 4) {
              float2 v = sh->sum_l[0][lane];
#pragma unroll
              for (int w = 1; w < kBkWarps; ++w) {
                v.x += sh->sum_l[w][lane].x;
                v.y += sh->sum_l[w][lane].y;
              }
              *reinterpret_cast<float2*>(p.parts.l + slot * 8 + 2 * lane) = v;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->sum_empty);
          }
          cur = tok.x;
          if (cur < 0) break;
          l0 = l1 = 0.f;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
          const uint32_t* qs = reinterpret_cast<const uint32_t*>(sq + st * kBkQ) + row * (kD / 2) + t;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            qb[kk][0] = row < kGroup && tok.y > 0 ? qs[kk * 8] : 0u;
            qb[kk][1] = row < kGroup && tok.y > 0 ? qs[kk * 8 + 4] : 0u;
          }
        }
        if (tok.y == 0) {  // (no block)
          release();
          continue;
        }
        const int key0 = warp * 16;
        const bool live = key0 < tok.y, tail = key0 + 16 > tok.y;
        uint32_t h0 = 0u, h1 = 0u, e0 = 0u, e1 = 0u;
        if (live) {
          const uint32_t kb = sbase + st * kBkTile;
          float s[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            uint32_t a[4];
            ldsm_x4(kb + (kk >> 2) * kBkBox + sw128_offset(key0 + (mi & 1) * 8 + mr, (kk & 3) * 16 + (mi >> 1) * 8),
                    a[0], a[1], a[2], a[3]);
            mma_bf16_16816(s[kk & 1], a, qb[kk][0], qb[kk][1]);
          }
          const bool in0 = key0 + row < tok.y, in1 = key0 + 8 + row < tok.y;
          const float w0 = in0 ? capped_weight_precise(s[0][0] + s[1][0]) : 0.f;
          const float w1 = in0 ? capped_weight_precise(s[0][1] + s[1][1]) : 0.f;
          const float w2 = in1 ? capped_weight_precise(s[0][2] + s[1][2]) : 0.f;
          const float w3 = in1 ? capped_weight_precise(s[0][3] + s[1][3]) : 0.f;
          l0 += w0 + w2;
          l1 += w1 + w3;
          split_bf16x2(w0, w1, h0, e0);
          split_bf16x2(w2, w3, h1, e1);
          h0 = movmatrix_trans(h0);
          h1 = movmatrix_trans(h1);
          e0 = movmatrix_trans(e0);
          e1 = movmatrix_trans(e1);
        }
        release();
        if (!__all_sync(0xffffffffu, mbar_wait(&sh->full[st], turn, abort, p.status))) break;
        if (live) {
          const uint32_t vb = sbase + st * kBkTile;
          uint32_t m0 = 0xFFFFFFFFu, m1 = 0xFFFFFFFFu;
          if (tail) {  // rows behind the last may hold anything
            const int k0 = key0 + 2 * t;
            m0 = (k0 < tok.y ? 0x0000FFFFu : 0u) | (k0 + 1 < tok.y ? 0xFFFF0000u : 0u);
            m1 = (k0 + 8 < tok.y ? 0x0000FFFFu : 0u) | (k0 + 9 < tok.y ? 0xFFFF0000u : 0u);
          }
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            uint32_t a[4];
            ldsm_x4_t(vb + (mt >> 2) * kBkBox + sw128_offset(key0 + (mi >> 1) * 8 + mr, (mt & 3) * 16 + (mi & 1) * 8),
                      a[0], a[1], a[2], a[3]);
            if (tail) {
              a[0] &= m0;
              a[1] &= m0;
              a[2] &= m1;
              a[3] &= m1;
            }
            mma_bf16_16816(o[mt], a, h0, h1);
            mma_bf16_16816(o[mt], a, e0, e1);
          }
        }
        release();
      }
    }
  }
  // Started as the dependent of the prefix kernel, this one ends behind it, so that the kernel that waits for this one
  // finds both results. (The last CTA alone waits: the others' places beside the prefix kernel are for the CTAs that follow.)
  if (!kList && blockIdx.x == gridDim.x - 1) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (kPair) {
    // The pair's parts are complete: each CTA of the cluster adds a share of the features and writes it.
    __syncwarp();
    __threadfence();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const int parts = (n0 + share_of - 1) / share_of, each = kBkPartO / ctas;
    const size_t first = (size_t)pair0 * ctas;
    for (int i = tid; i < each; i += kBkThreads) {
      const int at = rank * each + i, c = at % 4 * 2, d = at / 32 * 16 + at % 32 / 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float2 l = make_float2(0.f, 0.f);
#pragma unroll 8
      for (int r = 0; r < parts; ++r) {
        const float4 x = __ldcg(p.parts.o + (first + r) * kBkPartO + at);
        const float2 y = __ldcg(reinterpret_cast<const float2*>(p.parts.l + (first + r) * 8 + c));
        v.x += x.x;
        v.y += x.y;
        v.z += x.z;
        v.w += x.w;
        l.x += y.x;
        l.y += y.y;
      }
      if (c < kGroup) {
        const float i0 = l.x == 0.f ? 0.f : 1.0f / l.x, i1 = l.y == 0.f ? 0.f : 1.0f / l.y;
        const uint32_t lo0 = pack_bf16x2(v.x * i0, v.z * i0), lo1 = pack_bf16x2(v.y * i1, v.w * i1);
        grok_bf16* out = p.out + ((size_t)pair0 * kGroup + c) * kD + d;
        out[0] = grok_bf16(lo0);
        out[8] = grok_bf16(lo0 >> 16);
        out[kD] = grok_bf16(lo1);
        out[kD + 8] = grok_bf16(lo1 >> 16);
      }
    }
  }
}

// ----------------------------------------------------------------------------
// out = (sum of the partial O) / (sum of the partial l) of one (sequence, KV head). Each team of 256 threads adds every
// kTeams-th part: four teams where there are few CTAs and many parts each, one where there are many CTAs.
template <bool kPrefix, int kTeams>
__global__ void __launch_bounds__(kTeams* kBkPartO)
    block_join_kernel(const BlockParts parts, const PrefixParts prefix, const PageMap pm, uint2* out,
                      int32_t* status) {
  __shared__ float4 so[kTeams][kBkPartO];
  __shared__ float sl[kTeams][8];
  __shared__ float acc[kGroup][kD + 4];
  __shared__ float4 po[kPrefix && kTeams > 1 ? kTeams - 1 : 1][kPrefix && kTeams > 1 ? kGroup * kD / 4 : 1];
  __shared__ float psum[kTeams][kPxSums][kGroup];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int g = blockIdx.x, b = blockIdx.y, pair = b * kKVHeads + g;
  const int tid = threadIdx.x, team = tid / kBkPartO, at = tid % kBkPartO;
  const int2 mine = parts.pair[pair];
  const int4 pre = kPrefix ? prefix.pair[pair] : make_int4(0, 0, 0, 0);
  if (mine.y < 0) return;  // (the whole CTA)
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = 0.f;
#pragma unroll 4
  for (int i = team; i < mine.y; i += kTeams) {
    const size_t s = (size_t)mine.x + i;
    const float4 x = parts.o[s * kBkPartO + at];
    v.x += x.x;
    v.y += x.y;
    v.z += x.z;
    v.w += x.w;
    if (at < 8) l += parts.l[s * 8 + at];
  }
  // The prefix's parts: thread (head, feature quad) of a team. The other threads: does the table agree with the one that
  // was read?
  float4 pv = make_float4(0.f, 0.f, 0.f, 0.f);
  float pl = 0.f;
  const int h = at % kGroup, quad = at / kGroup;
  if (kPrefix && quad < kD / 4) {
    const int r = pre.z + h;
#pragma unroll 4
    for (int i = team; i < pre.y; i += kTeams) {
      const size_t s = (size_t)pre.x + i;
      const float4 x = prefix.o[(s * (kD / 4) + quad) * kPxRows + r];
      pv.x += x.x;
      pv.y += x.y;
      pv.z += x.z;
      pv.w += x.w;
      if (quad < kPxSums) pl += prefix.l[(s * kPxSums + quad) * kPxRows + r];
    }
    if (quad < kPxSums) psum[team][quad][h] = pl;
    if (kTeams > 1 && team > 0) po[team - 1][at] = pv;
  } else if (kPrefix && g == 0) {
    constexpr int kEach = kBkPartO - kGroup * kD / 4;
    const int seq = pre.w & 0xFFFF;
    for (int i = team * kEach + at - kGroup * kD / 4; i < int(uint32_t(pre.w) >> 16); i += kTeams * kEach)
      if (pm.table[(size_t)b * pm.max_pages + i] != pm.table[(size_t)seq * pm.max_pages + i])
        report(status, GROK_DEV_BAD_GROUP);
  }
  if (at < 8) sl[team][at] = l;
  if (kTeams > 1) {
    so[team][at] = v;
    __syncthreads();
  }
  if (team == 0) {
#pragma unroll
    for (int w = 1; w < kTeams; ++w) {
      const float4 x = so[w][at];
      v.x += x.x;
      v.y += x.y;
      v.z += x.z;
      v.w += x.w;
    }
    // accumulator layout: features 16 mt + row (+ 8) of heads 2 t, 2 t + 1
    const int d = at / 32 * 16 + at % 32 / 4, c = at % 4 * 2;
    if (c < kGroup) {
      acc[c][d] = v.x;
      acc[c + 1][d] = v.y;
      acc[c][d + 8] = v.z;
      acc[c + 1][d + 8] = v.w;
    }
  }
  __syncthreads();
  if (team == 0 && quad < kD / 4) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kTeams; ++w) sum += sl[w][h];
    if (kPrefix) {
#pragma unroll
      for (int w = 0; w < kTeams; ++w) {
#pragma unroll
        for (int i = 0; i < kPxSums; ++i) sum += psum[w][i][h];
        if (w > 0) {
          const float4 x = po[w - 1][at];
          pv.x += x.x;
          pv.y += x.y;
          pv.z += x.z;
          pv.w += x.w;
        }
      }
    }
    const float inv = sum == 0.f ? 0.f : 1.0f / sum;  // (a list without a block: zeros)
    const float* x = &acc[h][quad * 4];
    out[((size_t)pair * kGroup + h) * (kD / 4) + quad] =
        make_uint2(pack_bf16x2((x[0] + pv.x) * inv, (x[1] + pv.y) * inv),
                   pack_bf16x2((x[2] + pv.z) * inv, (x[3] + pv.w) * inv));
  }
}

// ----------------------------------------------------------------------------
static size_t up256(size_t n) { return (n + 255) & ~size_t(255); }
static size_t bk_slots(int B, int sms) { return (size_t)B * kKVHeads + (size_t)kBkCtas * sms; }
static BlockParts block_parts(char* ws, int B, int sms) {
  const size_t slots = bk_slots(B, sms);
  BlockParts p;
  p.o = reinterpret_cast<float4*>(ws);
  ws += up256(slots * kBkPartO * sizeof(float4));
  p.l = reinterpret_cast<float*>(ws);
  ws += up256(slots * 8 * sizeof(float));
  p.pair = reinterpret_cast<int2*>(ws);
  return p;
}
size_t block_parts_bytes(int B, int sms) {
  const size_t slots = bk_slots(B, sms);
  return up256(slots * kBkPartO * sizeof(float4)) + up256(slots * 8 * sizeof(float)) +
         up256((size_t)B * kKVHeads * sizeof(int2));
}

// Query tiles of the prefix kernel: the sum of ceil(n_i / 21) over groups of two sequences at least.
static size_t px_slots(int B, int n_groups, int sms) {
  const size_t tiles = std::min(B / 2, B / kPxSeqs + n_groups);
  return tiles * kKVHeads + sms;
}
PrefixParts prefix_parts(char* ws, int B, int n_groups, int sms) {
  const size_t slots = px_slots(B, n_groups, sms);
  PrefixParts p;
  p.o = reinterpret_cast<float4*>(ws);
  ws += slots * kPxRows * kD * 4;
  p.l = reinterpret_cast<float*>(ws);
  ws += slots * kPxSums * kPxRows * 4;
  p.pair = reinterpret_cast<int4*>(ws);
  return p;
}
size_t prefix_parts_bytes(int B, int n_groups, int sms) {
  return px_slots(B, n_groups, sms) * kPxRows * (kD + kPxSums) * 4 + up256((size_t)B * kKVHeads * sizeof(int4));
}

// A pool as (64 features, row, half of the features, KV head).
static grok_status encode_pool(CUtensorMap* map, const grok_bf16* pool, int n_pages, bool last) {
  const uint64_t dims[4] = {kD / 2, uint64_t(n_pages) * GROK_PAGE_TOKENS, 2, kKVHeads};
  const uint64_t strides[3] = {uint64_t(kKVHeads) * kD * 2, kD, kD * 2};
  const uint32_t box[4] = {kD / 2, last ? 16u : uint32_t(kBlk), last ? 1u : 2u, 1};
  return encode_tmap_bf16_4d(map, pool, dims, strides, box);
}

grok_status encode_pools(BlockArgs* a, const grok_bf16* k_pool, const grok_bf16* v_pool, int n_pages) {
  grok_status st = encode_pool(&a->tm_k, k_pool, n_pages, false);
  if (st == GROK_OK) st = encode_pool(&a->tm_v, v_pool, n_pages, false);
  if (st == GROK_OK) st = encode_pool(&a->tm_k16, k_pool, n_pages, true);
  if (st == GROK_OK) st = encode_pool(&a->tm_v16, v_pool, n_pages, true);
  return st;
}

template <int kMode>
static grok_status bk_launch(const BlockArgs& a, const BkParams& p, int sms, int ctas) {
  constexpr int kSmem = kBkSmem<kMode != kOwn>;
  grok_status st;
  static bool attr_set[kMaxDevices] = {};  // per device; idempotent: every thread would set the same value
  int dev = 0;
  if ((st = device_index(&dev)) != GROK_OK) return st;
  cudaError_t e;
  if (!attr_set[dev]) {
    e = cudaFuncSetAttribute(block_decode_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(block_decode_kernel<kMode>, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return fail(cuda_status(e), "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    attr_set[dev] = true;
  }
  const int grid = kMode == kPairs ? a.B * kKVHeads * ctas : kBkCtas * sms;
  e = launch(kMode == kOwn, kMode == kPairs ? ctas : 1, block_decode_kernel<kMode>, dim3(grid), kBkThreads, kSmem, a.stream,
             a.tm_k, a.tm_v, a.tm_k16, a.tm_v16, p);
  if (e != cudaSuccess) return fail(cuda_status(e), "block decode launch: %s", cudaGetErrorString(e));
  return check_launch("block decode");
}

grok_status block_decode_run(const BlockArgs& a, char* ws, const PrefixParts* prefix, int sms) {
  BkParams p;
  p.q = reinterpret_cast<const uint8_t*>(a.q_rot);
  p.pm = a.pm;
  p.kv_len = a.kv_len;
  p.B = a.B;
  p.sel = a.sel;
  p.budget = a.sel ? a.budget : kBlkMax;
  p.groups = a.groups;
  p.parts = block_parts(ws, a.B, sms);
  p.prefix_pair = prefix ? prefix->pair : nullptr;
  p.status = a.status;
  p.out = a.out;
  if (a.sel && (long long)a.B * kKVHeads <= kBkCtas * sms) {
    // One wave of clusters holds all pairs. That saves the plan and the join, but a pair's blocks stay with its cluster,
    // whatever the other sequences' lengths, which are not known here: clusters take the call where no CTA can get more
    // than kBkPairMost blocks. Equal shares against clusters, us, lists all full, and one sequence's full beside others of
    // two blocks: budget 16, 2 sequences, 2 blocks to a CTA, 10.0 and 7.8, 9.5 and 7.2; 32, 8 sequences, 8 blocks, 19.0 and
    // 17.5, 10.7 and 11.4; 8, 32 sequences, 8 blocks, 19.2 and 16.9, 10.7 and 11.8. Beyond, the gain stays (32, 32
    // sequences, 32 blocks: 49.4 and 44.9) and the loss grows (12.7 and 26.0).
    int ctas = 8;
    while (a.B * kKVHeads * ctas > kBkCtas * sms) ctas /= 2;
    if ((a.budget + ctas - 1) / ctas <= kBkPairMost)
      return bk_launch<kPairs>(a, p, sms, ctas);
  }
  grok_status st = a.sel ? bk_launch<kLists>(a, p, sms, 1) : bk_launch<kOwn>(a, p, sms, 1);
  if (st != GROK_OK) return st;
  const int teams = a.B * kKVHeads <= 2 * sms ? 4 : 1;
  auto kernel = prefix ? (teams == 4 ? block_join_kernel<true, 4> : block_join_kernel<true, 1>)
                       : (teams == 4 ? block_join_kernel<false, 4> : block_join_kernel<false, 1>);
  const cudaError_t e = launch(true, 1, kernel, dim3(kKVHeads, a.B), teams * kBkPartO, 0, a.stream, p.parts,
                                       prefix ? *prefix : PrefixParts{}, a.pm, reinterpret_cast<uint2*>(a.out), a.status);
  if (e != cudaSuccess) return fail(cuda_status(e), "block join launch: %s", cudaGetErrorString(e));
  return check_launch("block join");
}

grok_status page_args(int n_pages, int max_pages, int B, const char* who) {
  if (n_pages < 1 || max_pages < 1 || (long long)n_pages * GROK_PAGE_TOKENS > (1LL << 31) - 1 ||
      (long long)max_pages * GROK_PAGE_TOKENS > GROK_MAX_POSITION || B < 1 || B > 65535)
    return fail(GROK_ERR_INVALID_ARG,
                "%s: need 1 <= n_pages < 2^24, 1 <= max_pages <= %d, 1 <= B <= 65535 (n_pages=%d max_pages=%d B=%d)", who,
                GROK_MAX_POSITION / GROK_PAGE_TOKENS, n_pages, max_pages, B);
  return GROK_OK;
}

}  // namespace grok

using namespace grok;

extern "C" grok_status grok_attn_decode_sparse_workspace(int B, int budget, size_t* bytes) {
  if (!bytes) return fail(GROK_ERR_INVALID_ARG, "grok_attn_decode_sparse_workspace: null pointer");
  if (B < 1 || B > 65535 || budget < 1 || budget > kBlkMax)
    return fail(GROK_ERR_INVALID_ARG,
                "grok_attn_decode_sparse_workspace: need 1 <= B <= 65535, 1 <= budget <= %d (B=%d budget=%d)", kBlkMax, B,
                budget);
  int sms = 0;
  const grok_status st = device_sm_count(&sms);
  if (st != GROK_OK) return st;
  *bytes = block_parts_bytes(B, sms);
  return GROK_OK;
}

extern "C" grok_status grok_attn_decode_sparse_paged(const grok_bf16* q_rot, const grok_bf16* k_pool,
                                                     const grok_bf16* v_pool, int n_pages, const int32_t* block_table,
                                                     int max_pages, const int32_t* kv_len, const int32_t* sel,
                                                     int budget, int B, void* workspace, size_t workspace_bytes,
                                                     grok_bf16* out, int32_t* dev_status, void* stream) {
  const char* who = "grok_attn_decode_sparse_paged";
  if (!q_rot || !k_pool || !v_pool || !block_table || !kv_len || !sel || !workspace || !out)
    return fail(GROK_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned16(q_rot) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return fail(GROK_ERR_INVALID_ARG, "%s: bf16 tensors must be 16-byte aligned", who);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(GROK_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  grok_status st = page_args(n_pages, max_pages, B, who);
  if (st != GROK_OK) return st;
  if (budget < 1 || budget > kBlkMax)
    return fail(GROK_ERR_INVALID_ARG, "%s: need 1 <= budget <= %d (budget=%d)", who, kBlkMax, budget);
  int sms = 0;
  if ((st = device_sm_count(&sms)) != GROK_OK) return st;
  const size_t need = block_parts_bytes(B, sms);
  if (workspace_bytes < need)
    return fail(GROK_ERR_INVALID_ARG, "%s: workspace of %zu bytes is smaller than the %zu needed", who, workspace_bytes,
                need);
  BlockArgs a = {};
  if ((st = encode_pools(&a, k_pool, v_pool, n_pages)) != GROK_OK) return st;
  a.q_rot = q_rot;
  a.pm = PageMap{block_table, max_pages, n_pages};
  a.kv_len = kv_len;
  a.B = B;
  a.sel = sel;
  a.budget = budget;
  a.out = out;
  a.status = dev_status;
  a.stream = static_cast<cudaStream_t>(stream);
  return block_decode_run(a, static_cast<char*>(workspace), nullptr, sms);
}
