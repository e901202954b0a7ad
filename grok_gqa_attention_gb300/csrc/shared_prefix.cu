// Decode for a batch whose sequences share long prefixes: the prefix is read once
// for all of a group's queries, on the 5th-generation tensor cores (tcgen05, TMEM, TMA).
//
// Code-reading guide ch. 4 §4.4.1, §4.5.2-§4.5.4. One query row per (sequence, query
// head): the 6 heads of a KV head times 21 sequences are 126 of a tile's 128 rows. All of
// them see every row of the prefix, so nothing is masked. Weights are taken relative to
// the bound 30 of the capped logits, w = exp(30 tanh(x / 30) - 30), so partial sums add
// without a maximum: the prefix's, and those of each sequence's own rows
// (block_decode.cu), which runs beside this kernel.
//
// Work: (group, KV head, query tile, 64-key tile) in this order, dealt out to one CTA per
// SM in equal contiguous shares; a share that leaves a (group, KV head, query tile) writes
// a part of its unnormalised O and row sums. Per key tile
//   S = Q K^T (128 x 64, one of five buffers of 64 TMEM columns; Q is in TMEM too), P over S
//   in place as two bf16 halves that sum to P to 2^-16, O += P_hi V + P_lo V.
// Warps: 0 TMA, 1 the issue of S, 18 that of P V, 2-17 the softmax, four warps to a key
// tile. S runs up to five tiles ahead of P V.
//
// Bound by the products, beside 32 KB of tiles loaded a step: a step takes 1190 clocks,
// its products alone 770 (S with Q from TMEM 256, with Q from shared memory 360, P V
// 512), its loads alone 820. 256 sequences behind 16384 rows: 110 us, 0.94 PFLOP/s
// (1.4 with the lo halves'). Tried and slower: two query tiles to a CTA, which halves the
// loads, with Q in shared memory (124 us) or one buffer of S each (188 us); K and V
// loaded in step (120 us); tiles in three places of each ring (136 us). Of 21 sequences
// or fewer the tiles come from HBM: 4 x 16 behind up to 16384 rows 36 us, 4.6 TB/s.
#include "block_decode.cuh"

namespace grok {

constexpr int kPxTeams = kPxSums;           // of four softmax warps, a key tile each in turn
constexpr int kPxEach = kD / kPxTeams;      // features that a team moves of Q and O
constexpr int kPxThreads = 32 * (3 + 4 * kPxTeams);
// Registers: the launch bound is above the launch, for at most 80 a thread, which leaves room beside this CTA for one of
// the kernel over the sequences' own rows.
constexpr int kPxBound = 768;
constexpr int kPxBox = kBlk * 128;          // [64 rows][64 bf16]: one half of the features of a key tile
constexpr int kPxTile = 2 * kPxBox;
constexpr int kPxStages = 4;                // of the K ring and of the V ring
constexpr int kPxLead = 2;                  // K tiles loaded ahead of the V tile of the same keys
// TMEM columns: O, Q, and the S (then P) of key tiles in turn
constexpr int kPxBufs = 5;
// (K of tile t + kPxLead waits for S of kPxStages tiles before it, and that for P V of kPxBufs tiles before that, whose V
// has to be loaded by then)
static_assert(kPxLead < kPxStages + kPxBufs, "the producer's order");
constexpr uint32_t kPxO = 0, kPxQ = kD, kPxS = kPxQ + kD / 2;
static_assert(kPxS + kPxBufs * kBlk <= 512, "TMEM columns");

struct PxShared {
  uint64_t q_full, q_empty, o_full, o_empty, done;
  uint64_t k_full[kPxStages], k_empty[kPxStages], v_full[kPxStages], v_empty[kPxStages];
  uint64_t s_full[kPxBufs], p_full[kPxBufs], s_empty[kPxBufs];
  GroupTable groups;
  int units[kGroupsMax + 1];  // key tiles before each group's
  int items[kGroupsMax + 1];  // (KV head, query tile) pairs before each group's
  int warp_units[kPxThreads / 32], warp_items[kPxThreads / 32];
  int2 place[64];  // of the key tiles in turn: row of the pools, KV head
  uint32_t tmem;
  int abort;
};
constexpr int kPxSmem = 1024 + kPxStages * 2 * kPxTile + int(sizeof(PxShared));
static_assert(kPxSmem <= kPxSmemMax, "shared memory");

struct PxParams {
  const uint4* q;
  Groups groups;
  PageMap pm;
  int B;
  PrefixParts parts;
  int32_t* status;
};

// A share's run of key tiles of one (group, KV head, query tile).
struct PxRun {
  int g, item;      // KV head; number of the (group, KV head, query tile)
  int k0, n, keys;  // first key tile, number of them, of the item
  int base;         // the item's first unit
  int seq0, seqs;   // sequences of the query tile
  int table;        // the sequence whose block table is read: the group's first
};

__device__ __forceinline__ PxRun px_run(const PxParams& p, const PxShared* sh, int unit, int hi) {
  PxRun r;
  int lo = 0, up = p.groups.n;
  while (up - lo > 1) {
    const int mid = (lo + up) >> 1;
    if (sh->units[mid] <= unit) lo = mid; else up = mid;
  }
  const int a = sh->groups.start[lo], n = sh->groups.start[lo + 1] - a;
  const int tiles = (n + kPxSeqs - 1) / kPxSeqs;
  r.table = a;
  r.keys = sh->groups.pages[lo] * kBlkPerPage;
  const int in = unit - sh->units[lo], it = in / r.keys;
  r.g = it / tiles;
  r.item = sh->items[lo] + it;
  r.k0 = in % r.keys;
  r.n = min(r.keys - r.k0, hi - unit);
  r.base = unit - r.k0;
  r.seq0 = a + it % tiles * kPxSeqs;
  r.seqs = min(kPxSeqs, a + n - r.seq0);
  return r;
}

// 32 lanes x 16 columns, waited for; and the store of 8.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Weights of 16 logits of a row: 2^(kT tanh(y) - kT) as bf16 halves hi and lo, their sum added to l. tanh runs on the
// special-function unit, exp2 there for half of the columns and as a polynomial on the FMA pipe for the others.
// (tanh.approx is off by 8e-6, a weight by 2.4e-4. The form of the other decodes, three special functions and 1e-5, takes 152 us
// of 256 sequences behind 16384 rows instead of 130, 79 of 128 behind 4096 instead of 78; an output is rounded by up to 2^-8.)
__device__ __forceinline__ void px_weights(const uint32_t (&s)[16], uint64_t& l, uint32_t (&hi)[8], uint32_t (&lo)[8]) {
  const uint64_t y2 = f2_pack(kY, kY), t2 = f2_pack(kT, kT), m2 = f2_pack(-kT, -kT), z2 = f2_pack(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    float y0, y1, w0, w1;
    f2_unpack(f2_mul(f2_pack(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), y2), y0, y1);
    const uint64_t t = f2_pack(tanh_approx(y0), tanh_approx(y1));
    const uint64_t x = f2_fma(t, t2, m2);
    if (e & 1) {
      exp2_poly_f2(x, w0, w1);
      l = f2_fma(t, z2, l);  // (the polynomial may lose a NaN)
    } else {
      float x0, x1;
      f2_unpack(x, x0, x1);
      w0 = ex2_approx(x0);
      w1 = ex2_approx(x1);
    }
    const uint64_t w = f2_pack(w0, w1);
    l = f2_add(l, w);
    hi[e] = pack_bf16x2(w0, w1);
    float r0, r1;
    f2_unpack(f2_sub(w, f2_pack(bf16lo_to_f32(hi[e]), bf16hi_to_f32(hi[e]))), r0, r1);
    lo[e] = pack_bf16x2(r0, r1);
  }
}

__global__ void __launch_bounds__(kPxBound, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const PxParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sK = smem;
  uint8_t* sV = sK + kPxStages * kPxTile;
  PxShared* sh = reinterpret_cast<PxShared*>(sV + kPxStages * kPxTile);
  volatile int* abort = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // The kernel over the sequences' own rows starts beside this one.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    mbar_init(&sh->q_full, kPxTeams * 128);
    mbar_init(&sh->q_empty, 1);
    mbar_init(&sh->o_full, 1);
    mbar_init(&sh->o_empty, kPxTeams * 128);
    mbar_init(&sh->done, 2);
    for (int i = 0; i < kPxStages; ++i) {
      mbar_init(&sh->k_full[i], 1);
      mbar_init(&sh->k_empty[i], 1);
      mbar_init(&sh->v_full[i], 1);
      mbar_init(&sh->v_empty[i], 1);
    }
    for (int i = 0; i < kPxBufs; ++i) {
      mbar_init(&sh->s_full[i], 1);
      mbar_init(&sh->p_full[i], 128);
      mbar_init(&sh->s_empty[i], 1);
    }
    sh->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // The plan: key tiles and items before each group's, a group a thread. (Groups that are not usable are dropped: every
  // sequence is then decoded by itself, by the other kernel, which reports it.)
  const bool fine = load_groups(p.groups, p.B, p.pm.max_pages, &sh->groups, tid);
  if (fine && tid < p.groups.n)  // (the group's table entries come closer meanwhile)
    for (int i = 0; i < sh->groups.pages[tid]; i += 32)
      asm volatile("prefetch.global.L2 [%0];" ::"l"(p.pm.table + (size_t)sh->groups.start[tid] * p.pm.max_pages + i));
  if (warp == 1) {
    tmem_alloc(&sh->tmem, 512);
    tmem_relinquish();
  }
  const int n_groups = __syncthreads_and(fine) ? p.groups.n : 0;
  static_assert(kGroupsMax <= kPxThreads, "a group a thread");
  {
    const int pages = tid < n_groups ? sh->groups.pages[tid] : 0;
    const int tiles = pages ? (sh->groups.start[tid + 1] - sh->groups.start[tid] + kPxSeqs - 1) / kPxSeqs : 0;
    const int items = tiles * kKVHeads, units = items * pages * kBlkPerPage;
    int iu = units, ii = items;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int a = __shfl_up_sync(0xffffffffu, iu, d), c = __shfl_up_sync(0xffffffffu, ii, d);
      if (lane >= d) iu += a, ii += c;
    }
    if (n_groups > 32) {
      if (lane == 31) sh->warp_units[warp] = iu, sh->warp_items[warp] = ii;
      __syncthreads();
      for (int w = 0; w < warp && w < kGroupsMax / 32; ++w) iu += sh->warp_units[w], ii += sh->warp_items[w];
    }
    if (tid < n_groups) {
      sh->units[tid] = iu - units;
      sh->items[tid] = ii - items;
      if (tid == n_groups - 1) sh->units[n_groups] = iu;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem;
  const int total = n_groups ? sh->units[n_groups] : 0;
  const int share = max(1, (total + int(gridDim.x) - 1) / int(gridDim.x));
  const int u0 = int(min((long long)blockIdx.x * share, (long long)total)), u1 = min(u0 + share, total), n_tiles = u1 - u0;

  if (n_tiles > 0) {
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      // K runs kPxLead tiles ahead of V, as S does of P V. The tiles' places are looked up 32 at a time, one a lane, so that a
      // tile costs this warp few instructions: it shares its scheduler with softmax warps. (With 100 or 150 to a tile, as a
      // lookup in the loop takes, the loads bound the kernel at 800 clocks each: 256 sequences behind 16384 rows 145 us.)
      int k_loads = 0, v_loads = 0, k_st = 0, v_st = 0;
      uint32_t k_turn = 1, v_turn = 1;
      bool ok = true;
      for (int t = 0; t < n_tiles + kPxLead && ok; ++t) {
        if (t % 32 == 0) {
          if (t + lane < n_tiles) {
            const PxRun run = px_run(p, sh, u0 + t + lane, u1);
            sh->place[(t + lane) % 64] =
                make_int2(max(0, blk_page(p.pm, run.table, run.k0, p.status)) * GROK_PAGE_TOKENS + run.k0 % kBlkPerPage * kBlk,
                          run.g);
          }
          __syncwarp();
        }
        if (lane == 0) {
          if (t < n_tiles) {
            ok = mbar_wait(&sh->k_empty[k_st], k_turn, abort, p.status);
            if (ok) {
              const int2 at = sh->place[t % 64];
              mbar_arrive_expect_tx(&sh->k_full[k_st], kPxTile);
              tma_load_4d(sK + k_st * kPxTile, &tm_k, &sh->k_full[k_st], 0, at.x, 0, at.y);
              ++k_loads;
              if (++k_st == kPxStages) k_st = 0, k_turn ^= 1;
            }
          }
          if (ok && t >= kPxLead) {
            ok = mbar_wait(&sh->v_empty[v_st], v_turn, abort, p.status);
            if (ok) {
              const int2 at = sh->place[(t - kPxLead) % 64];
              mbar_arrive_expect_tx(&sh->v_full[v_st], kPxTile);
              tma_load_4d(sV + v_st * kPxTile, &tm_v, &sh->v_full[v_st], 0, at.x, 0, at.y);
              ++v_loads;
              if (++v_st == kPxStages) v_st = 0, v_turn ^= 1;
            }
          }
        }
        ok = __shfl_sync(0xffffffffu, int(ok), 0);
      }
      for (int u = u0; u < u1;) {  // the items' parts: one of each CTA from the first on that takes some of it
        const PxRun run = px_run(p, sh, u, u1);
        if (run.k0 == 0 && lane < run.seqs)
          p.parts.pair[(size_t)(run.seq0 + lane) * kKVHeads + run.g] =
              make_int4(int(blockIdx.x) + run.item, (run.base + run.keys - 1) / share - int(blockIdx.x) + 1,
                        lane * kGroup, int(uint32_t(run.keys / kBlkPerPage) << 16 | uint32_t(run.table)));
        u += run.n;
      }
      // Copies in flight (only after an abort) land before the CTA exits.
      if (lane == 0) {
        volatile int never = 0;
        for (int i = max(0, k_loads - kPxStages); i < k_loads; ++i)
          mbar_wait(&sh->k_full[i % kPxStages], (i / kPxStages) & 1, &never, p.status);
        for (int i = max(0, v_loads - kPxStages); i < v_loads; ++i)
          mbar_wait(&sh->v_full[i % kPxStages], (i / kPxStages) & 1, &never, p.status);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ S = Q K^T
      // (The issuing warps run converged through the waits; one fixed lane issues the products and commits.)
      const bool leader = elect_one();
      const uint64_t kd = make_sdesc_sw128(smem_u32(sK), 16, 1024);
      constexpr uint32_t idesc = make_idesc_bf16(kPxRows, kBlk, 0);
      int end = 0, runs = -1, st = 0, buf = 0;
      uint32_t turn = 0, free_turn = 1;
      for (int t = 0; t < n_tiles; ++t) {
        bool w = true;
        if (t == end) {
          end += px_run(p, sh, u0 + t, u1).n;
          ++runs;
          w = mbar_wait(&sh->q_full, runs & 1, abort, p.status);
        }
        w = w && mbar_wait(&sh->k_full[st], turn, abort, p.status) &&
            mbar_wait(&sh->s_empty[buf], free_turn, abort, p.status);
        if (!__all_sync(0xffffffffu, w)) break;
        tc_fence_after();
        if (leader) {
          const uint64_t k = kd + uint64_t((st * kPxTile) >> 4);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_ts(tmem + kPxS + buf * kBlk, tmem + kPxQ + kk * 8, k + uint64_t(((kk >> 2) * kPxBox + (kk & 3) * 32) >> 4),
                    idesc, kk > 0);
          umma_commit(&sh->s_full[buf]);
          umma_commit(&sh->k_empty[st]);
          if (t == end - 1) umma_commit(&sh->q_empty);
        }
        __syncwarp();
        if (++st == kPxStages) st = 0, turn ^= 1;
        if (++buf == kPxBufs) buf = 0, free_turn ^= 1;
      }
      // No product may still run when TMEM is released.
      if (leader) umma_commit(&sh->done);
      __syncwarp();
      volatile int never = 0;
      mbar_wait(&sh->done, 0, &never, p.status);
    } else if (warp == kPxThreads / 32 - 1) {
      // ------------------------------------------------------------ O += P V
      const bool leader = elect_one();
      const uint64_t vd = make_sdesc_sw128(smem_u32(sV), kPxBox, 1024);
      constexpr uint32_t idesc = make_idesc_bf16(kPxRows, kD, 1);
      int first = 0, end = px_run(p, sh, u0, u1).n, runs = 0, st = 0, buf = 0;
      uint32_t turn = 0, p_turn = 0;
      for (int t = 0; t < n_tiles; ++t) {
        bool w = true;
        if (t == end) {
          first = end;
          end += px_run(p, sh, u0 + t, u1).n;
          ++runs;
          w = mbar_wait(&sh->o_empty, (runs & 1) ^ 1, abort, p.status);
        }
        w = w && mbar_wait(&sh->v_full[st], turn, abort, p.status) && mbar_wait(&sh->p_full[buf], p_turn, abort, p.status);
        if (!__all_sync(0xffffffffu, w)) break;
        tc_fence_after();
        if (leader) {
          const uint64_t v = vd + uint64_t((st * kPxTile) >> 4);
          const uint32_t pc = tmem + kPxS + buf * kBlk;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {  // 16 keys each
            umma_ts(tmem + kPxO, pc + kk * 16, v + uint64_t((kk * 2048) >> 4), idesc, t > first || kk > 0);
            umma_ts(tmem + kPxO, pc + kk * 16 + 8, v + uint64_t((kk * 2048) >> 4), idesc, 1u);
          }
          umma_commit(&sh->s_empty[buf]);
          umma_commit(&sh->v_empty[st]);
          if (t == end - 1) umma_commit(&sh->o_full);
        }
        __syncwarp();
        if (++st == kPxStages) st = 0, turn ^= 1;
        if (++buf == kPxBufs) buf = 0, p_turn ^= 1;
      }
      if (leader) umma_commit(&sh->done);
      __syncwarp();
      volatile int never = 0;
      mbar_wait(&sh->done, 0, &never, p.status);
    } else {
      // ------------------------------------------------------------ softmax of the key tiles t = team (mod 4), epilogue
      const int team = (warp - 2) >> 2, quad = warp & 3, r = quad * 32 + lane;
      const uint32_t trow = tmem + (uint32_t(quad * 32) << 16);
      // Q of a run into TMEM: this thread's row, a team's share of the features (zeros for rows without a query).
      auto load_q = [&](const PxRun& run) {
        if (quad * 32 < run.seqs * kGroup) {
          const bool mine = r < run.seqs * kGroup;
          const uint4* src = p.q + ((size_t)(run.seq0 + r / kGroup) * kQHeads + run.g * kGroup + r % kGroup) * (kD / 8) +
                             team * (kPxEach / 8);
#pragma unroll
          for (int c = 0; c < kPxEach / 16; ++c) {
            const uint4 z = make_uint4(0, 0, 0, 0), x = mine ? src[2 * c] : z, y = mine ? src[2 * c + 1] : z;
            const uint32_t w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
            tmem_st8(trow + kPxQ + team * (kPxEach / 2) + c * 8, w);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        mbar_arrive(&sh->q_full);
      };
      int t = team, t0 = 0, runs = 0, u = u0;
      PxRun run = px_run(p, sh, u0, u1);
      load_q(run);
      while (true) {
        const int rows = run.seqs * kGroup;
        const bool live = quad * 32 < rows;  // (of the warp; the other warps' P is never looked at)
        uint64_t l = f2_pack(0.f, 0.f);
        bool ok = true;
        t0 += run.n;
        u += run.n;
        for (; t < t0; t += kPxTeams) {
          const int buf = t % kPxBufs;
          ok = __all_sync(0xffffffffu, mbar_wait(&sh->s_full[buf], (t / kPxBufs) & 1, abort, p.status));
          if (!ok) break;
          tc_fence_after();
          if (live) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {  // P of 16 keys over their S: hi in 8 columns, lo in 8
              uint32_t s[16], hi[8], lo[8];
              const uint32_t col = trow + kPxS + buf * kBlk + c * 16;
              tmem_ld16(col, s);
              px_weights(s, l, hi, lo);
              tmem_st8(col, hi);
              tmem_st8(col + 8, lo);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          mbar_arrive(&sh->p_full[buf]);
        }
        if (!ok) break;
        const size_t slot = (size_t)blockIdx.x + run.item;
        if (u < u1) {  // the next run's Q, once this one's is read, ahead of this one's O
          run = px_run(p, sh, u, u1);
          if (!__all_sync(0xffffffffu, mbar_wait(&sh->q_empty, runs & 1, abort, p.status))) break;
          tc_fence_after();
          load_q(run);
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&sh->o_full, runs & 1, abort, p.status))) break;
        ++runs;
        tc_fence_after();
        if (live) {
          float4* po = p.parts.o + (slot * (kD / 4) + team * (kPxEach / 4)) * kPxRows + r;
#pragma unroll
          for (int c = 0; c < kPxEach / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(trow + kPxO + team * kPxEach + c * 16, o);
            if (r < rows)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                po[(c * 4 + q) * kPxRows] = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                                        __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
          }
          float l0, l1;
          f2_unpack(l, l0, l1);
          if (r < rows) p.parts.l[(slot * kPxSums + team) * kPxRows + r] = l0 + l1;
        }
        tc_fence_before();
        mbar_arrive(&sh->o_empty);
        if (t0 >= n_tiles) break;
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace grok

using namespace grok;

static grok_status shared_args(int B, int max_pages, int n_groups, const char* who) {
  if (B < 1 || B > 65535 || max_pages < 1 || (long long)max_pages * GROK_PAGE_TOKENS > GROK_MAX_POSITION ||
      n_groups < 1 || n_groups > kGroupsMax)
    return fail(GROK_ERR_INVALID_ARG,
                "%s: need 1 <= B <= 65535, 1 <= max_pages <= %d, 1 <= n_groups <= %d (B=%d max_pages=%d n_groups=%d)", who,
                GROK_MAX_POSITION / GROK_PAGE_TOKENS, kGroupsMax, B, max_pages, n_groups);
  return GROK_OK;
}

extern "C" grok_status grok_attn_decode_shared_workspace(int B, int max_pages, int n_groups, size_t* bytes) {
  if (!bytes) return fail(GROK_ERR_INVALID_ARG, "grok_attn_decode_shared_workspace: null pointer");
  grok_status st = shared_args(B, max_pages, n_groups, "grok_attn_decode_shared_workspace");
  if (st != GROK_OK) return st;
  int sms = 0;
  if ((st = device_sm_count(&sms)) != GROK_OK) return st;
  *bytes = block_parts_bytes(B, sms) + prefix_parts_bytes(B, n_groups, sms);
  return GROK_OK;
}

extern "C" grok_status grok_attn_decode_shared_paged(const grok_bf16* q_rot, const grok_bf16* k_pool,
                                                     const grok_bf16* v_pool, int n_pages, const int32_t* block_table,
                                                     int max_pages, const int32_t* kv_len, int B,
                                                     const int32_t* group_start, const int32_t* shared_pages,
                                                     int n_groups, void* workspace, size_t workspace_bytes,
                                                     grok_bf16* out, int32_t* dev_status, void* stream) {
  const char* who = "grok_attn_decode_shared_paged";
  if (!q_rot || !k_pool || !v_pool || !block_table || !kv_len || !group_start || !shared_pages || !workspace || !out)
    return fail(GROK_ERR_INVALID_ARG, "%s: null pointer", who);
  if (!aligned16(q_rot) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return fail(GROK_ERR_INVALID_ARG, "%s: bf16 tensors must be 16-byte aligned", who);
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(GROK_ERR_INVALID_ARG, "%s: workspace must be 256-byte aligned", who);
  grok_status st = page_args(n_pages, max_pages, B, who);
  if (st == GROK_OK) st = shared_args(B, max_pages, n_groups, who);
  if (st != GROK_OK) return st;
  int sms = 0;
  if ((st = device_sm_count(&sms)) != GROK_OK) return st;
  const size_t blocks = block_parts_bytes(B, sms), need = blocks + prefix_parts_bytes(B, n_groups, sms);
  if (workspace_bytes < need)
    return fail(GROK_ERR_INVALID_ARG, "%s: workspace of %zu bytes is smaller than the %zu needed", who, workspace_bytes,
                need);
  static bool attr_set[kMaxDevices] = {};  // per device; idempotent: every thread would set the same value
  int dev = 0;
  if ((st = device_index(&dev)) != GROK_OK) return st;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPxSmem);
    // (the SM's whole shared memory, so that the next kernel's CTAs fit beside this one's)
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(prefix_kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return fail(cuda_status(e), "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    attr_set[dev] = true;
  }
  BlockArgs a = {};
  if ((st = encode_pools(&a, k_pool, v_pool, n_pages)) != GROK_OK) return st;
  char* ws = static_cast<char*>(workspace);
  const PrefixParts prefix = prefix_parts(ws + blocks, B, n_groups, sms);
  PxParams p;
  p.q = reinterpret_cast<const uint4*>(q_rot);
  p.groups = Groups{group_start, shared_pages, n_groups};
  p.pm = PageMap{block_table, max_pages, n_pages};
  p.B = B;
  p.parts = prefix;
  p.status = dev_status;
  const cudaError_t e = launch(false, 1, prefix_kernel, dim3(sms), kPxThreads, kPxSmem, static_cast<cudaStream_t>(stream),
                               a.tm_k, a.tm_v, p);
  if (e != cudaSuccess) return fail(cuda_status(e), "prefix launch: %s", cudaGetErrorString(e));
  a.q_rot = q_rot;
  a.pm = p.pm;
  a.kv_len = kv_len;
  a.B = B;
  a.groups = p.groups;
  a.out = out;
  a.status = dev_status;
  a.stream = static_cast<cudaStream_t>(stream);
  return block_decode_run(a, ws, &prefix, sms);
}
