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
//   S = Q K^T (128 x 64, 64 TMEM columns of one of four buffers), P over S in place as two
//   bf16 halves that sum to P to 2^-16, O += P_hi V + P_lo V.
// Warps: 0 TMA, 1 MMA, 2-5 and 6-9 the softmax of even and of odd key tiles. Products of
// the next tiles are issued ahead of the softmax of this one.
#include "block_decode.cuh"

namespace grok {

constexpr int kPxThreads = 320;
constexpr int kPxStages = 3;
constexpr int kPxAhead = 2;                 // S products issued ahead of P V
static_assert(kPxAhead < kPxStages && kPxAhead < 4, "stages and S buffers");
constexpr int kPxQBox = kPxRows * 128;      // [128 rows][64 bf16]: one half of the features
constexpr int kPxBox = kBlk * 128;          // the same of a key tile
constexpr int kPxTile = 2 * kPxBox;
constexpr int kPxQLoad = 2 * kPxSeqs * kGroup * 128;

struct PxShared {
  uint64_t q_full, q_empty, o_full, o_empty, done;
  uint64_t kv_full[kPxStages], kv_empty[kPxStages];
  uint64_t s_full[4], p_full[4];
  int units[kGroupsMax + 1];  // key tiles before each group's
  int items[kGroupsMax + 1];  // (KV head, query tile) pairs before each group's
  int warp_units[kPxThreads / 32], warp_items[kPxThreads / 32];
  uint32_t tmem;
  int abort;
};
constexpr int kPxSmem = 1024 + 2 * kPxQBox + kPxStages * 2 * kPxTile + int(sizeof(PxShared));

struct PxParams {
  Groups groups;
  PageMap pm;
  int B;
  PrefixParts parts;
  int32_t* status;
};

// A share's run of key tiles of one (group, KV head, query tile).
struct PxRun {
  int group, g, mt;  // group, KV head, query tile
  int item;          // number of the (group, KV head, query tile)
  int k0, n;         // first key tile and number of them
  int first, last;   // units: the item's first one and the one behind its last
  int seq0, seqs;    // sequences of the query tile
};

__device__ __forceinline__ PxRun px_run(const PxParams& p, const PxShared* sh, int unit, int hi) {
  PxRun r;
  int lo = 0, up = p.groups.n;
  while (up - lo > 1) {
    const int mid = (lo + up) >> 1;
    if (sh->units[mid] <= unit) lo = mid; else up = mid;
  }
  r.group = lo;
  const int a = p.groups.start[lo], n = p.groups.start[lo + 1] - a;
  const int tiles = (n + kPxSeqs - 1) / kPxSeqs, keys = p.groups.pages[lo] * kBlkPerPage;
  const int in = unit - sh->units[lo], it = in / keys;
  r.g = it / tiles;
  r.mt = it % tiles;
  r.item = sh->items[lo] + it;
  r.k0 = in % keys;
  r.n = min(keys - r.k0, hi - unit);
  r.first = unit - r.k0;
  r.last = r.first + keys;
  r.seq0 = a + r.mt * kPxSeqs;
  r.seqs = min(kPxSeqs, a + n - r.seq0);
  return r;
}

// Weights of 32 logits of a row: 2^(kT tanh(y) - kT) as bf16 halves hi and lo, their sum added to l. tanh runs on the
// special-function unit, exp2 there for half of the columns and as a polynomial on the FMA pipe for the others.
__device__ __forceinline__ void px_weights(const uint32_t (&s)[32], uint64_t& l, uint32_t (&hi)[16], uint32_t (&lo)[16]) {
  const uint64_t y2 = f2_pack(kY, kY), t2 = f2_pack(kT, kT), m2 = f2_pack(-kT, -kT), z2 = f2_pack(0.f, 0.f);
#pragma unroll
  for (int e = 0; e < 16; ++e) {
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

__global__ void __launch_bounds__(kPxThreads, 1)
    prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const PxParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * kPxQBox;  // stages: K halves, V halves
  PxShared* sh = reinterpret_cast<PxShared*>(sKV + kPxStages * 2 * kPxTile);
  volatile int* abort = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // The kernel over the sequences' own rows starts beside this one.
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (tid == 0) {
    mbar_init(&sh->q_full, 1);
    mbar_init(&sh->q_empty, 1);
    mbar_init(&sh->o_full, 1);
    mbar_init(&sh->o_empty, 256);
    mbar_init(&sh->done, 1);
    for (int s = 0; s < kPxStages; ++s) {
      mbar_init(&sh->kv_full[s], 1);
      mbar_init(&sh->kv_empty[s], 1);
    }
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sh->s_full[s], 1);
      mbar_init(&sh->p_full[s], 128);
    }
    sh->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  // The plan: key tiles and items before each group's. (Groups that are not usable are dropped: every sequence is then
  // decoded by itself, by the other kernel, which reports it.)
  const bool usable = groups_ok(p.groups, p.B, p.pm.max_pages);
  const int n_groups = usable ? p.groups.n : 0;
  {
    const int per = (n_groups + kPxThreads - 1) / kPxThreads;
    const int i0 = min(tid * per, n_groups), i1 = min(i0 + per, n_groups);
    auto of = [&](int i, int& items) {
      const int pages = group_pages(p.groups, i);
      items = pages == 0 ? 0 : (p.groups.start[i + 1] - p.groups.start[i] + kPxSeqs - 1) / kPxSeqs * kKVHeads;
      return items * pages * kBlkPerPage;
    };
    int units = 0, items = 0;
    for (int i = i0; i < i1; ++i) {
      int n;
      units += of(i, n);
      items += n;
    }
    int iu = units, ii = items;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const int a = __shfl_up_sync(0xffffffffu, iu, d), c = __shfl_up_sync(0xffffffffu, ii, d);
      if (lane >= d) iu += a, ii += c;
    }
    if (lane == 31) sh->warp_units[warp] = iu, sh->warp_items[warp] = ii;
    __syncthreads();
    int u = iu - units, m = ii - items;
    for (int w = 0; w < warp; ++w) u += sh->warp_units[w], m += sh->warp_items[w];
    for (int i = i0; i < i1; ++i) {
      int n;
      sh->units[i] = u;
      sh->items[i] = m;
      u += of(i, n);
      m += n;
    }
    if (i1 == n_groups && i0 < i1) sh->units[n_groups] = u;
  }
  if (warp == 1) {
    tmem_alloc(&sh->tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh->tmem, o_tm = tmem + 256;
  const int total = n_groups ? sh->units[n_groups] : 0;
  const int share = max(1, (total + int(gridDim.x) - 1) / int(gridDim.x));
  const int u0 = int(min((long long)blockIdx.x * share, (long long)total)), u1 = min(u0 + share, total);

  if (u0 < u1) {
    if (warp == 0) {
      // ------------------------------------------------------------ TMA producer
      int t = 0, runs = 0, q_loads = 0;
      bool ok = true;
      for (int u = u0; u < u1 && ok; ++runs) {
        const PxRun r = px_run(p, sh, u, u1);
        if (r.k0 == 0 && lane < r.seqs) {  // the item's parts: one of each CTA from this one on that takes some of it
          const int last = (r.last - 1) / share;
          p.parts.pair[(size_t)(r.seq0 + lane) * kKVHeads + r.g] =
              make_int4(int(blockIdx.x) + r.item, last - int(blockIdx.x) + 1, lane * kGroup,
                        int(uint32_t(r.last - r.first) / kBlkPerPage << 16 | uint32_t(r.seq0)));
        }
        if (lane == 0) {
          if (!mbar_wait(&sh->q_empty, (runs & 1) ^ 1, abort, p.status)) {
            ok = false;
          } else {
            mbar_arrive_expect_tx(&sh->q_full, kPxQLoad);
            ++q_loads;
            tma_load_4d(sQ, &tm_q, &sh->q_full, 0, r.g * kGroup, r.seq0, 0);
            tma_load_4d(sQ + kPxQBox, &tm_q, &sh->q_full, 64, r.g * kGroup, r.seq0, 0);
            for (int k = 0; k < r.n; ++k, ++t) {
              const int st = t % kPxStages;
              if (!mbar_wait(&sh->kv_empty[st], ((t / kPxStages) & 1) ^ 1, abort, p.status)) {
                ok = false;
                break;
              }
              const int blk = r.k0 + k;
              const int row = max(0, blk_page(p.pm, r.seq0, blk, p.status)) * GROK_PAGE_TOKENS + blk % kBlkPerPage * kBlk;
              uint8_t* dst = sKV + st * 2 * kPxTile;
              mbar_arrive_expect_tx(&sh->kv_full[st], 2 * kPxTile);
              tma_load_4d(dst, &tm_k, &sh->kv_full[st], 0, r.g, row, 0);
              tma_load_4d(dst + kPxBox, &tm_k, &sh->kv_full[st], 64, r.g, row, 0);
              tma_load_4d(dst + kPxTile, &tm_v, &sh->kv_full[st], 0, r.g, row, 0);
              tma_load_4d(dst + kPxTile + kPxBox, &tm_v, &sh->kv_full[st], 64, r.g, row, 0);
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        u += r.n;
      }
      // Copies in flight (only after an abort) land before the CTA exits.
      if (lane == 0) {
        volatile int never = 0;
        for (int i = max(0, t - kPxStages); i < t; ++i)
          mbar_wait(&sh->kv_full[i % kPxStages], (i / kPxStages) & 1, &never, p.status);
        if (q_loads > 0) mbar_wait(&sh->q_full, (q_loads - 1) & 1, &never, p.status);
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA issuer
      // (converged through the waits; one fixed lane issues the products and commits)
      const bool leader = elect_one();
      const uint64_t qd = make_sdesc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t kd = make_sdesc_sw128(smem_u32(sKV), 16, 1024);
      const uint64_t vd = make_sdesc_sw128(smem_u32(sKV + kPxTile), kPxBox, 1024);
      constexpr uint32_t idesc_s = make_idesc_bf16(kPxRows, kBlk, 0), idesc_o = make_idesc_bf16(kPxRows, kD, 1);
      const int n = u1 - u0;
      PxRun rs = px_run(p, sh, u0, u1), ro = rs;
      int ts = 0, s_end = rs.n, s_runs = 0;       // next S product, the end of its run, its run's number
      int o_first = 0, o_end = ro.n, o_runs = 0;  // run of the next P V
      bool ok = true;
      for (int t = 0; t < n && ok; ++t) {
        while (ts < n && ts <= t + kPxAhead) {
          if (ts == s_end) {
            rs = px_run(p, sh, u0 + ts, u1);
            s_end += rs.n;
            ++s_runs;
          }
          const int st = ts % kPxStages;
          bool w = mbar_wait(&sh->kv_full[st], (ts / kPxStages) & 1, abort, p.status);
          if (ts == s_end - rs.n) w = w && mbar_wait(&sh->q_full, s_runs & 1, abort, p.status);
          ok = __all_sync(0xffffffffu, w);
          if (!ok) break;
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              umma_ss(tmem + (ts & 3) * 64, qd + uint64_t(((kk >> 2) * kPxQBox + (kk & 3) * 32) >> 4),
                      kd + uint64_t((st * 2 * kPxTile + (kk >> 2) * kPxBox + (kk & 3) * 32) >> 4), idesc_s, kk > 0);
            umma_commit(&sh->s_full[ts & 3]);
            if (ts == s_end - 1) umma_commit(&sh->q_empty);
          }
          __syncwarp();
          ++ts;
        }
        if (!ok) break;
        if (t == o_end) {
          ro = px_run(p, sh, u0 + t, u1);
          o_first = o_end;
          o_end += ro.n;
          ++o_runs;
          ok = __all_sync(0xffffffffu, mbar_wait(&sh->o_empty, (o_runs & 1) ^ 1, abort, p.status));
          if (!ok) break;
        }
        ok = __all_sync(0xffffffffu, mbar_wait(&sh->p_full[t & 3], (t >> 2) & 1, abort, p.status));
        if (!ok) break;
        tc_fence_after();
        if (leader) {
          const int st = t % kPxStages;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {  // 16 keys each
            const uint32_t pc = tmem + (t & 3) * 64 + (kk >> 1) * 32 + (kk & 1) * 8;
            const uint64_t v = vd + uint64_t((st * 2 * kPxTile + kk * 2048) >> 4);
            umma_ts(o_tm, pc, v, idesc_o, t > o_first || kk > 0);
            umma_ts(o_tm, pc + 16, v, idesc_o, 1u);
          }
          umma_commit(&sh->kv_empty[st]);
          if (t == o_end - 1) umma_commit(&sh->o_full);
        }
        __syncwarp();
      }
      // No product may still run when TMEM is released.
      if (leader) umma_commit(&sh->done);
      __syncwarp();
      volatile int never = 0;
      mbar_wait(&sh->done, 0, &never, p.status);
    } else {
      // ------------------------------------------------------------ softmax of the key tiles t = team (mod 2), epilogue
      const int team = warp < 6 ? 0 : 1, quad = warp & 3, r = quad * 32 + lane;
      const uint32_t trow = tmem + (uint32_t(quad * 32) << 16);
      int t0 = 0, runs = 0;
      bool ok = true;
      for (int u = u0; u < u1; ++runs) {
        const PxRun run = px_run(p, sh, u, u1);
        const int rows = run.seqs * kGroup;
        const bool live = quad * 32 < rows;  // (of the warp; the other warps' P is never looked at)
        uint64_t l = f2_pack(0.f, 0.f);
        for (int t = t0 + ((t0 ^ team) & 1); t < t0 + run.n; t += 2) {
          ok = __all_sync(0xffffffffu, mbar_wait(&sh->s_full[t & 3], (t >> 2) & 1, abort, p.status));
          if (!ok) break;
          tc_fence_after();
          if (live) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              uint32_t s[32], hi[16], lo[16];
              const uint32_t col = trow + (t & 3) * 64 + c * 32;
              tmem_ld32(col, s);
              tmem_wait_ld_dep(s);
              px_weights(s, l, hi, lo);
              tmem_st16(col, hi);
              tmem_st16(col + 16, lo);
            }
            tmem_wait_st();
          }
          tc_fence_before();
          mbar_arrive(&sh->p_full[t & 3]);
        }
        if (!ok) break;
        t0 += run.n;
        u += run.n;
        ok = __all_sync(0xffffffffu, mbar_wait(&sh->o_full, runs & 1, abort, p.status));
        if (!ok) break;
        tc_fence_after();
        const size_t slot = (size_t)blockIdx.x + run.item;
        if (live) {
          float4* po = p.parts.o + (slot * (kD / 4) + team * 16) * kPxRows + r;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t o[32];
            tmem_ld32(trow + 256 + team * 64 + c * 32, o);
            tmem_wait_ld_dep(o);
            if (r < rows)
#pragma unroll
              for (int q = 0; q < 8; ++q)
                po[(c * 8 + q) * kPxRows] = make_float4(__uint_as_float(o[4 * q]), __uint_as_float(o[4 * q + 1]),
                                                        __uint_as_float(o[4 * q + 2]), __uint_as_float(o[4 * q + 3]));
          }
          float l0, l1;
          f2_unpack(l, l0, l1);
          if (r < rows) p.parts.l[(slot * 2 + team) * kPxRows + r] = l0 + l1;
        }
        tc_fence_before();
        mbar_arrive(&sh->o_empty);
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
  CUtensorMap tq, tk, tv;
  {
    const uint64_t dims[4] = {kD, kQHeads, uint64_t(B), 1};
    const uint64_t strides[3] = {kD * 2, uint64_t(kQHeads) * kD * 2, uint64_t(B) * kQHeads * kD * 2};
    const uint32_t box[4] = {64, kGroup, kPxSeqs, 1};
    if ((st = encode_tmap_bf16_4d(&tq, q_rot, dims, strides, box)) != GROK_OK) return st;
  }
  {
    const uint64_t rows = uint64_t(n_pages) * GROK_PAGE_TOKENS;
    const uint64_t dims[4] = {kD, kKVHeads, rows, 1};
    const uint64_t strides[3] = {kD * 2, uint64_t(kKVHeads) * kD * 2, rows * kKVHeads * kD * 2};
    const uint32_t box[4] = {64, 1, kBlk, 1};
    if ((st = encode_tmap_bf16_4d(&tk, k_pool, dims, strides, box)) != GROK_OK) return st;
    if ((st = encode_tmap_bf16_4d(&tv, v_pool, dims, strides, box)) != GROK_OK) return st;
  }
  static bool attr_set[kMaxDevices] = {};  // per device; idempotent: every thread would set the same value
  int dev = 0;
  if ((st = device_index(&dev)) != GROK_OK) return st;
  if (!attr_set[dev]) {
    cudaError_t e = cudaFuncSetAttribute(prefix_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPxSmem);
    if (e != cudaSuccess) return fail(cuda_status(e), "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    attr_set[dev] = true;
  }
  char* ws = static_cast<char*>(workspace);
  const PrefixParts prefix = prefix_parts(ws + blocks, B, n_groups, sms);
  PxParams p;
  p.groups = Groups{group_start, shared_pages, n_groups};
  p.pm = PageMap{block_table, max_pages, n_pages};
  p.B = B;
  p.parts = prefix;
  p.status = dev_status;
  prefix_kernel<<<sms, kPxThreads, kPxSmem, static_cast<cudaStream_t>(stream)>>>(tq, tk, tv, p);
  if ((st = check_launch("prefix")) != GROK_OK) return st;
  BlockArgs a = {};
  a.q_rot = q_rot;
  a.k_pool = k_pool;
  a.v_pool = v_pool;
  a.pm = p.pm;
  a.kv_len = kv_len;
  a.B = B;
  a.groups = p.groups;
  a.out = out;
  a.status = dev_status;
  a.stream = static_cast<cudaStream_t>(stream);
  return block_decode_run(a, ws, &prefix, sms);
}
