// RoPE on Q and K and the append to the 8-bit KV cache.
//
// Code-reading guide ch. 4 §4.3.1, §4.4 (rotation, cache write) with the cache
// in 8 bits: scale = RN32(max|x| / Q) over the block's rows so far, code =
// round(RN32(x RN32(1 / scale))).
//
// One CTA per (block of the sequence's rows, KV head, sequence): it rotates the
// block's new keys and the six query heads of the same tokens (one read of
// each cos/sin pair serves all seven), takes the largest magnitude of keys and
// values, and writes the codes. The block that is open keeps its bf16 rows in
// open_k / open_v, so a later append can quantise the whole block again from
// the unrounded rows; that is needed only when the new rows raise the scale,
// otherwise the codes there already are the ones a new pass would give and only
// the new rows are written.
//
// Memory-bound: per token 16 KB of q, k, v read, 12 KB of q_rot and 2 KB of codes
// written. Measured (graph replays, one GB300): 8192 tokens (257 MB) 44.5 us,
// 5.7 TB/s, 0.85 of the copy rate (1032 CTAs are 1.7 rounds of the resident ones);
// 8 ragged sequences of up to 2048 (467 MB) 73.0 us, 0.95; one token 4.1 us.
#include "host.cuh"
#include "kv8.cuh"
#include "rope_math.cuh"

namespace grok {

constexpr int kApThreads = 256;

struct ApParams {
  grok_kv8_cache c;
  const uint4 *q, *k, *v;
  uint4* q_rot;
  const int32_t *start_pos, *cache_len, *valid_len;
  const float4 *cos_tab, *sin_tab;
  int T, tab_n;
  int32_t* status;
};

// Largest |x| of packed bf16 pairs, as bit patterns (NaN and infinity rank last).
__device__ __forceinline__ uint32_t absmax4(uint32_t m, const uint4& x) {
  m = __vmaxu2(m, x.x & 0x7FFF7FFFu);
  m = __vmaxu2(m, x.y & 0x7FFF7FFFu);
  m = __vmaxu2(m, x.z & 0x7FFF7FFFu);
  return __vmaxu2(m, x.w & 0x7FFF7FFFu);
}

// The block's largest magnitudes of keys and values (bf16 bits) over the CTA.
__device__ __forceinline__ void cta_absmax(uint32_t& k, uint32_t& v, uint32_t (*red)[2]) {
  const int warp = threadIdx.x >> 5;
  k = __reduce_max_sync(0xffffffffu, max(k & 0xFFFFu, k >> 16));
  v = __reduce_max_sync(0xffffffffu, max(v & 0xFFFFu, v >> 16));
  if ((threadIdx.x & 31) == 0) {
    red[warp][0] = k;
    red[warp][1] = v;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kApThreads / 32; ++w) {
    k = max(k, red[w][0]);
    v = max(v, red[w][1]);
  }
}

template <int kKind>
__device__ __forceinline__ float scale_of(uint32_t bits) {
  if (bits >= 0x7F80u) return __uint_as_float(0x7FC00000u);  // a NaN or an infinity in the block
  const float a = __uint_as_float(bits << 16);
  return a < 0x1p-100f ? 0.f : __fdiv_rn(a, kKind == GROK_KV8_INT8 ? 127.f : 448.f);
}

// Codes of four values: inv = 0 (zero or non-finite scale) gives zeros.
template <int kKind>
__device__ __forceinline__ uint32_t codes4(float x0, float x1, float x2, float x3, float inv) {
  if (inv == 0.f) return 0u;
  x0 = __fmul_rn(x0, inv), x1 = __fmul_rn(x1, inv), x2 = __fmul_rn(x2, inv), x3 = __fmul_rn(x3, inv);
  if (kKind == GROK_KV8_INT8) {
    const uint32_t a = __byte_perm(__float2int_rn(x0), __float2int_rn(x1), 0x0040);
    const uint32_t b = __byte_perm(__float2int_rn(x2), __float2int_rn(x3), 0x0040);
    return __byte_perm(a, b, 0x5410);
  }
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r)
      : "f"(x0), "f"(x1), "f"(x2), "f"(x3));
  return r;
}

__device__ __forceinline__ float bf16_at(const uint4& x, int e) {
  const uint32_t w = e < 2 ? x.x : e < 4 ? x.y : e < 6 ? x.z : x.w;
  return e & 1 ? bf16hi_to_f32(w) : bf16lo_to_f32(w);
}

template <int kKind>
__device__ __forceinline__ uint2 codes8(const uint4& x, float inv) {
  return make_uint2(codes4<kKind>(bf16lo_to_f32(x.x), bf16hi_to_f32(x.x), bf16lo_to_f32(x.y), bf16hi_to_f32(x.y), inv),
                    codes4<kKind>(bf16lo_to_f32(x.z), bf16hi_to_f32(x.z), bf16lo_to_f32(x.w), bf16hi_to_f32(x.w), inv));
}

// cos and sin of the eight pairs 8c .. 8c+7 at a position.
__device__ __forceinline__ void load_cs(const ApParams& p, int pos, int c, float (&tc)[8], float (&ts)[8]) {
  const size_t t0 = (size_t)pos * 16 + 2 * c;
  const float4 c0 = __ldg(p.cos_tab + t0), c1 = __ldg(p.cos_tab + t0 + 1);
  const float4 s0 = __ldg(p.sin_tab + t0), s1 = __ldg(p.sin_tab + t0 + 1);
  tc[0] = c0.x, tc[1] = c0.y, tc[2] = c0.z, tc[3] = c0.w, tc[4] = c1.x, tc[5] = c1.y, tc[6] = c1.z, tc[7] = c1.w;
  ts[0] = s0.x, ts[1] = s0.y, ts[2] = s0.z, ts[3] = s0.w, ts[4] = s1.x, ts[5] = s1.y, ts[6] = s1.z, ts[7] = s1.w;
}

// Keys and values of the sequence's j-th touched block (block len / 64 + j).
template <int kKind>
__device__ void append_block(const ApParams& p, int b, int g, int j, int len, int n, int start, uint32_t (*red)[2]) {
  const int tid = threadIdx.x;
  const int blk = len / kKv8Block + j;
  const int lo = j == 0 ? len % kKv8Block : 0;                    // rows [0, lo) were there before
  const int hi = min(kKv8Block, len + n - blk * kKv8Block);       // rows [lo, hi) are new
  const int first = blk * kKv8Block - len;                        // new token of row 0
  const size_t head = (size_t)b * kKVHeads + g;
  const int id = kv8_block_id(p.c.table, head * p.c.max_blocks + blk, p.c.n_blocks, tid == 0 ? p.status : nullptr);
  if (id < 0) return;  // uniform over the CTA
  const float k_was = lo > 0 ? p.c.k_scale[id] : 0.f, v_was = lo > 0 ? p.c.v_scale[id] : 0.f;

  // Keys: this thread's rows kr and kr + 32, pairs 8 kc .. 8 kc + 7. Values: rows 4 vq .. 4 vq + 3, features 8 vc ..
  const int kr = tid >> 3, kc = tid & 7, vq = tid & 15, vc = tid >> 4;
  uint4 kx[2][2], vx[4];
  uint32_t km = 0, vm = 0;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    kx[m][0] = kx[m][1] = make_uint4(0, 0, 0, 0);
    const int row = kr + 32 * m;
    if (row >= lo && row < hi) {
      const uint4* src = p.k + (((size_t)b * p.T + first + row) * kKVHeads + g) * 16;
      float tc[8], ts[8];
      load_cs(p, start + first + row, kc, tc, ts);
      rotate8(__ldg(src + kc), __ldg(src + kc + 8), tc, ts, kx[m][0], kx[m][1]);
      km = absmax4(absmax4(km, kx[m][0]), kx[m][1]);
    }
  }
#pragma unroll
  for (int m = 0; m < 4; ++m) {
    vx[m] = make_uint4(0, 0, 0, 0);
    const int row = 4 * vq + m;
    if (row >= lo && row < hi) {
      vx[m] = __ldg(p.v + (((size_t)b * p.T + first + row) * kKVHeads + g) * 16 + vc);
      vm = absmax4(vm, vx[m]);
    }
  }
  cta_absmax(km, vm, red);
  float ks = scale_of<kKind>(km), vs = scale_of<kKind>(vm);
  // With old rows in the block: while the new rows do not raise the scale, the old codes stand.
  const bool k_all = lo == 0 || !(ks <= k_was), v_all = lo == 0 || !(vs <= v_was);
  uint4* open_k = reinterpret_cast<uint4*>(p.c.open_k) + head * (kKv8Block * 16);
  uint4* open_v = reinterpret_cast<uint4*>(p.c.open_v) + head * (kKv8Block * 16);
  if (lo > 0 && (k_all || v_all)) {
    __syncthreads();  // red is read
#pragma unroll
    for (int m = 0; m < 2; ++m)
      if (kr + 32 * m < lo) {
        kx[m][0] = open_k[(kr + 32 * m) * 16 + kc];
        kx[m][1] = open_k[(kr + 32 * m) * 16 + kc + 8];
        km = absmax4(absmax4(km, kx[m][0]), kx[m][1]);
      }
#pragma unroll
    for (int m = 0; m < 4; ++m)
      if (4 * vq + m < lo) {
        vx[m] = open_v[(4 * vq + m) * 16 + vc];
        vm = absmax4(vm, vx[m]);
      }
    cta_absmax(km, vm, red);
    ks = scale_of<kKind>(km), vs = scale_of<kKind>(vm);
  }
  if (!k_all) ks = k_was;
  if (!v_all) vs = v_was;
  const int k_lo = k_all ? 0 : lo, v_lo = v_all ? 0 : lo;
  const float k_inv = ks > 0.f ? __fdiv_rn(1.f, ks) : 0.f, v_inv = vs > 0.f ? __fdiv_rn(1.f, vs) : 0.f;
  if (tid == 0) {
    if (k_all) p.c.k_scale[id] = ks;
    if (v_all) p.c.v_scale[id] = vs;
  }
  uint8_t* k_dst = static_cast<uint8_t*>(p.c.k_pool) + (size_t)id * kKv8Bytes;
  uint8_t* v_dst = static_cast<uint8_t*>(p.c.v_pool) + (size_t)id * kKv8Bytes;
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int row = kr + 32 * m;
    if (row >= k_lo && row < hi) {
      *reinterpret_cast<uint2*>(k_dst + row * 64 + 8 * kc) = codes8<kKind>(kx[m][0], k_inv);
      *reinterpret_cast<uint2*>(k_dst + kKv8Bytes / 2 + row * 64 + 8 * kc) = codes8<kKind>(kx[m][1], k_inv);
    }
  }
  // Four rows of a feature make one word of the feature's 64 bytes.
  const int r0 = 4 * vq;
  if (r0 + 3 >= v_lo && r0 < hi) {
    const bool whole = r0 >= v_lo && r0 + 4 <= hi;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t w =
          codes4<kKind>(bf16_at(vx[0], e), bf16_at(vx[1], e), bf16_at(vx[2], e), bf16_at(vx[3], e), v_inv);
      uint8_t* dst = v_dst + (8 * vc + e) * kKv8Block + r0;
      if (whole) {
        *reinterpret_cast<uint32_t*>(dst) = w;
      } else {
#pragma unroll
        for (int m = 0; m < 4; ++m)
          if (r0 + m >= v_lo && r0 + m < hi) dst[m] = uint8_t(w >> (8 * m));
      }
    }
  }
  if (hi < kKv8Block) {  // the block stays open: keep the new rows
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const int row = kr + 32 * m;
      if (row >= lo && row < hi) {
        open_k[row * 16 + kc] = kx[m][0];
        open_k[row * 16 + kc + 8] = kx[m][1];
      }
    }
#pragma unroll
    for (int m = 0; m < 4; ++m)
      if (r0 + m >= lo && r0 + m < hi) open_v[(r0 + m) * 16 + vc] = vx[m];
  }
}

// kHeads: query heads loaded at a time. Three leave room for a fourth CTA on an SM
// (8192 tokens: 47.9 -> 44.6 us; eight of 64 sequences 10.3 -> 9.0); six are
// quicker where three CTAs per SM take the whole call (one token of one sequence:
// 4.3 us against 4.5; 104 of 11 11.2 against 12.0; 2048 of one 14.9 against 15.8).
template <int kKind, int kHeads>
__global__ void __launch_bounds__(kApThreads, kHeads == kGroup ? 3 : 4) kv8_append_kernel(const ApParams p) {
  __shared__ uint32_t red[kApThreads / 32][2];
  const int j = blockIdx.x, g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int start = __ldg(p.start_pos + b), len = __ldg(p.cache_len + b);
  const int n = p.valid_len ? __ldg(p.valid_len + b) : p.T;
  int bad = 0;
  if (start < 0 || (long long)start + p.T > p.tab_n) bad |= GROK_DEV_BAD_START;
  if (n < 1 || n > p.T) bad |= GROK_DEV_BAD_VALID;
  if (len < 0 || (long long)len + max(n, 0) > (long long)p.c.max_blocks * kKv8Block) bad |= GROK_DEV_BAD_KV_LEN;
  if (bad) {
    if (j == 0 && g == 0 && tid == 0) report(p.status, bad);
    return;
  }
  const int used = len % kKv8Block;
  // The rotated queries of this block's tokens, the KV head's six heads.
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int i = j * kKv8Block - used + (tid >> 3) + 32 * m, c = tid & 7;
    if (i >= 0 && i < p.T) {
      const size_t at = (((size_t)b * p.T + i) * kQHeads + g * kGroup) * 16 + c;
      float tc[8], ts[8];
#pragma unroll
      for (int h0 = 0; h0 < kGroup; h0 += kHeads) {
        uint4 x1[kHeads], x2[kHeads];
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          x1[h] = __ldg(p.q + at + (h0 + h) * 16);
          x2[h] = __ldg(p.q + at + (h0 + h) * 16 + 8);
        }
        if (h0 == 0) load_cs(p, start + i, c, tc, ts);
#pragma unroll
        for (int h = 0; h < kHeads; ++h) {
          uint4 y1, y2;
          rotate8(x1[h], x2[h], tc, ts, y1, y2);
          p.q_rot[at + (h0 + h) * 16] = y1;
          p.q_rot[at + (h0 + h) * 16 + 8] = y2;
        }
      }
    }
  }
  const int last = (used + n - 1) / kKv8Block;  // the last touched block
  if (j > last) return;
  // The rows of an open block that this call closes and those of the block that
  // it leaves open share open_k / open_v: one CTA reads the first, then writes
  // the second.
  const bool tail = used > 0 && last > 0 && (used + n) % kKv8Block != 0;
  if (j == last && tail) return;
  append_block<kKind>(p, b, g, j, len, n, start, red);
  if (j == 0 && tail) {
    __syncthreads();
    append_block<kKind>(p, b, g, last, len, n, start, red);
  }
}

// One token of many sequences: a CTA per sequence, a warp per KV head, where the
// kernel above has a CTA of 256 threads for a few dozen live ones and runs them in
// rounds. Where a token raises its block's scale (in a block of r random rows with
// probability 1 / r for K and for V), the CTA's threads share the old rows of all such
// heads. Steps of random rows, us, this kernel against the one above: 32 sequences
// 7.1 to 8.1 against 5.9 to 7.0, 64 8.3 to 9.8 against 8.6 to 9.3, 128 8.6 to 10.7
// against 14.5, 256 10.7 to 13.0 against 25.
constexpr int kApMany = 64;  // sequences from which it is used

template <int kKind>
__global__ void __launch_bounds__(kApThreads, 4) kv8_append_one_kernel(const ApParams p) {
  constexpr int kHeadsQ = kGroup * 8;  // (head, chunk) pairs of a KV head's queries
  __shared__ uint32_t s_top[2][kKVHeads];  // largest magnitudes of the blocks that are written again; 0: none
  __shared__ int s_id[kKVHeads], s_list[2][kKVHeads];
  const int b = blockIdx.x, tid = threadIdx.x, g = tid >> 5, lane = tid & 31, c = lane & 7;
  const int start = __ldg(p.start_pos + b), len = __ldg(p.cache_len + b);
  const int n = p.valid_len ? __ldg(p.valid_len + b) : 1;
  int bad = 0;
  if (start < 0 || start >= p.tab_n) bad |= GROK_DEV_BAD_START;
  if (n != 1) bad |= GROK_DEV_BAD_VALID;
  if (len < 0 || (long long)len + max(n, 0) > (long long)p.c.max_blocks * kKv8Block) bad |= GROK_DEV_BAD_KV_LEN;
  if (bad) {
    if (tid == 0) report(p.status, bad);
    return;
  }
  const int row = len % kKv8Block;
  const size_t head = (size_t)b * kKVHeads + g;
  const int id = kv8_block_id(p.c.table, head * p.c.max_blocks + len / kKv8Block, p.c.n_blocks,
                              lane == 0 ? p.status : nullptr);
  uint4 x1[2], x2[2], kx[2] = {}, vx = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (lane + 32 * u < kHeadsQ) {
      const size_t at = (head * kGroup + (lane + 32 * u) / 8) * 16 + c;
      x1[u] = __ldg(p.q + at);
      x2[u] = __ldg(p.q + at + 8);
    }
  if (lane < 8) {  // the key: pairs 8 c .. 8 c + 7; the value, next lanes: features 8 (lane - 8) ..
    kx[0] = __ldg(p.k + head * 16 + c);
    kx[1] = __ldg(p.k + head * 16 + c + 8);
  } else if (lane < 24) {
    vx = __ldg(p.v + head * 16 + lane - 8);
  }
  float tc[8], ts[8];
  load_cs(p, start, c, tc, ts);
  const float k_was = row > 0 && id >= 0 ? p.c.k_scale[id] : 0.f, v_was = row > 0 && id >= 0 ? p.c.v_scale[id] : 0.f;
#pragma unroll
  for (int u = 0; u < 2; ++u)
    if (lane + 32 * u < kHeadsQ) {
      const size_t at = (head * kGroup + (lane + 32 * u) / 8) * 16 + c;
      uint4 y1, y2;
      rotate8(x1[u], x2[u], tc, ts, y1, y2);
      p.q_rot[at] = y1;
      p.q_rot[at + 8] = y2;
    }
  if (lane < 8) rotate8(kx[0], kx[1], tc, ts, kx[0], kx[1]);
  uint32_t km = absmax4(absmax4(0u, kx[0]), kx[1]), vm = absmax4(0u, vx);
  km = __reduce_max_sync(0xffffffffu, max(km & 0xFFFFu, km >> 16));
  vm = __reduce_max_sync(0xffffffffu, max(vm & 0xFFFFu, vm >> 16));
  float ks = scale_of<kKind>(km), vs = scale_of<kKind>(vm);
  // (as in append_block)
  const bool k_all = row == 0 || !(ks <= k_was), v_all = row == 0 || !(vs <= v_was);
  const bool again = row > 0 && id >= 0 && (k_all || v_all);
  if (lane == 0) {
    s_top[0][g] = again && k_all ? max(km, 1u) : 0u;
    s_top[1][g] = again && v_all ? max(vm, 1u) : 0u;
    s_id[g] = id;
  }
  const bool any = __syncthreads_or(again);
  const uint4* open_k = reinterpret_cast<const uint4*>(p.c.open_k) + (size_t)b * kKVHeads * (kKv8Block * 16);
  const uint4* open_v = reinterpret_cast<const uint4*>(p.c.open_v) + (size_t)b * kKVHeads * (kKv8Block * 16);
  int again_n[2] = {0, 0};  // heads whose K, V blocks are written again, listed
  if (any) {
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint32_t set = __ballot_sync(0xffffffffu, lane < kKVHeads && s_top[kv][lane & 7] != 0);
      again_n[kv] = __popc(set);  // (every warp writes the same list)
      if ((set >> lane) & 1) s_list[kv][__popc(set & ((1u << lane) - 1))] = lane;
    }
    __syncthreads();  // (the flags are read before they grow)
    // the old rows' largest magnitudes: (head, row, chunk) over the threads
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const uint4* old = kv ? open_v : open_k;
#pragma unroll 2
      for (int e = tid; e < again_n[kv] * 8 * row; e += kApThreads) {
        const int h = s_list[kv][(e >> 3) / row];
        const size_t at = ((size_t)h * kKv8Block + (e >> 3) % row) * 16 + (e & 7);
        const uint32_t m = absmax4(absmax4(0u, old[at]), old[at + 8]);
        atomicMax(&s_top[kv][h], max(m & 0xFFFFu, m >> 16));
      }
    }
    __syncthreads();
    if (again && k_all) ks = scale_of<kKind>(s_top[0][g]);
    if (again && v_all) vs = scale_of<kKind>(s_top[1][g]);
  }
  if (id >= 0) {  // the new row
    if (!k_all) ks = k_was;
    if (!v_all) vs = v_was;
    const float k_inv = ks > 0.f ? __fdiv_rn(1.f, ks) : 0.f, v_inv = vs > 0.f ? __fdiv_rn(1.f, vs) : 0.f;
    if (lane == 0) {
      if (k_all) p.c.k_scale[id] = ks;
      if (v_all) p.c.v_scale[id] = vs;
    }
    const bool open = row + 1 < kKv8Block;
    uint4* my_k = reinterpret_cast<uint4*>(p.c.open_k) + (head * kKv8Block + row) * 16;
    uint4* my_v = reinterpret_cast<uint4*>(p.c.open_v) + (head * kKv8Block + row) * 16;
    if (lane < 8) {
      uint8_t* dst = static_cast<uint8_t*>(p.c.k_pool) + (size_t)id * kKv8Bytes + row * 64 + 8 * c;
      *reinterpret_cast<uint2*>(dst) = codes8<kKind>(kx[0], k_inv);
      *reinterpret_cast<uint2*>(dst + kKv8Bytes / 2) = codes8<kKind>(kx[1], k_inv);
      if (open) my_k[c] = kx[0], my_k[c + 8] = kx[1];
    } else if (lane < 24) {
      uint8_t* dst = static_cast<uint8_t*>(p.c.v_pool) + (size_t)id * kKv8Bytes + (lane - 8) * 8 * kKv8Block + row;
      const uint2 w = codes8<kKind>(vx, v_inv);
#pragma unroll
      for (int e = 0; e < 8; ++e) dst[e * kKv8Block] = uint8_t((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
      if (open) my_v[lane - 8] = vx;
    }
  }
  if (!any) return;
  // the old rows' codes on the new scales
#pragma unroll 2
  for (int e = tid; e < again_n[0] * 8 * row; e += kApThreads) {
    const int h = s_list[0][(e >> 3) / row], r = (e >> 3) % row, ch = e & 7;
    const float scale = scale_of<kKind>(s_top[0][h]), inv = scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
    const size_t at = ((size_t)h * kKv8Block + r) * 16 + ch;
    uint8_t* dst = static_cast<uint8_t*>(p.c.k_pool) + (size_t)s_id[h] * kKv8Bytes + r * 64 + 8 * ch;
    *reinterpret_cast<uint2*>(dst) = codes8<kKind>(open_k[at], inv);
    *reinterpret_cast<uint2*>(dst + kKv8Bytes / 2) = codes8<kKind>(open_k[at + 8], inv);
  }
  const int quads = (row + 3) / 4;  // four rows of a feature make one word of the feature's 64 bytes
  for (int e = tid; e < again_n[1] * 16 * quads; e += kApThreads) {
    const int h = s_list[1][(e >> 4) / quads], r0 = (e >> 4) % quads * 4, ch = e & 15;
    const float scale = scale_of<kKind>(s_top[1][h]), inv = scale > 0.f ? __fdiv_rn(1.f, scale) : 0.f;
    uint4 x[4];
#pragma unroll
    for (int m = 0; m < 4; ++m)
      x[m] = r0 + m < row ? open_v[((size_t)h * kKv8Block + r0 + m) * 16 + ch] : make_uint4(0, 0, 0, 0);
    uint8_t* dst = static_cast<uint8_t*>(p.c.v_pool) + (size_t)s_id[h] * kKv8Bytes + ch * 8 * kKv8Block + r0;
#pragma unroll
    for (int f = 0; f < 8; ++f, dst += kKv8Block) {
      const uint32_t w = codes4<kKind>(bf16_at(x[0], f), bf16_at(x[1], f), bf16_at(x[2], f), bf16_at(x[3], f), inv);
      if (r0 + 4 <= row) {
        *reinterpret_cast<uint32_t*>(dst) = w;
      } else {
#pragma unroll
        for (int m = 0; m < 3; ++m)
          if (r0 + m < row) dst[m] = uint8_t(w >> (8 * m));
      }
    }
  }
}

}  // namespace grok

using namespace grok;

namespace grok {

grok_status kv8_check(const grok_kv8_cache* c, const char* who) {
  if (!c) return fail(GROK_ERR_INVALID_ARG, "%s: null cache", who);
  if (!c->k_pool || !c->v_pool || !c->k_scale || !c->v_scale || !c->table || !c->open_k || !c->open_v)
    return fail(GROK_ERR_INVALID_ARG, "%s: null pointer in the cache", who);
  if (!aligned16(c->k_pool) || !aligned16(c->v_pool) || !aligned16(c->open_k) || !aligned16(c->open_v) ||
      !aligned16(c->k_scale) || !aligned16(c->v_scale) || !aligned16(c->table))
    return fail(GROK_ERR_INVALID_ARG, "%s: the cache's pointers must be 16-byte aligned", who);
  if (c->kind != GROK_KV8_INT8 && c->kind != GROK_KV8_E4M3)
    return fail(GROK_ERR_INVALID_ARG, "%s: unknown kind %d", who, c->kind);
  if (c->B < 1 || c->B > 65535 || c->max_blocks < 1 || c->max_blocks > kKv8MaxBlocks || c->n_blocks < 1)
    return fail(GROK_ERR_INVALID_ARG, "%s: need 1 <= B <= 65535, 1 <= max_blocks <= %d, n_blocks >= 1 (B=%d "
                "max_blocks=%d n_blocks=%d)", who, kKv8MaxBlocks, c->B, c->max_blocks, c->n_blocks);
  return GROK_OK;
}

}  // namespace grok

extern "C" grok_status grok_kv8_append(const grok_kv8_cache* cache, const grok_bf16* q, const grok_bf16* k,
                                       const grok_bf16* v, const int32_t* start_pos, const int32_t* cache_len,
                                       const int32_t* valid_len, int T, const float* cos_tab, const float* sin_tab,
                                       int tab_positions, grok_bf16* q_rot, int32_t* dev_status, void* stream) {
  grok_status st = kv8_check(cache, "grok_kv8_append");
  if (st != GROK_OK) return st;
  if (!q || !k || !v || !start_pos || !cache_len || !cos_tab || !sin_tab || !q_rot)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_append: null pointer");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_rot) || !aligned16(cos_tab) ||
      !aligned16(sin_tab))
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_append: bf16 tensors and tables must be 16-byte aligned");
  if (q == q_rot) return fail(GROK_ERR_INVALID_ARG, "grok_kv8_append: q_rot may not alias q");
  if (T < 1 || T > GROK_MAX_POSITION || tab_positions < 1 || tab_positions > GROK_MAX_POSITION)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_append: need 1 <= T, tab_positions <= %d (T=%d tab_positions=%d)",
                GROK_MAX_POSITION, T, tab_positions);
  int sms = 0;
  if ((st = device_sm_count(&sms)) != GROK_OK) return st;
  const ApParams p{*cache,
                   reinterpret_cast<const uint4*>(q),
                   reinterpret_cast<const uint4*>(k),
                   reinterpret_cast<const uint4*>(v),
                   reinterpret_cast<uint4*>(q_rot),
                   start_pos,
                   cache_len,
                   valid_len,
                   reinterpret_cast<const float4*>(cos_tab),
                   reinterpret_cast<const float4*>(sin_tab),
                   T,
                   tab_positions,
                   dev_status};
  // T tokens behind up to 63 open rows touch at most (T + 126) / 64 blocks
  const dim3 grid((T + 2 * kKv8Block - 2) / kKv8Block, kKVHeads, cache->B);
  if (T == 1 && cache->B >= kApMany) {
    auto one =
        cache->kind == GROK_KV8_INT8 ? kv8_append_one_kernel<GROK_KV8_INT8> : kv8_append_one_kernel<GROK_KV8_E4M3>;
    one<<<cache->B, kApThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
    return check_launch("kv8_append_one");
  }
  // CTAs with tokens, about: three on an SM at once with six heads, four with three
  const bool few = (long long)cache->B * ((T + kKv8Block - 1) / kKv8Block) * kKVHeads <= 3 * sms;
  auto kernel = cache->kind == GROK_KV8_INT8
                    ? (few ? kv8_append_kernel<GROK_KV8_INT8, kGroup> : kv8_append_kernel<GROK_KV8_INT8, kGroup / 2>)
                    : (few ? kv8_append_kernel<GROK_KV8_E4M3, kGroup> : kv8_append_kernel<GROK_KV8_E4M3, kGroup / 2>);
  kernel<<<grid, kApThreads, 0, static_cast<cudaStream_t>(stream)>>>(p);
  return check_launch("kv8_append");
}
