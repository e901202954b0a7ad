// Attention of many tokens over the 8-bit KV cache.
//
// Code-reading guide ch. 4 §4.5.2-§4.5.4, ch. 6 §6.4.2, over code * scale. A first
// kernel lays the blocks that the call sees out for the tensor cores: K codes
// as bf16 (exact) and V as fp16, rows of a sequence and head in order. The
// attention kernel (prefill.cu, kQ8) multiplies the logits of each 64-key
// step by the block's K scale and the outputs by the head's V scale: a V value is
// rounded once to fp16 on the scale vs / max vs of its block, 2^-11 relative.
//
// Tensor-bound for all but short calls: the copies cost 1 byte read, 2 written
// and 2 read per code. Measured (graph replays, one GB300): 8192 tokens in an empty
// cache 670 us, 1231 TFLOP/s, 0.63 of the library GEMM's rate, of which the copies
// are 12 us; 4 x 256 tokens behind 6144 rows 181 us, 26 of them the copies (52 MB of
// codes read, 105 MB written, 6 TB/s); 128 tokens behind 8192 rows 51 us.
#include "host.cuh"
#include "kv8.cuh"
#include "prefill.cuh"

namespace grok {

constexpr int kUnThreads = 256;

struct UnParams {
  grok_kv8_cache c;
  const int32_t *cache_len, *valid_len;
  int T, rows;         // rows of a sequence's copies
  uint4 *k_copy, *v_copy;  // [B][8][rows][128] bf16, fp16
  float* k_scale;      // [B][8][rows / 64]
  float* o_scale;      // [B][8]
  int32_t* fb_count;   // words that the attention passes expect to be zero: the fallback count and the split's
  int32_t* zero;
  int n_zero;
  int32_t* status;
};

// V values on the copy's common scale: codes up to 127 or 448 times vs / max vs times this stay below 65504.
constexpr float kVTop = 128.f;

// Four int8 or e4m3 codes to bf16 pairs, exactly. int8: the seven low bits b behind 0x43 are 128 + b, the sign bit there
// is 128 or 256, and the difference is the code.
template <int kKind>
__device__ __forceinline__ void kv8_to_bf16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if (kKind == GROK_KV8_INT8) {
    const uint32_t a = __byte_perm(w, 0x43434343u, 0x4140), b = __byte_perm(w, 0x43434343u, 0x4342);
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(lo) : "r"(a & 0xFF7FFF7Fu), "r"(a & 0xFF80FF80u));
    asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(hi) : "r"(b & 0xFF7FFF7Fu), "r"(b & 0xFF80FF80u));
  } else {
    uint32_t x[2];
    kv8_to_half<kKind>(w, x[0], x[1]);
    const float2 a = __half22float2(reinterpret_cast<const __half2&>(x[0]));
    const float2 b = __half22float2(reinterpret_cast<const __half2&>(x[1]));
    lo = pack_bf16x2(a.x, a.y);
    hi = pack_bf16x2(b.x, b.y);
  }
}

__device__ __forceinline__ uint32_t scale_half2(uint32_t x, float f) {
  const float2 a = __half22float2(reinterpret_cast<const __half2&>(x));
  return pack_f16x2(a.x * f, a.y * f);
}

// Grid (parts, KV head, sequence): a CTA takes every parts-th block of its head.
template <int kKind>
__global__ void __launch_bounds__(kUnThreads) kv8_unpack_kernel(const UnParams p) {
  __shared__ float s_top[kUnThreads / 32];
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int g = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  if (blockIdx.x == 0 && g == 0 && b == 0) {
    if (tid == 0) *p.fb_count = 0;
    for (int i = tid; i < p.n_zero; i += kUnThreads) p.zero[i] = 0;
  }
  const int s = __ldg(p.cache_len + b), n = p.valid_len ? __ldg(p.valid_len + b) : p.T;
  if (s < 0 || n < 1 || n > p.T || (long long)s + n > (long long)p.c.max_blocks * kKv8Block) return;  // reported later
  const int len = s + n, blocks = (len + kKv8Block - 1) / kKv8Block;
  const size_t head = (size_t)b * kKVHeads + g;
  const int32_t* table = p.c.table + head * p.c.max_blocks;
  // The head's scales: the largest V scale, and every block's K scale. A block whose values are not finite shows it
  // in the logits (a NaN in the copy of V would reach rows that do not see the block).
  float top = 0.f;
  for (int i = tid; i < blocks; i += kUnThreads) {
    const int id = max(0, kv8_block_id(table, i, p.c.n_blocks, p.status));
    const float vs = __ldg(p.c.v_scale + id);
    if (vs == vs) top = fmaxf(top, vs);
    if (blockIdx.x == 0) p.k_scale[head * (p.rows / kKv8Block) + i] = vs == vs ? __ldg(p.c.k_scale + id) : vs;
  }
#pragma unroll
  for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  if ((tid & 31) == 0) s_top[tid >> 5] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kUnThreads / 32; ++w) top = fmaxf(top, s_top[w]);
  if (blockIdx.x == 0 && tid == 0) p.o_scale[head] = top / kVTop;
  const float per = top > 0.f ? kVTop / top : 0.f;

  // Rows up to the next multiple of 128: those behind the last are zeros (in V they meet zero weights).
  const int pad = (blocks + 1) / 2 * 2;
  uint4* k_out = p.k_copy + head * p.rows * 16;
  uint4* v_out = p.v_copy + head * p.rows * 16;
  const int q = tid & 15, c = tid >> 4;
  for (int i = blockIdx.x; i < pad; i += gridDim.x) {
    const int left = min(kKv8Block, len - i * kKv8Block);  // rows of this block (negative in the padding)
    const int id = left > 0 ? max(0, kv8_block_id(table, i, p.c.n_blocks, nullptr)) : 0;
    const uint8_t* k_src = static_cast<const uint8_t*>(p.c.k_pool) + (size_t)id * kKv8Bytes;
    const uint8_t* v_src = static_cast<const uint8_t*>(p.c.v_pool) + (size_t)id * kKv8Bytes;
    float f = left > 0 ? __ldg(p.c.v_scale + id) : 0.f;
    // K: 8 codes of a row of one half, four times; V: four rows (4 q ..) of eight features (8 c ..)
    uint2 kw[4];
    uint32_t vw[8];
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int e = tid + m * kUnThreads, row = (e >> 3) & 63;
      kw[m] = row < left ? __ldg(reinterpret_cast<const uint2*>(k_src + 8 * e)) : make_uint2(0, 0);
    }
#pragma unroll
    for (int d = 0; d < 8; ++d)
      vw[d] = left > 4 * q ? __ldg(reinterpret_cast<const uint32_t*>(v_src + (8 * c + d) * 64 + 4 * q)) : 0u;
    f = f == f ? f * per : 0.f;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const int e = tid + m * kUnThreads, row = (e >> 3) & 63;
      uint4 x;
      kv8_to_bf16<kKind>(kw[m].x, x.x, x.y);
      kv8_to_bf16<kKind>(kw[m].y, x.z, x.w);
      k_out[(size_t)(i * kKv8Block + row) * 16 + (e >> 9) * 8 + (e & 7)] = x;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {  // turned in registers
      uint4 x = make_uint4(0, 0, 0, 0);
      if (4 * q + r < left) {
        uint32_t a, z;
        const uint32_t sel = r | (r + 4) << 4;
        const uint32_t w0 = __byte_perm(__byte_perm(vw[0], vw[1], sel), __byte_perm(vw[2], vw[3], sel), 0x5410);
        const uint32_t w1 = __byte_perm(__byte_perm(vw[4], vw[5], sel), __byte_perm(vw[6], vw[7], sel), 0x5410);
        kv8_to_half<kKind>(w0, a, z);
        x.x = scale_half2(a, f), x.y = scale_half2(z, f);
        kv8_to_half<kKind>(w1, a, z);
        x.z = scale_half2(a, f), x.w = scale_half2(z, f);
      }
      v_out[(size_t)(i * kKv8Block + 4 * q + r) * 16 + c] = x;
    }
  }
}

// The fallback pass multiplies bf16: when an item is listed, the copy of V is rounded to bf16 in its place, 128 rows
// of a head at a time, up to the rows that the copies have.
__global__ void __launch_bounds__(256) kv8_v_to_bf16_kernel(const UnParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the fp16 passes, which list the items
  if (*p.fb_count == 0) return;
  const int tiles = p.rows / kPfKeys;
  const long long n = (long long)p.c.B * kKVHeads * tiles;
  for (long long e = blockIdx.x; e < n; e += gridDim.x) {
    const long long head = e / tiles;
    const int tile = int(e % tiles), b = int(head / kKVHeads);
    const int s = p.cache_len[b], valid = p.valid_len ? p.valid_len[b] : p.T;
    if (s < 0 || valid < 1 || valid > p.T || (long long)s + valid > (long long)p.c.max_blocks * kKv8Block) continue;
    if (tile * kPfKeys >= s + valid) continue;
    uint4* v = p.v_copy + ((size_t)head * p.rows + (size_t)tile * kPfKeys) * 16;
#pragma unroll
    for (int m = 0; m < kPfKeys * 16 / 256; ++m) {
      const int i = m * 256 + threadIdx.x;
      uint4 x = v[i];
      uint32_t* w = reinterpret_cast<uint32_t*>(&x);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float2 a = __half22float2(reinterpret_cast<const __half2&>(w[q]));
        w[q] = pack_bf16x2(a.x, a.y);
      }
      v[i] = x;
    }
  }
}

}  // namespace grok

using namespace grok;

namespace {

size_t up256(size_t n) { return (n + 255) & ~size_t(255); }

// Calls of up to this many tokens run on the codes (kv8_decode.cu, four tokens to a pass): no copies of the cache, and
// the split over the key range that single tokens have. Above, the copies cost less than the passes. Measured, us, codes
// against copies:
//   1 sequence behind 16000 rows: 4 tokens 21 against 78, 32 66 against 78, 48 85 against 78
//   8 behind 8000: 4 41 against 256, 32 226 against 257, 48 326 against 257
//   32 behind 4000: 16 239 against 518; 256 behind 1000: 16 658 against 1024; 64 behind 100: 16 62 against 68, 20 82
//   against 68; 32 behind 300: 16 43 against 74, 32 88 against 80
//   small caches of one or two sequences, where the copies' four launches are most of the time: 1 behind 300, 4 10
//   against 17, 96 15 against 19, 128 20 against 20; 1 behind 2000, 96 34 against 35; 2 behind 1000, 48 23 against 30
//   caches of one key tile, which need two launches: 8 sequences behind 20 rows, 12 12 against 14, 20 15 against 14.5;
//   1 behind 20, 4 10.2 against 9.1
int few_tokens(int B, int max_blocks) {
  if (max_blocks * kKv8Block <= kPfKeys) return 12;
  if (B <= 2 && B * max_blocks <= 36) return 96 / B;
  return B <= 8 ? 32 : 16;
}

// Groups of tokens in such a call: at least as many as B sequences or fewer with any capacity have (96 / 4 for one or
// two, 8 each for up to eight, 4 each for more), so that a workspace for a cache serves every smaller one too.
int few_groups(int B) { return std::max({24, 8 * std::min(B, 8), 4 * B}); }

// Workspace: fallback count and list, K scales, output factors, the copies of K and V, the split's area.
struct Layout {
  int rows;
  size_t k_scale, o_scale, k_copy, v_copy, split, bytes;
};

Layout layout(int B, int max_blocks, int sms) {
  Layout w;
  w.rows = (max_blocks + 1) / 2 * 2 * kKv8Block;
  w.k_scale = up256((1 + size_t(ws_fb_cap(B, w.rows))) * sizeof(int32_t));
  w.o_scale = w.k_scale + up256(size_t(B) * kKVHeads * (w.rows / kKv8Block) * sizeof(float));
  w.k_copy = w.o_scale + up256(size_t(B) * kKVHeads * sizeof(float));
  const size_t copy = size_t(B) * w.rows * kKVHeads * kD * 2;
  w.v_copy = w.k_copy + copy;
  w.split = w.v_copy + copy;
  w.bytes = w.split + (split_allowed(w.rows) ? split_area_bytes(sms) : 0);
  w.bytes = std::max(w.bytes, kv8_decode_bytes(few_groups(B), 1, max_blocks, false, sms));
  return w;
}

grok_status sizes_ok(int B, int max_blocks, const char* who) {
  if (B < 1 || B > 65535 || max_blocks < 1 || max_blocks > kKv8MaxBlocks || (long long)B * max_blocks > (1 << 21))
    return fail(GROK_ERR_INVALID_ARG, "%s: need 1 <= B <= 65535, 1 <= max_blocks <= %d, B * max_blocks <= %d", who,
                kKv8MaxBlocks, 1 << 21);
  return GROK_OK;
}

}  // namespace

extern "C" grok_status grok_kv8_prefill_workspace(int B, int max_blocks, size_t* bytes) {
  if (!bytes) return fail(GROK_ERR_INVALID_ARG, "grok_kv8_prefill_workspace: null pointer");
  grok_status st = sizes_ok(B, max_blocks, "grok_kv8_prefill_workspace");
  if (st != GROK_OK) return st;
  int sms = 0;
  if ((st = device_sm_count(&sms)) != GROK_OK) return st;
  *bytes = layout(B, max_blocks, sms).bytes;
  return GROK_OK;
}

extern "C" grok_status grok_kv8_prefill(const grok_kv8_cache* cache, const grok_bf16* q_rot, const int32_t* cache_len,
                                        const int32_t* valid_len, int T, grok_bf16* out, void* workspace,
                                        size_t workspace_bytes, int32_t* dev_status, void* stream) {
  grok_status st = kv8_check(cache, "grok_kv8_prefill");
  if (st != GROK_OK) return st;
  if (!q_rot || !cache_len || !out || !workspace)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_prefill: null pointer");
  if (!aligned16(q_rot) || !aligned16(out))
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_prefill: bf16 tensors must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_prefill: workspace must be 256-byte aligned");
  if (q_rot == out) return fail(GROK_ERR_INVALID_ARG, "grok_kv8_prefill: out may not alias q_rot");
  const int B = cache->B, max_blocks = cache->max_blocks;
  if ((st = sizes_ok(B, max_blocks, "grok_kv8_prefill")) != GROK_OK) return st;
  if (T < 1 || T > max_blocks * kKv8Block)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_prefill: need 1 <= T <= max_blocks * %d (T=%d max_blocks=%d)", kKv8Block,
                T, max_blocks);
  int sms = 0;
  if ((st = device_sm_count(&sms)) != GROK_OK) return st;
  const Layout w = layout(B, max_blocks, sms);
  if (workspace_bytes < w.bytes)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_prefill: workspace of %zu bytes is smaller than the %zu needed",
                workspace_bytes, w.bytes);
  if (T <= few_tokens(B, max_blocks))
    return kv8_decode_run(*cache, q_rot, cache_len, valid_len, T, static_cast<char*>(workspace), out, nullptr, nullptr, sms,
                          dev_status, static_cast<cudaStream_t>(stream));
  char* ws = static_cast<char*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int n_items = prefill_items(B, T);
  int n_whole, n_parts;
  split_plan(n_items, sms, split_allowed(w.rows), kPfMaxPartsQ8, n_whole, n_parts);
  const int n_split = n_items - n_whole;

  int32_t* fb_count = reinterpret_cast<int32_t*>(ws);
  const UnParams u{*cache,
                   cache_len,
                   valid_len,
                   T,
                   w.rows,
                   reinterpret_cast<uint4*>(ws + w.k_copy),
                   reinterpret_cast<uint4*>(ws + w.v_copy),
                   reinterpret_cast<float*>(ws + w.k_scale),
                   reinterpret_cast<float*>(ws + w.o_scale),
                   fb_count,
                   reinterpret_cast<int32_t*>(ws + w.split),
                   2 * n_split,
                   dev_status};
  const int heads = B * kKVHeads;
  const int parts = std::max(1, std::min((max_blocks + 1) / 2 * 2, (sms * 6 + heads - 1) / heads));
  auto unpack = cache->kind == GROK_KV8_INT8 ? kv8_unpack_kernel<GROK_KV8_INT8> : kv8_unpack_kernel<GROK_KV8_E4M3>;
  unpack<<<dim3(parts, kKVHeads, B), kUnThreads, 0, s>>>(u);
  if ((st = check_launch("kv8_unpack")) != GROK_OK) return st;

  const Q8Prefill a{q_rot,
                    out,
                    u.k_copy,
                    u.v_copy,
                    w.rows,
                    u.k_scale,
                    u.o_scale,
                    cache_len,
                    valid_len,
                    B,
                    T,
                    max_blocks * kKv8Block,
                    sms,
                    fb_count,
                    fb_count + 1,
                    ws_fb_cap(B, w.rows),
                    n_whole,
                    n_parts,
                    ws + w.split,
                    dev_status};
  if ((st = prefill_q8_passes(a, false, s)) != GROK_OK) return st;
  // No weight of a single key tile outgrows the reference that the tile itself sets.
  if (w.rows <= kPfKeys) return GROK_OK;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(sms);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kv8_v_to_bf16_kernel, u);
  if (e != cudaSuccess) return fail(cuda_status(e), "kv8_v_to_bf16 launch: %s", cudaGetErrorString(e));
  if ((st = check_launch("kv8_v_to_bf16")) != GROK_OK) return st;
  return prefill_q8_passes(a, true, s);
}
