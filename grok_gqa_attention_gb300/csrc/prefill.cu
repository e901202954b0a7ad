// K2: prefill attention over the bf16 cache: the fp16 mode's pre-pass and the
// entry points. The kernel, and what it follows of the code-reading guide (ch. 4
// §4.5.2-§4.5.4, ch. 6 §6.4.2), is in prefill_kernel.cuh.
#include "prefill_kernel.cuh"

namespace grok {

// ----------------------------------------------------------------------------
// fp16 mode pre-pass: the fp16 copy of V. For sequence b with a valid start s,
// rows [0, s + T) of the cache (contiguous, or through the block table) are
// rounded to nearest fp16 and rows [s + T, round_up(s + T, 128)) are zeroed, so
// every key tile the fp16 pass reads is finite. A finite |v| >= 65520 (beyond
// fp16) sets v_flags[b]: the fp16 pass then hands all of that sequence's items
// to the fallback pass.
__global__ void __launch_bounds__(256) v_to_half_kernel(const uint4* __restrict__ cache_v, PageMap pm,
                                                        const int32_t* start_pos, int T, int Tmax, int vh_rows,
                                                        int from_start, uint4* __restrict__ vh, int32_t* v_flags,
                                                        int32_t* zero, int n_zero, int32_t* status) {
  // the key-range split's per-item counters start at zero
  if (blockIdx.y == 0)
    for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < n_zero; i += gridDim.x * blockDim.x) zero[i] = 0;
  const int b = blockIdx.y;
  const int s = __ldg(start_pos + b);
  if (s < 0 || (long long)s + T > Tmax) return;  // the attention passes skip this sequence
  const int rows = s + T, rows_pad = min(vh_rows, (rows + kPfKeys - 1) / kPfKeys * kPfKeys);
  const int first = from_start ? s : 0;  // rows below `first` are already converted (reuse)
  constexpr int kChunks = kKVHeads * kD / 8;  // 16-byte chunks (8 values) per row
  bool over = false;
  for (long long e = (long long)first * kChunks + (long long)blockIdx.x * blockDim.x + threadIdx.x;
       e < (long long)rows_pad * kChunks; e += (long long)gridDim.x * blockDim.x) {
    const int row = int(e / kChunks), ch = int(e % kChunks);
    uint4 out = make_uint4(0, 0, 0, 0);
    if (row < rows) {
      int src_row, src_b;
      kv_coord(pm, b, row, src_row, src_b, status);  // (row, b) contiguous, (page row, 0) paged
      const size_t rows_per_seq = pm.table ? size_t(0) : size_t(Tmax);
      const uint4 in = __ldg(cache_v + ((size_t)src_b * rows_per_seq + src_row) * kChunks + ch);
      const uint32_t w[4] = {in.x, in.y, in.z, in.w};
      uint32_t o[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float a = bf16lo_to_f32(w[q]), c = bf16hi_to_f32(w[q]);
        over |= (fabsf(a) >= 65520.f && fabsf(a) != INFINITY) || (fabsf(c) >= 65520.f && fabsf(c) != INFINITY);
        o[q] = pack_f16x2(a, c);
      }
      out = make_uint4(o[0], o[1], o[2], o[3]);
    }
    vh[((size_t)b * vh_rows + row) * kChunks + ch] = out;
  }
  if (__any_sync(0xffffffffu, over) && (threadIdx.x & 31) == 0) atomicOr(v_flags + b, 1);
}

}  // namespace grok

using namespace grok;

// Extra inputs of the fp16 mode and of the fallback pass.
struct PfExtra {
  bool f16 = false;                 // fp16 mode: v_half holds the fp16 copy of V, [B][vh_rows][8][128]
  const void* v_half = nullptr;
  int vh_rows = 0;
  const int32_t* v_flags = nullptr;
  int32_t* fb_count = nullptr;      // fallback list (written by the fp16 pass, read by the fallback pass)
  int32_t* fb_list = nullptr;
  int fb_cap = 0;
  bool fallback = false;            // bf16 mode over the listed items only, launched as a dependent
  int n_units = -1;                 // units of this pass (-1: every item, whole)
  bool split = false;               // fp16 split pass: items [item_base, ...) shared among n_parts units each
  int item_base = 0, n_parts = 1;
  float4* part_o = nullptr;
  float2* part_lm = nullptr;
  int32_t* part_cnt = nullptr;
};

static grok_status prefill_launch(const grok_bf16* q_rot, const grok_bf16* k_src, const grok_bf16* v_src,
                                  uint64_t kv_rows, uint64_t kv_seqs, PageMap pm, const int32_t* start_pos,
                                  const int32_t* valid_len, int B, int T, int Tmax, grok_bf16* out, int32_t* dev_status,
                                  void* stream, const PfExtra& ex = PfExtra()) {
  int sms = 0;
  grok_status st = device_sm_count(&sms);
  if (st != GROK_OK) return st;

  CUtensorMap tq, tk, tv, to;
  const uint32_t box[4] = {64, 1, 128, 1};
  {
    const uint64_t dims[4] = {kD, kQHeads, uint64_t(T), uint64_t(B)};
    const uint64_t strides[3] = {kD * 2, uint64_t(kQHeads) * kD * 2, uint64_t(T) * kQHeads * kD * 2};
    if ((st = encode_tmap_bf16_4d(&tq, q_rot, dims, strides, box)) != GROK_OK) return st;
    const uint32_t obox[4] = {64, 1, 32, 1};  // one epilogue warp's 32 rows x 64 features
    if ((st = encode_tmap_bf16_4d(&to, out, dims, strides, obox)) != GROK_OK) return st;
  }
  {
    const uint64_t dims[4] = {kD, kKVHeads, kv_rows, kv_seqs};
    const uint64_t strides[3] = {kD * 2, uint64_t(kKVHeads) * kD * 2, kv_rows * kKVHeads * kD * 2};
    if ((st = encode_tmap_bf16_4d(&tk, k_src, dims, strides, box)) != GROK_OK) return st;
    if (ex.f16) {
      const uint64_t hdims[4] = {kD, kKVHeads, uint64_t(ex.vh_rows), uint64_t(B)};
      const uint64_t hstrides[3] = {kD * 2, uint64_t(kKVHeads) * kD * 2, uint64_t(ex.vh_rows) * kKVHeads * kD * 2};
      if ((st = encode_tmap_f16_4d(&tv, ex.v_half, hdims, hstrides, box)) != GROK_OK) return st;
    } else if ((st = encode_tmap_bf16_4d(&tv, v_src, dims, strides, box)) != GROK_OK) {
      return st;
    }
  }
  PfParams prm;
  prm.B = B;
  prm.T = T;
  prm.Tmax = Tmax;
  prm.pm = pm;
  prm.n_qt = (T + kPfRows - 1) / kPfRows;
  prm.n_items = prm.n_qt * B * kKVHeads * 3;
  prm.start_pos = start_pos;
  prm.valid_len = valid_len;
  prm.status = dev_status;
  prm.v_flags = ex.v_flags;
  prm.fb_count = ex.fb_count;
  prm.fb_list = ex.fb_list;
  prm.fb_cap = ex.fb_cap;
  prm.item_list = ex.fallback ? ex.fb_list : nullptr;
  prm.item_count = ex.fallback ? ex.fb_count : nullptr;
  prm.n_units = ex.n_units >= 0 ? ex.n_units : prm.n_items;
  prm.item_base = ex.split ? ex.item_base : 0;
  prm.n_parts = ex.split ? ex.n_parts : 1;
  prm.part_o = ex.part_o;
  prm.part_lm = ex.part_lm;
  prm.part_cnt = ex.part_cnt;

  static bool attr_set[kMaxDevices][4] = {};  // per device and kernel instance; idempotent
  int dev = 0;
  grok_status dst = device_index(&dev);
  if (dst != GROK_OK) return dst;
  const int mode = ex.split ? 3 : ex.f16 ? 1 : ex.fallback ? 2 : 0;
  auto kernel = mode == 3   ? prefill_kernel<true, false, true>
                : mode == 1 ? prefill_kernel<true, false, false>
                : mode == 2 ? prefill_kernel<false, true, false>
                            : prefill_kernel<false, false, false>;
  if (!attr_set[dev][mode]) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPfSmem);
    if (e != cudaSuccess) return fail(cuda_status(e), "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
    attr_set[dev][mode] = true;
  }
  // The fallback pass does not know how many items it has (the list is on the
  // device), so it takes one CTA per SM; it is a programmatic dependent of the
  // fp16 pass, so its launch overlaps that pass's tail, and it waits for the
  // whole fp16 grid (griddepcontrol.wait) before reading the list.
  const int grid = ex.fallback ? sms : (prm.n_units < sms ? prm.n_units : sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kPfThreads);
  cfg.dynamicSmemBytes = kPfSmem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = ex.fallback ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, tq, tk, tv, to, prm);
  if (e != cudaSuccess) return fail(cuda_status(e), "prefill launch: %s", cudaGetErrorString(e));
  return check_launch("prefill");
}

extern "C" grok_status grok_attn_prefill(const grok_bf16* q_rot, const grok_bf16* cache_k,
                                         const grok_bf16* cache_v, const int32_t* start_pos,
                                         const int32_t* valid_len, int B, int T, int Tmax, grok_bf16* out,
                                         int32_t* dev_status, void* stream) {
  if (!q_rot || !cache_k || !cache_v || !start_pos || !out)
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill: null pointer");
  if (!aligned16(q_rot) || !aligned16(cache_k) || !aligned16(cache_v) || !aligned16(out))
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill: bf16 tensors must be 16-byte aligned");
  if (B < 1 || T < 1 || Tmax < 1 || T > Tmax || Tmax > GROK_MAX_POSITION)
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill: need B >= 1, 1 <= T <= Tmax <= %d (B=%d T=%d Tmax=%d)",
                GROK_MAX_POSITION, B, T, Tmax);
  return prefill_launch(q_rot, cache_k, cache_v, uint64_t(Tmax), uint64_t(B), PageMap{nullptr, 0, 0}, start_pos,
                        valid_len, B, T, Tmax, out, dev_status, stream);
}

extern "C" grok_status grok_attn_prefill_paged(const grok_bf16* q_rot, const grok_bf16* k_pool,
                                               const grok_bf16* v_pool, int n_pages, const int32_t* block_table,
                                               int max_pages, const int32_t* start_pos, const int32_t* valid_len,
                                               int B, int T, grok_bf16* out, int32_t* dev_status, void* stream) {
  if (!q_rot || !k_pool || !v_pool || !block_table || !start_pos || !out)
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill_paged: null pointer");
  if (!aligned16(q_rot) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill_paged: bf16 tensors must be 16-byte aligned");
  const long long Tmax = (long long)max_pages * GROK_PAGE_TOKENS;
  if (B < 1 || T < 1 || n_pages < 1 || max_pages < 1 || T > Tmax || Tmax > GROK_MAX_POSITION ||
      (long long)n_pages * GROK_PAGE_TOKENS > (1LL << 31))
    return fail(GROK_ERR_INVALID_ARG,
                "grok_attn_prefill_paged: need B, T, n_pages, max_pages >= 1, T <= max_pages * %d <= %d "
                "(B=%d T=%d max_pages=%d n_pages=%d)",
                GROK_PAGE_TOKENS, GROK_MAX_POSITION, B, T, max_pages, n_pages);
  return prefill_launch(q_rot, k_pool, v_pool, uint64_t(n_pages) * GROK_PAGE_TOKENS, 1,
                        PageMap{block_table, max_pages, n_pages}, start_pos, valid_len, B, T, int(Tmax), out,
                        dev_status, stream);
}

// ----------------------------------------------------------------------------
// Prefill with fp16 softmax weights (grok_attn_prefill_ws). Workspace layout:
//   int32 v_flags[B], fb_count, fb_list[fb_cap]  (padded to 256 bytes)
//   fp16 V copy [B][round_up(Tmax, 128)][8][128]
//   optional, for the key-range split (at most one unit per SM):
//     int32 part_cnt[sms][2] (padded to 256 bytes), float2 part_lm[sms][2][128],
//     float4 part_o[sms][2][2][16][128]
static int ws_vh_rows(int Tmax) { return (Tmax + kPfKeys - 1) / kPfKeys * kPfKeys; }
static size_t ws_header_bytes(int B, int Tmax) {
  return ((size_t(B) + 1 + size_t(ws_fb_cap(B, Tmax))) * sizeof(int32_t) + 255) & ~size_t(255);
}

// The part every call needs: the header and the fp16 V copy.
static size_t ws_base_bytes(int B, int Tmax) {
  return ws_header_bytes(B, Tmax) + size_t(B) * ws_vh_rows(Tmax) * kKVHeads * kD * 2;
}

extern "C" grok_status grok_attn_prefill_workspace_min(int B, int Tmax, size_t* bytes) {
  if (!bytes) return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill_workspace_min: null pointer");
  if (B < 1 || Tmax < 1 || Tmax > GROK_MAX_POSITION || (long long)B * ws_vh_rows(Tmax) > (1LL << 31))
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill_workspace_min: need B >= 1, 1 <= Tmax <= %d",
                GROK_MAX_POSITION);
  *bytes = ws_base_bytes(B, Tmax);
  return GROK_OK;
}

extern "C" grok_status grok_attn_prefill_workspace(int B, int Tmax, size_t* bytes) {
  grok_status st = grok_attn_prefill_workspace_min(B, Tmax, bytes);
  if (st != GROK_OK || !split_allowed(Tmax)) return st;
  int sms = 0;
  if ((st = device_sm_count(&sms)) != GROK_OK) return st;
  *bytes += split_area_bytes(sms);
  return GROK_OK;
}

// The fp16-weight prefill over a contiguous cache or a paged pool (pm), its
// arguments already checked: V pre-pass, whole items, the split pass, then the
// bf16 fallback pass over the listed items.
static grok_status prefill_ws_run(const grok_bf16* q_rot, const grok_bf16* k_src, const grok_bf16* v_src,
                                  uint64_t kv_rows, uint64_t kv_seqs, PageMap pm, const int32_t* start_pos,
                                  const int32_t* valid_len, int B, int T, int Tmax, grok_bf16* out, void* workspace,
                                  size_t workspace_bytes, int reuse_v_half, int32_t* dev_status, void* stream,
                                  const char* what) {
  size_t need = 0;
  grok_status st = grok_attn_prefill_workspace_min(B, Tmax, &need);
  if (st != GROK_OK) return st;
  if (workspace_bytes < need)
    return fail(GROK_ERR_INVALID_ARG, "%s: workspace of %zu bytes is smaller than the %zu needed", what,
                workspace_bytes, need);
  int sms = 0;
  if ((st = device_sm_count(&sms)) != GROK_OK) return st;
  // items [0, n_whole) run whole; the rest, if the split applies, n_parts units each
  const int n_items = prefill_items(B, T);
  int n_whole, n_parts;
  split_plan(n_items, sms, split_allowed(Tmax) && workspace_bytes >= need + split_area_bytes(sms), n_whole, n_parts);
  const int n_split = n_items - n_whole;
  char* split_area = static_cast<char*>(workspace) + need;
  const int vh_rows = ws_vh_rows(Tmax);
  int32_t* v_flags = static_cast<int32_t*>(workspace);
  int32_t* fb_count = v_flags + B;
  int32_t* fb_list = fb_count + 1;
  void* vh = static_cast<char*>(workspace) + ws_header_bytes(B, Tmax);
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  // the list count, and unless the copy is reused the overflow flags (reused: they persist)
  cudaError_t e = reuse_v_half ? cudaMemsetAsync(fb_count, 0, sizeof(int32_t), s)
                               : cudaMemsetAsync(v_flags, 0, (size_t(B) + 1) * sizeof(int32_t), s);
  if (e != cudaSuccess) return fail(cuda_status(e), "cudaMemsetAsync: %s", cudaGetErrorString(e));
  {
    const long long per_seq = (long long)(reuse_v_half ? ((T + 2 * kPfKeys - 1) / kPfKeys * kPfKeys) : vh_rows) *
                              (kKVHeads * kD / 8);
    long long bx = (per_seq + 255) / 256;
    const long long cap = ((long long)sms * 8 + B - 1) / B;  // about 8 blocks per SM in all
    if (bx > cap) bx = cap;
    if (bx < 1) bx = 1;
    v_to_half_kernel<<<dim3(unsigned(bx), unsigned(B)), 256, 0, s>>>(
        reinterpret_cast<const uint4*>(v_src), pm, start_pos, T, Tmax, vh_rows, reuse_v_half ? 1 : 0,
        static_cast<uint4*>(vh), v_flags, reinterpret_cast<int32_t*>(split_area), 2 * n_split, dev_status);
    if ((st = check_launch("v_to_half")) != GROK_OK) return st;
  }
  PfExtra ex;
  ex.f16 = true;
  ex.v_half = vh;
  ex.vh_rows = vh_rows;
  ex.v_flags = v_flags;
  ex.fb_count = fb_count;
  ex.fb_list = fb_list;
  ex.fb_cap = ws_fb_cap(B, Tmax);
  if (n_whole > 0) {
    ex.n_units = n_whole;
    if ((st = prefill_launch(q_rot, k_src, v_src, kv_rows, kv_seqs, pm, start_pos,
                             valid_len, B, T, Tmax, out, dev_status, stream, ex)) != GROK_OK)
      return st;
  }
  if (n_split > 0) {
    ex.split = true;
    ex.item_base = n_whole;
    ex.n_parts = n_parts;
    ex.n_units = n_split * n_parts;
    ex.part_cnt = reinterpret_cast<int32_t*>(split_area);
    ex.part_lm = reinterpret_cast<float2*>(split_area + split_cnt_bytes(sms));
    ex.part_o = reinterpret_cast<float4*>(split_area + split_cnt_bytes(sms) + split_lm_bytes(sms));
    if ((st = prefill_launch(q_rot, k_src, v_src, kv_rows, kv_seqs, pm, start_pos,
                             valid_len, B, T, Tmax, out, dev_status, stream, ex)) != GROK_OK)
      return st;
  }
  ex.split = false;
  ex.n_units = -1;
  ex.f16 = false;
  ex.fallback = true;
  return prefill_launch(q_rot, k_src, v_src, kv_rows, kv_seqs, pm, start_pos,
                        valid_len, B, T, Tmax, out, dev_status, stream, ex);
}


extern "C" grok_status grok_attn_prefill_ws(const grok_bf16* q_rot, const grok_bf16* cache_k,
                                            const grok_bf16* cache_v, const int32_t* start_pos,
                                            const int32_t* valid_len, int B, int T, int Tmax, grok_bf16* out,
                                            void* workspace, size_t workspace_bytes, int reuse_v_half,
                                            int32_t* dev_status, void* stream) {
  if (!q_rot || !cache_k || !cache_v || !start_pos || !out || !workspace)
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill_ws: null pointer");
  if (!aligned16(q_rot) || !aligned16(cache_k) || !aligned16(cache_v) || !aligned16(out))
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill_ws: bf16 tensors must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill_ws: workspace must be 256-byte aligned");
  if (B < 1 || T < 1 || Tmax < 1 || T > Tmax || Tmax > GROK_MAX_POSITION)
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill_ws: need B >= 1, 1 <= T <= Tmax <= %d (B=%d T=%d Tmax=%d)",
                GROK_MAX_POSITION, B, T, Tmax);
  return prefill_ws_run(q_rot, cache_k, cache_v, uint64_t(Tmax), uint64_t(B), PageMap{nullptr, 0, 0}, start_pos,
                        valid_len, B, T, Tmax, out, workspace, workspace_bytes, reuse_v_half, dev_status, stream,
                        "grok_attn_prefill_ws");
}

extern "C" grok_status grok_attn_prefill_ws_paged(const grok_bf16* q_rot, const grok_bf16* k_pool,
                                                  const grok_bf16* v_pool, int n_pages, const int32_t* block_table,
                                                  int max_pages, const int32_t* start_pos, const int32_t* valid_len,
                                                  int B, int T, grok_bf16* out, void* workspace,
                                                  size_t workspace_bytes, int reuse_v_half, int32_t* dev_status,
                                                  void* stream) {
  if (!q_rot || !k_pool || !v_pool || !block_table || !start_pos || !out || !workspace)
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill_ws_paged: null pointer");
  if (!aligned16(q_rot) || !aligned16(k_pool) || !aligned16(v_pool) || !aligned16(out))
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill_ws_paged: bf16 tensors must be 16-byte aligned");
  if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return fail(GROK_ERR_INVALID_ARG, "grok_attn_prefill_ws_paged: workspace must be 256-byte aligned");
  const long long Tmax = (long long)max_pages * GROK_PAGE_TOKENS;
  if (B < 1 || T < 1 || n_pages < 1 || max_pages < 1 || T > Tmax || Tmax > GROK_MAX_POSITION ||
      (long long)n_pages * GROK_PAGE_TOKENS > (1LL << 31))
    return fail(GROK_ERR_INVALID_ARG,
                "grok_attn_prefill_ws_paged: need B, T, n_pages, max_pages >= 1, T <= max_pages * %d <= %d "
                "(B=%d T=%d max_pages=%d n_pages=%d)",
                GROK_PAGE_TOKENS, GROK_MAX_POSITION, B, T, max_pages, n_pages);
  return prefill_ws_run(q_rot, k_pool, v_pool, uint64_t(n_pages) * GROK_PAGE_TOKENS, 1,
                        PageMap{block_table, max_pages, n_pages}, start_pos, valid_len, B, T, int(Tmax), out,
                        workspace, workspace_bytes, reuse_v_half, dev_status, stream, "grok_attn_prefill_ws_paged");
}
