// Host side of the prefill passes that the bf16 cache's and the 8-bit cache's
// entry points share: work items, the key-range split, the fallback list, and the
// attention passes over copies of an 8-bit cache.
#pragma once

#include <algorithm>

#include "host.cuh"

namespace grok {

constexpr int kPfRows = 128;   // query rows per tile (MMA M)
constexpr int kPfKeys = 128;   // keys per K/V tile (MMA N for Q K^T, K for P V)
constexpr int kPfMaxParts = 4;       // key-range split: most units one item's key tiles are shared among
constexpr int kPfMaxPartsQ8 = 8;     // the same over an 8-bit cache (24 items, 8192 rows behind: 6 parts, not 4)
constexpr int kPfMinPartTiles = 8;   // key-range split: fewest key tiles per unit

inline int prefill_items(int B, int T) { return B * ((T + kPfRows - 1) / kPfRows) * GROK_N_KV_HEADS * 3; }

// The key-range split. With fewer than two work items per SM, the items left
// for the ragged last round (all of them when there are fewer items than SMs)
// would hold their SMs while the rest idle: 192 equal items of a chunk over a
// long cache on 152 SMs keep 40 SMs for two items. Those items are instead
// shared among P = min(4, SMs / items) units each, run by a second pass, and
// combined by each item's last unit to finish (at most one unit per SM, so the
// partial outputs take at most SMs x 130 KB). Only caches of 16 key tiles or
// more qualify, since a unit holds at least 8 tiles.
inline bool split_allowed(int Tmax) { return (Tmax + kPfKeys - 1) / kPfKeys >= 2 * kPfMinPartTiles; }
inline size_t split_cnt_bytes(int sms) { return (size_t(sms) * 2 * sizeof(int32_t) + 255) & ~size_t(255); }
inline size_t split_lm_bytes(int sms) { return size_t(sms) * 2 * kPfRows * sizeof(float2); }
inline size_t split_area_bytes(int sms) {
  return split_cnt_bytes(sms) + split_lm_bytes(sms) + size_t(sms) * 2 * 2 * 16 * kPfRows * sizeof(float4);
}
inline int ws_fb_cap(int B, int Tmax) {
  // items of the largest call (T = Tmax); an item is listed once, or once for each
  // slot by each of up to 4 units (split items of a bf16 cache), plus once for its
  // sequence's V
  return 9 * ((Tmax + kPfRows - 1) / kPfRows) * B * GROK_N_KV_HEADS * 3;
}

// How many items run whole and how many units share each of the rest.
inline void split_plan(int n_items, int sms, bool allowed, int max_parts, int& n_whole, int& n_parts) {
  n_whole = n_items;
  n_parts = 1;
  if (n_items < 2 * sms && allowed) {
    const int rest = n_items % sms;
    const int parts = rest > 0 ? std::min(max_parts, sms / rest) : 1;
    if (parts > 1) {
      n_whole = n_items - rest;
      n_parts = parts;
    }
  }
}

// Attention over copies of an 8-bit cache (kv8_prefill.cu makes them): k_copy
// [B][8][rows][128] bf16 codes, v_copy the same in fp16 (fp16 passes) or bf16
// (fallback pass), K scales [B][8][rows / 64], the outputs' factors [B][8].
struct Q8Prefill {
  const grok_bf16* q;
  grok_bf16* out;
  const void *k_copy, *v_copy;
  int rows;
  const float *k_scale, *o_scale;
  const int32_t *cache_len, *valid_len;
  int B, T, Tmax, sms;
  int32_t *fb_count, *fb_list;
  int fb_cap;
  int n_whole, n_parts;  // split_plan
  char* split_area;
  int32_t* status;
};
// fallback false: the fp16 passes; true: the listed items with bf16 weights. Every
// pass is launched as the programmatic dependent of the kernel before it.
grok_status prefill_q8_passes(const Q8Prefill& a, bool fallback, cudaStream_t stream);

}  // namespace grok
