// Eviction from the 8-bit KV cache by accumulated attention weight.
//
// One warp per (sequence, KV head): it holds the head's row of the table and its
// weights in registers (up to 1024 entries, 32 a lane), finds the threshold weight
// bit by bit from the top (a count of the candidates at or above a trial value per
// bit, until the count is the one wanted), and writes each entry to its place in
// the new row, a prefix count of ballots. No shared memory and no barrier; the
// codes stay where they are. What is read and written is 16 bytes per entry.
#include "host.cuh"
#include "kv8.cuh"

namespace grok {

// Order of floats as unsigned integers: NaN like minus infinity, -0 like +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0x007FFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kEvWarps = 4;

// kPer: entries a lane holds; entry 32 e + lane of the row is e of the lane.
template <int kPer>
__global__ void __launch_bounds__(kEvWarps * 32, 4) kv8_evict_kernel(const int32_t* table, const float* weight,
                                                                  const int32_t* kv_len, int n_rows, int max_blocks,
                                                                  int keep, int sink, int recent, int32_t* table_out,
                                                                  float* weight_out, int32_t* kv_len_out,
                                                                  int32_t* status) {
  const int r = blockIdx.x * kEvWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= n_rows) return;
  const int b = r / kKVHeads;
  const size_t row = (size_t)r * max_blocks;
  const int len = kv_len[b];
  int id[kPer];
  float w[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int i = 32 * e + lane;
    id[e] = i < max_blocks ? table[row + i] : 0;
    w[e] = i < max_blocks ? weight[row + i] : 0.f;
  }
  const bool bad = len < 0 || len > max_blocks * kKv8Block;
  const int closed = bad ? 0 : len / kKv8Block;
  const bool cut = closed > keep;
  if (lane == 0 && r % kKVHeads == 0) {
    if (bad) report(status, GROK_DEV_BAD_KV_LEN);
    kv_len_out[b] = cut ? keep * kKv8Block + len % kKv8Block : len;
  }
  __syncwarp();  // the row is read before it is written (the outputs may be the inputs)
  if (!cut) {
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (32 * e + lane < max_blocks) {
        table_out[row + 32 * e + lane] = id[e];
        weight_out[row + 32 * e + lane] = w[e];
      }
    return;
  }
  // Blocks [sink, free_end) are chosen by weight: the `quota` largest of them (there are more).
  const int free_end = closed - recent, quota = keep - min(sink, closed) - recent;
  uint32_t edge = 0;
  int above = 0;  // candidates at or above `edge`
  uint32_t key[kPer];  // 0 for the others (a candidate's key is not)
#pragma unroll
  for (int e = 0; e < kPer; ++e) key[e] = 32 * e + lane >= sink && 32 * e + lane < free_end ? order_key(w[e]) : 0u;
  if (quota > 0) {
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t trial = edge | (1u << bit);
      int n = 0;
#pragma unroll
      for (int e = 0; e < kPer; ++e) n += key[e] >= trial;
      n = __reduce_add_sync(0xffffffffu, n);
      if (n >= quota) {
        edge = trial;
        above = n;
        if (n == quota) break;  // exactly those at or above it
      }
    }
  } else {
    edge = 0xFFFFFFFFu;
  }
  // Unless the search ended early, the blocks equal to `edge` are too many by above - quota: the last ones go.
  int ties = 0x7FFFFFFF;
  if (above > quota) {
    int equal = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) equal += key[e] == edge;
    ties = __reduce_add_sync(0xffffffffu, equal) - (above - quota);
  }
  const uint32_t lower = (1u << lane) - 1u;
  int32_t* t_out = table_out + row;
  float* w_out = weight_out + row;
  const int gone_at = keep + (closed < max_blocks ? 1 : 0);  // behind the open block
  int rank = 0;  // blocks that stay, before this run of 32
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int i = 32 * e + lane;
    bool stays = i < closed && (i < sink || i >= free_end || key[e] >= edge);
    if (ties < kPer * 32) {
      const bool tie = key[e] == edge;  // (edge is not 0 here)
      const uint32_t tied = __ballot_sync(0xffffffffu, tie);
      stays = stays && !(tie && __popc(tied & lower) >= ties);
      ties -= min(ties, __popc(tied));
    }
    const uint32_t staying = __ballot_sync(0xffffffffu, stays);
    const int before = rank + __popc(staying & lower);
    rank += __popc(staying);
    int to = before;
    if (!stays) to = i < closed ? gone_at + i - before : i == closed ? keep : i;
    if (i < max_blocks) {
      t_out[to] = id[e];
      w_out[to] = i < closed && !stays ? 0.f : w[e];
    }
  }
}

}  // namespace grok

using namespace grok;

extern "C" grok_status grok_kv8_evict(const int32_t* table, const float* weight, const int32_t* kv_len, int B,
                                      int max_blocks, int keep, int sink, int recent, int32_t* table_out,
                                      float* weight_out, int32_t* kv_len_out, int32_t* dev_status, void* stream) {
  if (!table || !weight || !kv_len || !table_out || !weight_out || !kv_len_out)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_evict: null pointer");
  if (kv_len_out == kv_len) return fail(GROK_ERR_INVALID_ARG, "grok_kv8_evict: kv_len_out may not alias kv_len");
  if (B < 1 || B > 65535 || max_blocks < 1 || max_blocks > kKv8MaxBlocks)
    return fail(GROK_ERR_INVALID_ARG, "grok_kv8_evict: need 1 <= B <= 65535, 1 <= max_blocks <= %d (B=%d max_blocks=%d)",
                kKv8MaxBlocks, B, max_blocks);
  if (keep < 1 || sink < 0 || recent < 0 || (long long)sink + recent > keep)
    return fail(GROK_ERR_INVALID_ARG,
                "grok_kv8_evict: need keep >= 1, sink, recent >= 0, sink + recent <= keep (keep=%d sink=%d recent=%d)",
                keep, sink, recent);
  int sms = 0;
  grok_status st = device_sm_count(&sms);
  if (st != GROK_OK) return st;
  const int n_rows = B * kKVHeads;
  auto kernel = max_blocks <= 128   ? kv8_evict_kernel<4>
                : max_blocks <= 256 ? kv8_evict_kernel<8>
                : max_blocks <= 512 ? kv8_evict_kernel<16>
                                    : kv8_evict_kernel<32>;
  kernel<<<(n_rows + kEvWarps - 1) / kEvWarps, kEvWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(
      table, weight, kv_len, n_rows, max_blocks, keep, sink, recent, table_out, weight_out, kv_len_out, dev_status);
  return check_launch("kv8_evict");
}
