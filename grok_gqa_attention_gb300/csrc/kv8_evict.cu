// Eviction from the 8-bit KV cache by accumulated attention weight.
//
// One CTA per (sequence, KV head), one thread per table entry (at most 1024).
// The threshold weight is found bit by bit from the top: a block-wide count of
// the candidates at or above a trial value per bit, 32 barriers, no memory
// traffic. Ranks among equals and the places in the new row are prefix counts.
// The codes stay where they are; what is read and written is 16 bytes per entry.
#include "host.cuh"
#include "kv8.cuh"

namespace grok {

// Order of floats as unsigned integers: NaN like minus infinity, -0 like +0.
__device__ __forceinline__ uint32_t order_key(float w) {
  if (w != w) return 0x007FFFFFu;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Number of earlier threads of the CTA with `flag`; counts is shared, one per warp.
__device__ __forceinline__ int prefix_count(bool flag, int* counts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t ballot = __ballot_sync(0xffffffffu, flag);
  if (lane == 0) counts[warp] = __popc(ballot);
  __syncthreads();
  const int n_warps = blockDim.x >> 5;
  const int before = __reduce_add_sync(0xffffffffu, lane < warp && lane < n_warps ? counts[lane] : 0);
  return before + __popc(ballot & ((1u << lane) - 1u));
}

__global__ void __launch_bounds__(1024) kv8_evict_kernel(const int32_t* table, const float* weight,
                                                         const int32_t* kv_len, int max_blocks, int keep, int sink,
                                                         int recent, int32_t* table_out, float* weight_out,
                                                         int32_t* kv_len_out, int32_t* status) {
  __shared__ int counts[2][32];
  const int g = blockIdx.x, b = blockIdx.y, i = threadIdx.x;
  const size_t row = ((size_t)b * kKVHeads + g) * max_blocks;
  const int len = kv_len[b];
  const bool bad = len < 0 || len > max_blocks * kKv8Block;
  const int closed = bad ? 0 : len / kKv8Block;
  const bool cut = closed > keep;
  if (i == 0 && g == 0) {
    if (bad) report(status, GROK_DEV_BAD_KV_LEN);
    kv_len_out[b] = cut ? keep * kKv8Block + len % kKv8Block : len;
  }
  const bool in = i < max_blocks;
  const int id = in ? table[row + i] : 0;
  const float w = in ? weight[row + i] : 0.f;
  int to = i;
  bool gone = false;
  if (cut) {  // uniform over the CTA
    const bool must = i < closed && (i < sink || i >= closed - recent);
    const bool free = i < closed && !must;
    const uint32_t key = free ? order_key(w) : 0u;
    const int quota = keep - __syncthreads_count(must);
    // the quota-th largest key among the free blocks (there are more than quota of them)
    uint32_t edge = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t trial = edge | (1u << bit);
      if (__syncthreads_count(free && key >= trial) >= quota) edge = trial;
    }
    const int ties = quota - __syncthreads_count(free && key > edge);
    const bool tie = free && key == edge;
    const int tie_rank = prefix_count(tie, counts[0]);
    const bool stays = must || (free && quota > 0 && (key > edge || (tie && tie_rank < ties)));
    const int rank = prefix_count(stays, counts[1]);
    gone = i < closed && !stays;
    if (i < closed)
      to = stays ? rank : keep + (closed < max_blocks ? 1 : 0) + i - rank;
    else if (i == closed)
      to = keep;
  } else {
    __syncthreads();  // every entry is read before one is written (the outputs may be the inputs)
  }
  if (in) {
    table_out[row + to] = id;
    weight_out[row + to] = gone ? 0.f : w;
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
  const int threads = (max_blocks + 31) / 32 * 32;
  kv8_evict_kernel<<<dim3(kKVHeads, B), threads, 0, static_cast<cudaStream_t>(stream)>>>(
      table, weight, kv_len, max_blocks, keep, sink, recent, table_out, weight_out, kv_len_out, dev_status);
  return check_launch("kv8_evict");
}
