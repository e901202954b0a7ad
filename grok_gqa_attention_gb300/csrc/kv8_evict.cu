// Eviction from the 8-bit KV cache by accumulated attention weight.
//
// One CTA of four warps per (sequence, KV head): it holds the head's row of the
// table and its weights in registers (up to 1024 entries, 8 a thread), finds the
// threshold weight bit by bit from the top (a count of the entries at or above a
// trial value per bit, until the count is the one wanted), and writes each entry to
// its place in the new row, a prefix count of ballots. The codes stay where they
// are; what is read and written is 16 bytes per entry.
//
// Bound by that search (71 % of the issue slots are busy). 2048 rows of 1024: 41 us with a thread per
// entry (32 barriers of 1024 threads), 14.0 us with a warp per row (13 warps on an
// SM do not hide it), 13.2 us with four; reading and writing 34 MB takes 5 us.
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
constexpr int kEvThreads = kEvWarps * 32;

// Places of the flagged entries among all flagged ones, in the row's order: flag[e] is entry e * kEvThreads + thread.
// counts: shared, one per (e, warp).
template <int kPer>
__device__ __forceinline__ void flagged_before(const bool (&flag)[kPer], int (&before)[kPer], int* counts) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();  // counts may still be read
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const uint32_t ballot = __ballot_sync(0xffffffffu, flag[e]);
    before[e] = __popc(ballot & ((1u << lane) - 1u));
    if (lane == 0) counts[e * kEvWarps + warp] = __popc(ballot);
  }
  __syncthreads();
  // at most 32 counts: every warp sums those before each of its own
  const int mine = lane < kPer * kEvWarps ? counts[lane] : 0;
  int incl = mine;
#pragma unroll
  for (int d = 1; d < kPer * kEvWarps; d *= 2) {
    const int up = __shfl_up_sync(0xffffffffu, incl, d);
    if (lane >= d) incl += up;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) before[e] += __shfl_sync(0xffffffffu, incl - mine, e * kEvWarps + warp);
}

// kPer: entries a thread holds.
template <int kPer>
__global__ void __launch_bounds__(kEvThreads) kv8_evict_kernel(const int32_t* table, const float* weight,
                                                               const int32_t* kv_len, int max_blocks, int keep,
                                                               int sink, int recent, int32_t* table_out,
                                                               float* weight_out, int32_t* kv_len_out,
                                                               int32_t* status) {
  __shared__ int counts[32];
  __shared__ int4 sums[2];  // a count of each warp; trials alternate between the two
  const int b = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const size_t row = ((size_t)b * kKVHeads + blockIdx.x) * max_blocks;
  const int len = kv_len[b];
  int id[kPer];
  float w[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int i = kEvThreads * e + tid;
    id[e] = i < max_blocks ? table[row + i] : 0;
    w[e] = i < max_blocks ? weight[row + i] : 0.f;
  }
  const bool bad = len < 0 || len > max_blocks * kKv8Block;
  const int closed = bad ? 0 : len / kKv8Block;
  const bool cut = closed > keep;
  if (tid == 0 && blockIdx.x == 0) {
    if (bad) report(status, GROK_DEV_BAD_KV_LEN);
    kv_len_out[b] = cut ? keep * kKv8Block + len % kKv8Block : len;
  }
  __syncthreads();  // the row is read before it is written (the outputs may be the inputs)
  if (!cut) {
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      const int i = kEvThreads * e + tid;
      if (i < max_blocks) {
        table_out[row + i] = id[e];
        weight_out[row + i] = w[e];
      }
    }
    return;
  }
  // The `keep` largest keys stay: the first and last blocks have the largest key of all, blocks [sink, free_end) one by
  // their weight, and what is no full block has 0, which no other has.
  const int free_end = closed - recent;
  uint32_t key[kPer];
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int i = kEvThreads * e + tid;
    key[e] = i >= closed ? 0u : i < sink || i >= free_end ? 0xFFFFFFFFu : order_key(w[e]);
  }
  auto total = [&](int n, int turn) {
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) reinterpret_cast<int*>(&sums[turn & 1])[warp] = n;
    __syncthreads();
    const int4 x = sums[turn & 1];
    return x.x + x.y + x.z + x.w;
  };
  uint32_t edge = 0;
  int above = 0;  // keys at or above `edge`
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t trial = edge | (1u << bit);
    int n = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) n += key[e] >= trial;
    n = total(n, bit);
    if (n >= keep) {
      edge = trial;
      above = n;
      if (n == keep) break;  // exactly those at or above it
    }
  }
  bool flag[kPer];
  int before[kPer];
  // Unless the search ended early, the keys equal to `edge` are too many by above - keep: the last of them go.
  if (above > keep) {
    int equal = 0;
#pragma unroll
    for (int e = 0; e < kPer; ++e) {
      flag[e] = key[e] == edge;
      equal += flag[e];
    }
    __syncthreads();  // the last trial's sums are read
    const int ties = total(equal, 0) - (above - keep);
    flagged_before<kPer>(flag, before, counts);
#pragma unroll
    for (int e = 0; e < kPer; ++e)
      if (flag[e] && before[e] >= ties) key[e] = 0u;
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) flag[e] = key[e] >= edge;
  flagged_before<kPer>(flag, before, counts);
  const int gone_at = keep + (closed < max_blocks ? 1 : 0);  // behind the open block
#pragma unroll
  for (int e = 0; e < kPer; ++e) {
    const int i = kEvThreads * e + tid;
    int to = flag[e] ? before[e] : gone_at + i - before[e];
    float x = flag[e] ? w[e] : 0.f;
    if (i >= closed) {  // the open block, and what lies behind it
      to = i == closed ? keep : i;
      x = w[e];
    }
    if (i < max_blocks) {
      table_out[row + to] = id[e];
      weight_out[row + to] = x;
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
  auto kernel = max_blocks <= 128   ? kv8_evict_kernel<1>
                : max_blocks <= 256 ? kv8_evict_kernel<2>
                : max_blocks <= 512 ? kv8_evict_kernel<4>
                                    : kv8_evict_kernel<8>;
  kernel<<<dim3(kKVHeads, B), kEvThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      table, weight, kv_len, max_blocks, keep, sink, recent, table_out, weight_out, kv_len_out, dev_status);
  return check_launch("kv8_evict");
}
