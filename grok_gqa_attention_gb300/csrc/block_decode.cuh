// Attention of one token per sequence over 64-token blocks of a paged cache
// (block_decode.cu), used over a list of blocks per KV head (grok_attn_decode_sparse_paged)
// and over the rows behind a shared prefix (grok_attn_decode_shared_paged).
#pragma once

#include <utility>

#include "blocks.cuh"
#include "host.cuh"

namespace grok {

constexpr int kGroupsMax = 256;   // groups of sequences with a common prefix
constexpr int kPxSeqs = 21;       // sequences per query tile of the prefix kernel: 126 of its 128 rows

// Sequences [start[i], start[i + 1]) have their first pages[i] pages in common.
struct Groups {
  const int32_t* start;
  const int32_t* pages;
  int n;
};

// The groups in shared memory. One that is not usable, or of one sequence, which has nothing to share, has 0 pages.
struct GroupTable {
  int start[kGroupsMax + 1];
  int pages[kGroupsMax];
  // Pages that sequence b's group has in common.
  __device__ __forceinline__ int of_seq(int n, int b) const {
    if (b < start[0] || b >= start[n]) return 0;
    int lo = 0, hi = n;  // start[lo] <= b < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (start[mid] <= b) lo = mid; else hi = mid;
    }
    return pages[lo];
  }
};
// Loads them, by threads 0 to n - 1 of the CTA and without waiting for it; a thread's part of the check that starts
// ascend within [0, B] and pages lie within [0, max_pages] (where one fails, no group is used).
__device__ __forceinline__ bool load_groups(const Groups& gr, int B, int max_pages, GroupTable* t, int tid) {
  if (tid >= gr.n) return true;
  const int a = gr.start[tid], z = gr.start[tid + 1], pg = gr.pages[tid];
  t->start[tid] = a;
  if (tid == gr.n - 1) t->start[gr.n] = z;
  t->pages[tid] = z - a < 2 ? 0 : pg;
  return a >= 0 && z >= a && z <= B && pg >= 0 && pg <= max_pages;
}

// Partial results of the block kernel, per part: the sums O in the layout of the products' accumulators
// (float4 [8 tiles of 16 features][32 lanes]) and the weights' sums of 8 columns (6 heads, 2 unused).
constexpr int kBkWarps = 4;
constexpr int kBkPartO = 8 * 32;  // float4s
struct BlockParts {
  float4* o;
  float* l;
  int2* pair;  // [B * 8]: first part and number of parts; number -1: the sequence is skipped
};
// Partial results of the prefix kernel, per part: O as float4 [32 feature quads][128 rows], and four sums per row.
constexpr int kPxRows = 128;
constexpr int kPxSums = 4;
constexpr int kPxSmemMax = 134 * 1024;  // of the prefix kernel's CTA
struct PrefixParts {
  float4* o;
  float* l;
  // [B * 8]: first part, number of parts, the sequence's first row, pages << 16 | the sequence whose table is read
  int4* pair;
};

struct BlockArgs {
  const grok_bf16* q_rot;
  CUtensorMap tm_k, tm_v, tm_k16, tm_v16;  // of the pools (encode_pools)
  PageMap pm;
  const int32_t* kv_len;
  int B;
  const int32_t* sel;  // nullptr: the rows behind the groups' prefixes
  int budget;
  Groups groups;
  grok_bf16* out;
  int32_t* status;
  cudaStream_t stream;
};

size_t block_parts_bytes(int B, int sms);
size_t prefix_parts_bytes(int B, int n_groups, int sms);
// The block kernel, then the kernel that joins its partial results (and, where prefix is given, the prefix kernel's,
// which was launched before on the stream).
grok_status block_decode_run(const BlockArgs& a, char* ws, const PrefixParts* prefix, int sms);
PrefixParts prefix_parts(char* ws, int B, int n_groups, int sms);

// A launch in clusters of `cluster` CTAs. `beside`: as the programmatic dependent of the kernel before it on the stream,
// beside which it may start.
template <typename... Args, typename... Given>
cudaError_t launch(bool beside, int cluster, void (*kernel)(Args...), dim3 grid, int threads, int smem, cudaStream_t stream,
                   Given&&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = beside ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Given>(args)...);
}

// The tensor maps of the pools. One copy of tm_k or tm_v brings the 64 rows of a block of one head, as two tiles of [64
// rows][64 bf16], one of tm_k16 or tm_v16 16 rows of half of the features.
grok_status encode_pools(BlockArgs* a, const grok_bf16* k_pool, const grok_bf16* v_pool, int n_pages);

grok_status page_args(int n_pages, int max_pages, int B, const char* who);

}  // namespace grok
