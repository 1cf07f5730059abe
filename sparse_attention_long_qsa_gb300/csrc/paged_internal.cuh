// Launchers of the attention over whole caches and of the eviction.
#pragma once

#include "qsa_internal.cuh"

namespace qsa {

// Their kernel ids of qsa_profile_kernel (include/qsa.h), behind the step's.
enum PagedKernelId : int { kKPaged = kNumKernels, kKEvict, kNumAllKernels };
struct PagedProfileHook {
  cudaEvent_t before[kNumAllKernels - kNumKernels];
  cudaEvent_t after[kNumAllKernels - kNumKernels];
};
extern PagedProfileHook g_paged_profile;
inline void prof_before(PagedKernelId k, cudaStream_t s) {
  if (g_paged_profile.before[k - kNumKernels])
    cudaEventRecordWithFlags(g_paged_profile.before[k - kNumKernels], s, cudaEventRecordExternal);
}
inline void prof_after(PagedKernelId k, cudaStream_t s) {
  if (g_paged_profile.after[k - kNumKernels])
    cudaEventRecordWithFlags(g_paged_profile.after[k - kNumKernels], s, cudaEventRecordExternal);
}

// Attention over all cells of a paged cache, or a window of them (attn_paged.cu).
constexpr int kPagedPlan = 4096;       // tokens of one launch
constexpr int kPagedWeigh = 64;        // with block weights, whose workspace grows with them
constexpr int kPagedMaxParts = 320;    // CTAs of one launch
constexpr int kPagedMaxPairs = 80;     // pairs of CTAs
constexpr int kPagedMaxFew = 160;      // CTAs that take an SM each
constexpr int kPagedNear = 8;          // neighbouring tokens further apart than this do not share a group
constexpr int kPagedMaxLen = 1 << 30;  // positions of a sequence
struct PagedArgs {
  int n_tokens;
  int n_kv_heads;
  int r_shift;              // log2 of the cells per block
  int window;               // 0: all positions
  int n_sink;
  float attn_scale;
  const __half* q;
  const int32_t* tok_seq;
  const int32_t* tok_pos;
  const void* k_cache;
  const void* v_cache;
  int64_t n_cells;
  const int32_t* blk_cells;
  int64_t n_slots;
  const int64_t* seq_blk_off;
  const int32_t* seq_blk_slots;
  int n_seq;
  int64_t n_list;
  int64_t max_len;
  float* out;
  float* block_weight;
  int weigh;
  // workspace (paged_workspace_bytes fills these)
  // a group whose tiles go on from one part to the next: first token, tokens, first and last part.  One entry per token if
  // a launch has no more tokens than parts, else one per part (all of them but the last)
  int4* span;
  int span_by_token;
  int part_tokens;          // tokens of a partial result
  float* part_ml;
  float* part_o;
  int4* geo;                // per token: sinks, window start, positions read, sequence
  float2* lse;              // per row: max, 1 / sum
  float* em;                // per row and tile: its largest score
  float* e;                 // per row and block: its sum relative to that
  int64_t e_tiles, e_blocks;
  int e_cells;              // cells of a tile there
};
// Tokens that share a group at most, by what a call's sequences have on average.
int paged_group(const PagedArgs& a, int kv_type);
// Runs that each KV head's tiles of so many cells are dealt in, by `ctas` CTAs (or pairs), at most
// most_ctas of them.
int64_t paged_launch_parts(const PagedArgs& a, int64_t ctas, int64_t most_ctas, int cells);
// Adds the partial results of groups that several of the parts share (attn_paged.cu).
cudaError_t launch_paged_join(const PagedArgs& a, int64_t parts, cudaStream_t stream);
// One token of a sequence (attn_paged_one.cu).
cudaError_t launch_paged_one(const PagedArgs& a, int kv_type, unsigned* err, cudaStream_t stream);
// Two tokens and more (attn_paged_few.cu).
cudaError_t launch_paged_few(const PagedArgs& a, int kv_type, unsigned* err, cudaStream_t stream);
// Many tokens of a sequence, fp16 rows (attn_paged_tc.cu).
cudaError_t launch_paged_prompt(PagedArgs a, unsigned* err, cudaStream_t stream);
size_t paged_workspace_bytes(int n_tokens, int n_kv_heads, int64_t max_len, int r_shift, bool weigh, PagedArgs* a, void* ws);
cudaError_t launch_paged_attn(const PagedArgs& a, int kv_type, unsigned* err, cudaStream_t stream);

// Eviction by attention weight (evict.cu).
struct EvictArgs {
  int keep;
  int n_sink;
  int n_recent;
  int r;
  int n_seq;
  int64_t n_list;
  int64_t max_blocks;
  const int32_t* seq_len;
  const int64_t* seq_blk_off;
  const int32_t* seq_blk_slots;
  const float* block_weight;
  int32_t* len_out;
  int32_t* slots_out;
  float* weight_out;
  int32_t* n_evicted;       // may be null
};
constexpr int64_t evict_max_blocks() { return 1 << 20; }   // entries of one sequence's list
cudaError_t launch_cache_evict(const EvictArgs& a, unsigned* err, cudaStream_t stream);

// Weights of entries behind the sequences' blocks to zero (cache_ops.cu).
cudaError_t launch_weight_trim(const int32_t* seq_len, const int64_t* seq_blk_off, int n_seq, int r, int64_t n_list, float* block_weight,
                               unsigned* err, cudaStream_t stream);

}  // namespace qsa
