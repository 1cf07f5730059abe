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
constexpr int kPagedOneCells = 64, kPagedFewCells = 64, kPagedPromptCells = 128;   // cells of a part at least
constexpr int kPagedNear = 8;          // neighbouring tokens further apart than this do not share a group
constexpr int kPagedMaxLen = 1 << 30;  // positions of a sequence
// Partial results, (max, sum) and sums: of each of a launch's parts two runs of `tokens` tokens.
struct PagedPartials {
  float* ml;
  float* o;
  int tokens, parts;
};
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
  PagedPartials of;         // of this launch's parts, at most
  PagedPartials kinds[2];   // of both, for the join
  int4* geo;                // per token: sinks, window start, positions read, cells of a tile
  float2* lse;              // per row: max, 1 / sum
  float* em;                // per row and tile: its largest score
  float* e;                 // per row and block: its sum relative to that
  int64_t e_tiles, e_blocks;
  // Of two launches that share a call's tokens (kMixed) each takes runs of neighbouring tokens of more than run_lo and at
  // most run_hi of them; the first leaves word in `left` whether there are others.  kind 0: tokens one by one, 1: groups.
  int run_lo, run_hi, second, kind;
  int* left;
};
// Tokens one by one (attn_paged_one.cu), in groups of 16 (attn_paged_few.cuh; kMixed: attn_paged_few_mixed.cu), in groups of
// 32 on pairs of CTAs, fp16 rows (attn_paged_tc.cu): the kernel, in a.of.parts parts.
cudaError_t launch_paged_one(const PagedArgs& a, int kv_type, bool mixed, unsigned* err, cudaStream_t stream);
cudaError_t launch_paged_few(const PagedArgs& a, int kv_type, unsigned* err, cudaStream_t stream);
cudaError_t launch_paged_few_mixed(const PagedArgs& a, int kv_type, unsigned* err, cudaStream_t stream);
cudaError_t launch_paged_prompt(const PagedArgs& a, bool mixed, unsigned* err, cudaStream_t stream);
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
