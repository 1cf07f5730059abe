// Attention over all cells of a paged cache (or a sliding window of them and a
// few first ones): which kernel takes a call, its workspace, and the block weights.
//
//   out[t][h] = sum_{j visible to t} softmax_j(scale * q[t][h] . K[c_j][g]) V[c_j][g]
//
// Three kernels share the work split.  Consecutive tokens of one sequence form
// groups, which read their cells once.  A group's positions are cut into tiles, and
// the tiles of all groups, laid end to end, are dealt in equal runs to the CTAs of a
// KV head, however long each sequence is (or, where no part gets much more than its
// share for that, in whole groups, see plan).  A run that covers a group whole writes
// its output; the others leave (max, sum, o) in the workspace, and k_paged_join adds
// them in the order of the runs.
//   attn_paged_one.cu   single tokens: bound by the reading of the rows
//   attn_paged_few.cuh  several tokens of a sequence, rows of any type: by forming
//                       operands
//   attn_paged_tc.cu    many tokens of fp16 rows: by the tensor cores; pairs of CTAs
//                       gather half the bytes that the kernel for few tokens would
// A call of both kinds goes to two of them (see route).
//
// Sums and the softmax are fp32.  K and V enter the products as they are stored, or
// codes times scales in parts that hold them exactly; probabilities go in as two fp16
// parts: 22 bits, less where they lie far below others that are read with them (each
// kernel says how far).
#include <algorithm>
#include <atomic>

#include "attn_paged.cuh"

namespace qsa {
namespace {

// Adds the runs of a group that is spread over several parts.  Entries per token: a
// block is a token and head; four dims a thread, every eighth part, the first of these
// loaded with the parts' (max, sum), so that a row costs one wait for memory.  Entries
// per part (more tokens than parts): four blocks of each of the group's parts share
// its rows; 64 threads take a row, eight parts at a time.
constexpr int kJoinThreads = 512, kJoinBlocks = 4;
static_assert(kPagedMaxParts <= kJoinThreads, "a thread a part");
template <bool kMixed>
__global__ void __launch_bounds__(kJoinThreads, 2) k_paged_join(const PagedArgs a) {
  __shared__ float w[kPagedMaxParts];
  __shared__ float4 o[7][64];
  __shared__ float red[2][kJoinThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = blockIdx.y, G = a.n_kv_heads;
  grid_dep_wait();
  grid_dep_launch();
  const int4 sp = a.span[blockIdx.x];
  if (sp.y == 0) return;
  const int first = sp.z, np = sp.w - first + 1;   // the group's parts
  const bool groups = kMixed && (sp.y >> 8) != 0;
  const int tokens = sp.y & 255, nth = blockIdx.x - (groups ? a.kinds[0].parts : 0) - first;   // (an entry a part: which of them)
  const float* part_ml = !kMixed ? a.of.ml : groups ? a.kinds[1].ml : a.kinds[0].ml;
  const float* part_o = !kMixed ? a.of.o : groups ? a.kinds[1].o : a.kinds[0].o;
  const int part_tokens = !kMixed ? a.of.tokens : groups ? a.kinds[1].tokens : 1;
  auto row_of = [&](int i, int t, int h) -> int64_t {
    return ((int64_t)(2 * (first + i) + (i == 0 ? 1 : 0)) * G + g) * (part_tokens * kGqa) + t * kGqa + h;
  };
  const int d = tid & 63, slice = tid >> 6;
  auto add = [](float4& s, float c, const float4& y) {
    s.x = fmaf(c, y.x, s.x), s.y = fmaf(c, y.y, s.y), s.z = fmaf(c, y.z, s.z), s.w = fmaf(c, y.w, s.w);
  };
  auto write = [&](int64_t row, const float4& s, float l) {
    const float inv = l != 0.f ? 1.f / l : 0.f;
    float* out = a.out + row * kHeadDim + 4 * d;
    out[0] = s.x * inv, out[1] = s.y * inv, out[2] = s.z * inv, out[3] = s.w * inv;
  };
  constexpr int kBatch = 8, kEarly = 6;
  if (!a.span_by_token) {
    const int share = nth * kJoinBlocks + blockIdx.z, shares = (np - 1) * kJoinBlocks;
    for (int r = share * 8 + slice; r < tokens * kGqa; r += shares * 8) {   // rows: token, head
      const int t = r / kGqa, hr = r % kGqa;
      float m = kNoMax, l = 0.f;
      float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int i0 = 0; i0 < np; i0 += kBatch) {
        float2 ml[kBatch];
        float4 x[kBatch];
        float nm = m, nan = 0.f;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          ml[i] = make_float2(kNoMax, 0.f);
          x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (i0 + i < np) {
            ml[i] = *reinterpret_cast<const float2*>(part_ml + 2 * row_of(i0 + i, t, hr));
            x[i] = *reinterpret_cast<const float4*>(part_o + row_of(i0 + i, t, hr) * kHeadDim + 4 * d);
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          nm = fmaxf(nm, ml[i].x);
          nan = fmaf(0.f, ml[i].x, nan);   // (fmaxf drops NaN)
        }
        nm += nan;
        const float f0 = ex2(m - nm);
        l *= f0;
        s.x *= f0, s.y *= f0, s.z *= f0, s.w *= f0;
        m = nm;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (i0 + i >= np) continue;
          const float f = ex2(ml[i].x - m);
          l = fmaf(f, ml[i].y, l);
          add(s, f, x[i]);
        }
      }
      const int64_t row = ((int64_t)(sp.x + t) * G + g) * kGqa + hr;
      if (d == 0 && a.weigh) a.lse[row] = make_float2(m, l != 0.f ? 1.f / l : 0.f);
      write(row, s, l);
    }
    return;
  }
  {
    const int h = blockIdx.z, t = blockIdx.x - sp.x;
    const float2 ml = tid < np ? *reinterpret_cast<const float2*>(part_ml + 2 * row_of(tid, t, h)) : make_float2(kNoMax, 0.f);
    float4 x[kEarly];
#pragma unroll
    for (int k = 0; k < kEarly; ++k) {
      const int i = slice + 8 * k;
      if (i < np) x[k] = *reinterpret_cast<const float4*>(part_o + row_of(i, t, h) * kHeadDim + 4 * d);
    }
    float m = ml.x;
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, s));
    if (lane == 0) red[0][warp] = m;
    __syncthreads();
    m = red[0][lane & 15];
#pragma unroll
    for (int s = 8; s >= 1; s >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, s));
    if (ml.x != ml.x) m = ml.x;   // (fmaxf drops NaN)
    const float f = ex2(ml.x - m);
    float l = f * ml.y;
    if (tid < np) w[tid] = f;
#pragma unroll
    for (int s = 16; s >= 1; s >>= 1) l += __shfl_xor_sync(kFull, l, s);
    if (lane == 0) red[1][warp] = l;
    __syncthreads();
    l = red[1][lane & 15];
#pragma unroll
    for (int s = 8; s >= 1; s >>= 1) l += __shfl_xor_sync(kFull, l, s);
    const int64_t row = ((int64_t)(sp.x + t) * G + g) * kGqa + h;
    if (tid == 0 && a.weigh) a.lse[row] = make_float2(m, l != 0.f ? 1.f / l : 0.f);
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kEarly; ++k)
      if (slice + 8 * k < np) add(s, w[slice + 8 * k], x[k]);
#pragma unroll 8
    for (int i = slice + 8 * kEarly; i < np; i += 8)
      add(s, w[i], *reinterpret_cast<const float4*>(part_o + row_of(i, t, h) * kHeadDim + 4 * d));
    if (slice > 0) o[slice - 1][d] = s;
    __syncthreads();
    if (slice == 0) {
#pragma unroll
      for (int i = 0; i < 7; ++i) {
        const float4 y = o[i][d];
        s.x += y.x, s.y += y.y, s.z += y.z, s.w += y.w;
      }
      write(row, s, l);
    }
  }
}

// block_weight[entry] += the probabilities of the entry's block, over the call's
// tokens of its sequence and their heads.  A block takes every gridDim.x-th 64 entries of
// the sequences that start at its share of the tokens.  A lane holds two entries; the warps
// take every eighth head, and their sums are added in warp order.  (Five tokens over
// 250k: 20 MB of block sums, 14 us; with one entry a lane and its loads one after the
// other it took 26.)
constexpr int kWeighThreads = 256, kWeighWarps = kWeighThreads / 32, kWeighBlocks = 2048, kWeighEntries = 64;
template <bool kMixed>
__global__ void __launch_bounds__(kWeighThreads) k_paged_weigh(const PagedArgs a, int tile_cells) {
  __shared__ float part[2][kWeighWarps][kWeighEntries];
  __shared__ int seq_of[kPagedWeigh], tok[kPagedWeigh];   // of all tokens; the sequence's
  __shared__ int4 geo[kPagedWeigh];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = a.n_kv_heads, heads = G * kGqa;
  const int one_tile = 31 - __clz(tile_cells) - a.r_shift;   // (the same for all tokens)
  grid_dep_wait();
  grid_dep_launch();
  if (tid < kPagedWeigh) {
    const int s = tid < a.n_tokens ? a.tok_seq[tid] : -1;
    seq_of[tid] = tid < a.n_tokens && token_pos(a, tid) >= 0 ? s : -1;
    if (tid < a.n_tokens) {
      geo[tid] = a.geo[tid];
      if (kMixed) geo[tid].w = 31 - __clz(geo[tid].w) - a.r_shift;   // log2 of the blocks of a tile
    }
  }
  __syncthreads();
  const int share = (a.n_tokens + gridDim.y - 1) / gridDim.y;
  for (int t0 = blockIdx.y * share; t0 < min((int)(blockIdx.y + 1) * share, a.n_tokens); ++t0) {
    const int seq = seq_of[t0];
    const unsigned lo32 = __ballot_sync(kFull, seq_of[lane] == seq), hi32 = __ballot_sync(kFull, seq_of[32 + lane] == seq);
    const uint64_t who = (uint64_t)hi32 << 32 | lo32;
    if (seq < 0 || __ffsll((long long)who) - 1 < t0) continue;   // not the sequence's first token
    const int64_t off = a.seq_blk_off[seq], n = a.seq_blk_off[seq + 1] - off;
    if (off < 0 || n < 0 || off + n > a.n_list) continue;
    __syncthreads();
    if (tid < kPagedWeigh && (who >> tid & 1)) tok[__popcll(who & ((UINT64_C(1) << tid) - 1))] = tid;
    __syncthreads();
    const int tokens = __popcll(who);
    int b01 = 0;
    for (int64_t first = (int64_t)blockIdx.x * kWeighEntries; first < n; first += (int64_t)gridDim.x * kWeighEntries, b01 ^= 1) {
      const int64_t j = first + lane;
      float sum[2] = {0.f, 0.f};
      // the warp's rows, four at a time: all their loads before the first is used
      constexpr int kRows = 4;
      for (int k = 0, h = 0; k < tokens;) {
        float2 l[kRows];
        float e[kRows][2], m[kRows][2];
        unsigned have = 0u;
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const bool row_there = k < tokens;
          const int t = tok[row_there ? k : 0];
          const int4 at = geo[t];
          const int ns = at.x >> a.r_shift, lo = at.y >> a.r_shift;
          const int64_t row = (int64_t)t * heads + h * kWeighWarps + warp;
          l[i] = a.lse[row];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int64_t x = j + 32 * c;
            int64_t b = x < ns ? x : x >= lo ? x - lo + ns : -1;
            const bool there = row_there && b >= 0 && x < n && (b << a.r_shift) < at.z;
            if (there) have |= 1u << (2 * i + c);
            else b = 0;   // (read, and not used)
            e[i][c] = a.e[row * a.e_blocks + b];
            m[i][c] = a.em[row * a.e_tiles + (b >> (kMixed ? at.w : one_tile))];
          }
          if (row_there && ++h == heads / kWeighWarps) h = 0, ++k;
        }
#pragma unroll
        for (int i = 0; i < kRows; ++i)
#pragma unroll
          for (int c = 0; c < 2; ++c)   // (a row may be NaN)
            if ((have >> (2 * i + c) & 1u) && e[i][c] != 0.f) sum[c] = fmaf(e[i][c], ex2(m[i][c] - l[i].x) * l[i].y, sum[c]);
      }
      part[b01][warp][lane] = sum[0];
      part[b01][warp][32 + lane] = sum[1];
      __syncthreads();
      if (tid < kWeighEntries) {
        float x = 0.f;
#pragma unroll
        for (int w = 0; w < kWeighWarps; ++w) x += part[b01][w][tid];
        if (x != 0.f) a.block_weight[off + first + tid] += x;   // (beyond the list: zero)
      }
    }
  }
}

// Which kernels a launch's tokens go to.  Tokens one by one read their rows once each; groups of 16, or on pairs of CTAs of
// 32, share them.  Measured, us, one by one / groups of 16 / pairs' groups of 32:
//   2 tokens of 50k f16 37 / 40 / 42, q8_0 32 / 37, q4_0 29 / 37; 24 x 2 tokens of 3,000 f16 42 / 50 / 52, q8_0 41 / 49
//   3 tokens of 50k f16 51 / 41 / 43, q8_0 47 / 39, q4_0 42 / 39
//   16 tokens of 50k f16 - / 46 / 45; 24 x 12 tokens of 3,000 - / 54 / 56; 24 x 24 - / 78 / 63; 48 x 8 of 1,000 - / 42 / 72
// Two tokens one by one read their rows twice, which pays as long as the second reading is L2's.
//
// What the call's tokens come to for each list on average says which; how many are neighbours only the device sees.  Where
// there are several lists the average may be far out: drafted tokens or a chunk of a prompt in a table of many lists, or
// beside single tokens (us, by the average / by both kinds: 5 of 250k q8_0 in 64 lists 246 / 145, and 63 single tokens
// beside them 413 / 173; 64 of 50k f16 634 / 88; 512 of 50k f16 in 64 lists 628 / 426, in 512 5,070 / 421).  So two kernels
// are launched, one for short runs of neighbours and one for long ones, of which either may find nothing to do.  That takes
// 2 to 3 us (64 single tokens of 300 in room for 100k f16 16.4 / 19.2, q8_0 15.8 / 18.5; of 11,000 254 / 251; with groups of
// 16 and 32, which have a join each, 5 to 8: 64 x 5 of 11,000 292 / 300).  So it is done where, by its lists' bound, the
// call takes a quarter of a millisecond if it is what its average says: tokens one by one read 5 TB/s, groups 3.
struct Route {
  enum Kernel { kOne, kFew, kPairs } kernel, high;   // `high` where `mixed`: for runs of more than `split` tokens
  bool mixed, high_first;
  int split;
};
Route route(const PagedArgs& a, int64_t call_tokens, int kv_type) {
  const int64_t per = ceil_div(call_tokens, a.n_seq > 0 ? a.n_seq : 1), seen = (int64_t)a.window + a.n_sink;
  const int64_t reach = a.window > 0 && seen < a.max_len ? seen : a.max_len;
  const int64_t row = kv_type == QSA_KV_F16 ? 512 : kv_type == QSA_KV_Q8_0 ? 272 : 144;
  const int64_t rows = 2 * reach * a.n_kv_heads * row;   // of a token
  const bool cached = rows <= INT64_C(100) << 20, pairs = kv_type == QSA_KV_F16 && !a.weigh;
  Route r{};
  r.kernel = per <= 1 || (per == 2 && cached) || a.n_tokens == 1 ? Route::kOne : per <= 16 || !pairs ? Route::kFew : Route::kPairs;
  const double bytes = (double)rows * (a.n_seq < a.n_tokens ? a.n_seq : a.n_tokens);
  r.mixed = a.n_seq > 1 && a.n_tokens > 2 && bytes >= (r.kernel == Route::kOne ? 1.25e9 : 0.75e9);
  const Route::Kernel groups = pairs && a.n_tokens > 16 ? Route::kPairs : Route::kFew;
  // (single tokens among groups of 16 cost much only where they are most)
  if (!r.mixed || (r.kernel == groups && groups == Route::kFew && per > 2)) {
    r.mixed = false;
    return r;
  }
  r.high = groups;
  r.high_first = r.kernel == groups;
  r.split = cached ? 2 : 1;
  if (r.kernel == Route::kFew && groups == Route::kPairs) r.split = 16;
  else r.kernel = Route::kOne;
  return r;
}

// Parts that each KV head's tiles are dealt in: by `ctas` CTAs (or pairs), at most most_ctas of them, no more than there can
// be tiles of so many cells.
int launch_parts(const PagedArgs& a, int64_t ctas, int64_t most_ctas, int cells) {
  const int64_t reach = a.window > 0 && a.window < a.max_len ? a.window : a.max_len;
  const int64_t most = (int64_t)a.n_tokens * ceil_div((reach < a.max_len - a.n_sink ? reach + a.n_sink : a.max_len) + cells, cells);
  return (int)std::min(std::max<int64_t>(std::min(ctas, most_ctas) / a.n_kv_heads, 1), most);
}

// The current device's.
cudaError_t multiprocessors(int* n) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  *n = known[dev].load(std::memory_order_relaxed);
  if (*n == 0) {
    e = cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) known[dev].store(*n, std::memory_order_relaxed);
  }
  return e;
}

// One of the kernels, without its join.
cudaError_t launch_kernel(const PagedArgs& a, Route::Kernel k, bool mixed, int kv_type, unsigned* err, cudaStream_t stream) {
  return k == Route::kOne     ? launch_paged_one(a, kv_type, mixed, err, stream)
         : k == Route::kPairs ? launch_paged_prompt(a, mixed, err, stream)
         : mixed              ? launch_paged_few_mixed(a, kv_type, err, stream)
                              : launch_paged_few(a, kv_type, err, stream);
}
// Adds the partial results of groups that several parts share.
cudaError_t launch_join(const PagedArgs& a, int parts, bool mixed, cudaStream_t stream) {
  const unsigned entries = (unsigned)(a.span_by_token ? a.n_tokens : parts), z = a.span_by_token ? kGqa : kJoinBlocks;
  const dim3 grid(entries, (unsigned)a.n_kv_heads, z);
  return mixed ? launch_pdl(k_paged_join<true>, grid, dim3(kJoinThreads), 0, stream, 1, a)
               : launch_pdl(k_paged_join<false>, grid, dim3(kJoinThreads), 0, stream, 1, a);
}

cudaError_t launch_tokens(PagedArgs a, const Route& r, int kv_type, int sms, unsigned* err, cudaStream_t stream) {
  auto partials = [&](Route::Kernel k) {
    PagedPartials x = a.kinds[k != Route::kOne];
    x.tokens = k == Route::kOne ? 1 : k == Route::kPairs ? 32 : a.n_tokens < 16 ? a.n_tokens : 16;
    x.parts = k == Route::kOne     ? launch_parts(a, sms, kPagedMaxParts, kPagedOneCells)
              : k == Route::kPairs ? launch_parts(a, sms / 2, kPagedMaxPairs, kPagedPromptCells)
                                   : launch_parts(a, sms, kPagedMaxFew, kPagedFewCells);
    return x;
  };
  cudaError_t e = cudaSuccess;
  if (!r.mixed) {
    a.of = partials(r.kernel);
    a.span_by_token = a.n_tokens <= a.of.parts;
    e = launch_kernel(a, r.kernel, false, kv_type, err, stream);
    return e == cudaSuccess && a.of.parts > 1 ? launch_join(a, a.of.parts, false, stream) : e;
  }
  // one by one and in groups: one join for both; groups of 16 and of 32 (whose partials take the same place): one each
  const bool joint = r.kernel == Route::kOne;
  a.kinds[0] = partials(r.kernel);
  a.kinds[1] = partials(r.high);
  a.span_by_token = joint && a.n_tokens <= std::min(a.kinds[0].parts, a.kinds[1].parts);
  for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
    const bool high = (i == 0) == r.high_first;
    PagedArgs b = a;
    b.second = i;
    b.run_lo = high ? r.split : 0;
    b.run_hi = high ? a.n_tokens : r.split;
    b.of = a.kinds[high];
    b.kind = joint && high;
    if (joint && high && !a.span_by_token) b.span += a.kinds[0].parts;
    e = launch_kernel(b, high ? r.high : r.kernel, true, kv_type, err, stream);
    if (e == cudaSuccess && !joint && b.of.parts > 1) e = launch_join(b, b.of.parts, false, stream);
  }
  if (e == cudaSuccess && joint && std::max(a.kinds[0].parts, a.kinds[1].parts) > 1)
    e = launch_join(a, a.kinds[0].parts + a.kinds[1].parts, true, stream);
  return e;
}

}  // namespace

// The workspace: spans, partials of two runs a part of either kind, and for block weights the
// tokens' geometry, rows' (max, 1 / sum) and block sums.
size_t paged_workspace_bytes(int n_tokens, int n_kv_heads, int64_t max_len, int r_shift, bool weigh, PagedArgs* a, void* ws) {
  unsigned char* base = static_cast<unsigned char*>(ws);
  size_t at = 0;
  auto take = [&](size_t bytes) -> unsigned char* {
    unsigned char* p = base == nullptr ? nullptr : base + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  const int64_t chunk = weigh ? kPagedWeigh : kPagedPlan;
  const int64_t tokens = n_tokens < chunk ? n_tokens : chunk, heads = tokens * n_kv_heads * kGqa;
  // rows of two runs a part: of the CTAs' groups (1 token, or up to 16), or of the pairs' (32)
  auto rows_of = [&](int64_t ctas, int64_t group) -> int64_t {
    const int64_t parts = ctas / n_kv_heads;
    return 2 * (parts > 0 ? parts : 1) * n_kv_heads * group * kGqa;
  };
  int64_t rows[2] = {rows_of(kPagedMaxParts, 1), 0};
  if (tokens > 1) rows[1] = rows_of(kPagedMaxFew, tokens < 16 ? tokens : 16);
  if (tokens > 16 && !weigh) rows[1] = std::max(rows[1], rows_of(kPagedMaxPairs, 32));
  PagedArgs x{};
  x.span = reinterpret_cast<int4*>(take(sizeof(int4) * (kPagedMaxParts + kPagedMaxFew)));
  x.left = reinterpret_cast<int*>(take(sizeof(int)));
  for (int i = 0; i < 2; ++i) {
    x.kinds[i].ml = reinterpret_cast<float*>(take(sizeof(float) * 2 * rows[i]));
    x.kinds[i].o = reinterpret_cast<float*>(take(sizeof(float) * kHeadDim * rows[i]));
  }
  if (weigh) {
    const int64_t tiles = ceil_div(max_len, 128) + 2, small = ceil_div(max_len, 16) + 2;
    x.geo = reinterpret_cast<int4*>(take(sizeof(int4) * tokens));
    x.lse = reinterpret_cast<float2*>(take(sizeof(float2) * heads));
    x.em = reinterpret_cast<float*>(take(sizeof(float) * heads * small));
    x.e = reinterpret_cast<float*>(take(sizeof(float) * heads * tiles * (128 >> r_shift)));
    x.e_tiles = small;
    x.e_blocks = tiles * (128 >> r_shift);
  }
  if (a != nullptr) {
    a->span = x.span, a->left = x.left, a->kinds[0] = x.kinds[0], a->kinds[1] = x.kinds[1];
    a->geo = x.geo, a->lse = x.lse, a->em = x.em, a->e = x.e, a->e_tiles = x.e_tiles, a->e_blocks = x.e_blocks;
  }
  return at;
}

cudaError_t launch_paged_attn(const PagedArgs& args, int kv_type, unsigned* err, cudaStream_t stream) {
  // the plan of a launch is held in shared memory, its tiles are counted in 31 bits
  const int64_t most = (INT64_C(1) << 31) / (ceil_div(args.max_len, 16) + 2) - 1, cap = args.weigh ? kPagedWeigh : kPagedPlan;
  const int chunk = (int)(most < cap ? most : cap);
  int sms = 0;
  cudaError_t e = multiprocessors(&sms);
  if (e != cudaSuccess) return e;
  for (int t = 0; t < args.n_tokens; t += chunk) {
    PagedArgs a = args;
    a.n_tokens = args.n_tokens - t < chunk ? args.n_tokens - t : chunk;
    a.tok_seq += t;
    a.tok_pos += t;
    a.q += (int64_t)t * a.n_kv_heads * kGqa * kHeadDim;
    a.out += (int64_t)t * a.n_kv_heads * kGqa * kHeadDim;
    prof_before(kKPaged, stream);
    const Route r = route(a, args.n_tokens, kv_type);
    e = launch_tokens(a, r, kv_type, sms, err, stream);
    if (e == cudaSuccess && a.weigh) {
      const int64_t blocks = std::max<int64_t>(ceil_div(ceil_div(a.max_len, (int64_t)1 << a.r_shift), kWeighEntries), 1);
      // a block a token while they are few: most start no sequence, and each sequence is a chain of loads
      const int64_t shares = std::max<int64_t>(std::min<int64_t>(a.n_tokens, kWeighBlocks / blocks), ceil_div(a.n_tokens, 8));
      const dim3 grid((unsigned)std::min<int64_t>(blocks, kWeighBlocks), (unsigned)shares);
      e = launch_pdl(r.mixed ? k_paged_weigh<true> : k_paged_weigh<false>, grid, dim3(kWeighThreads), 0, stream, 1, a,
                     r.kernel == Route::kOne ? 16 : 64);
    }
    prof_after(kKPaged, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace qsa
