// Shared by the kernels of qsa_paged_attn: the groups of tokens that read their
// cells together, and their tiles dealt to the CTAs.
#pragma once

#include "paged_internal.cuh"

namespace qsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr float kNoMax = -3.0e38f;         // no cell seen yet (below every score, and finite)

__device__ __forceinline__ uint32_t bits(__half2 h) {
  uint32_t u;
  memcpy(&u, &h, 4);
  return u;
}
__device__ __forceinline__ __half2 half2_of(uint32_t u) {
  __half2 h;
  memcpy(&h, &u, 4);
  return h;
}
// Bytes (i, j) of x as halves less `off` (bits of a half): a byte put under the exponent of 1024 is 1024 + it, exactly.
template <int kSel>
__device__ __forceinline__ __half2 bytes2(uint32_t x, uint32_t off) {
  return __hsub2(half2_of(__byte_perm(x, 0x64646464u, kSel)), half2_of(off));
}
// 2^x; results below the normal range are zero
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// The positions a group of tokens reads: [0, ns_al) (sinks, rounded up to whole
// blocks), then [lo_al, pmax] (lo rounded down).
struct Group {
  int t0, nt;          // tokens
  int seq;             // -1: nothing is visible
  int pmin, pmax;
  int lo, lo_al, ns_al;
  int nv, tiles;       // positions in order, tiles of them
};

// The position of a token, -1 if nothing is visible to it.
__device__ __forceinline__ int usable_pos(const PagedArgs& a, int s, int p) {
  return (unsigned)s < (unsigned)a.n_seq && p >= 0 && a.max_len > 0 ? (int)min((int64_t)p, a.max_len - 1) : -1;
}
__device__ __forceinline__ int token_pos(const PagedArgs& a, int t) { return usable_pos(a, a.tok_seq[t], a.tok_pos[t]); }
// Whether a token at p of sequence s starts a new run after one at q of sequence sq
// (runs: one sequence, positions close together).
__device__ __forceinline__ bool new_run(int s, int p, int sq, int q) {
  return p < 0 || q < 0 || s != sq || abs(p - q) > kPagedNear;
}

// Fills in what the tokens' number, sequence and positions decide.
template <int kCells>
__device__ __forceinline__ void reach(const PagedArgs& a, Group& g) {
  if (g.seq < 0) {
    g.lo = g.lo_al = g.ns_al = g.nv = 0;
    g.tiles = 1;
    return;
  }
  const int r = 1 << a.r_shift;
  g.lo = a.window > 0 ? max(0, g.pmin - a.window + 1) : 0;
  g.lo_al = g.lo & ~(r - 1);
  g.ns_al = (min(a.n_sink, g.lo) + r - 1) & ~(r - 1);
  if (g.ns_al >= g.lo_al) g.ns_al = g.lo_al = 0;   // one stretch
  g.nv = g.ns_al + g.pmax + 1 - g.lo_al;
  g.tiles = (g.nv + kCells - 1) / kCells;
}
__device__ __forceinline__ int pos_of(const Group& g, int v) { return v < g.ns_al ? v : v - g.ns_al + g.lo_al; }

// Shared memory that the plan takes while it is made, and where it leaves its parts.
constexpr int kPlanWords = kPagedPlan / 32;
constexpr int kPlanScratch = (3 * kPagedPlan + 3 * kPlanWords + 4) * 4;
constexpr int kLeaves = 1 << 30;   // beside a word's largest group: some tokens are the other launch's
// The tiles of a launch dealt to `parts` runs of them; what this CTA starts with.
struct Plan {
  int all, parts;      // tiles; parts that have any
  int u0, u1;          // this part's tiles
  int t0, first;       // the group of tile u0, and which of the group's tiles it is
};
template <bool kMixed>
struct PlanOf : Plan {};
template <>
struct PlanOf<true> : Plan {
  unsigned firsts[kPlanWords];   // the first tokens of this launch's groups
};
// The launch's group at token t or behind it.
template <bool kMixed>
__device__ __forceinline__ int next_group(const PagedArgs& a, const PlanOf<kMixed>& p, int t) {
  if constexpr (kMixed) {
    const int words = (a.n_tokens + 31) >> 5;
    int w = t >> 5;
    if (w >= words) return t;
    unsigned x = p.firsts[w] & (~0u << (t & 31));
    while (x == 0u && ++w < words) x = p.firsts[w];
    return x ? 32 * w + __ffs((int)x) - 1 : a.n_tokens;
  } else {
    return t;
  }
}

// all * part / parts, in 32 bits (part <= parts <= 2^15).
__device__ __forceinline__ int share_of(int all, int part, int parts) {
  const unsigned each = (unsigned)all / (unsigned)parts, rest = (unsigned)all % (unsigned)parts;
  return (int)(each * (unsigned)part + rest * (unsigned)part / (unsigned)parts);
}
// By all threads of a CTA.  `least`: tiles of a part, where that leaves a part a token.  `uncut`: groups of no more tiles
// are not shared by parts, as their join would take longer than their tiles (223 fp16 tokens of 255 positions 33 -> 19 us).
// Nor is any group where no part gets much more than its share for that (`more` tiles, what the join would take, which for
// more tokens than parts grows with them), so that nothing has to be joined (420 fp16 tokens of 700 43 -> 27 us, 3 x 900 of
// 1,000 110 -> 77, 35 x 8 of 500 q8_0 35 -> 29; whole all the same: 24 x 5 of 1,000 33 -> 42, 2 x 300 of 4,000 72 -> 79, 80
// tokens of 20,000 each 536 -> 782, of which some parts would have two).
// A warp takes 32 tokens at a time (a word of flags: which of them start a run); what crosses words is scanned by one warp.
// (4,096 tokens: 10 us, 512: 3, one: 1.)
// kMixed: of the runs in [run_lo + 1, run_hi] only.
template <int NT, int kCells, bool kMixed>
__device__ __forceinline__ void plan(const PagedArgs& a, int* scratch, PlanOf<kMixed>* out, int tid, int part, int max_parts, int least, int uncut,
                                     int more) {
  const int lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5, n = a.n_tokens, words = (n + 31) >> 5;
  int* seq = scratch;
  int* pos = seq + kPagedPlan;
  int* pre = pos + kPagedPlan;              // tiles of the word's groups up to and with each token
  unsigned* starts = reinterpret_cast<unsigned*>(pre + kPagedPlan);
  int* last = reinterpret_cast<int*>(starts + kPlanWords);   // the last start before each word
  int* sum = last + kPlanWords;             // tiles before each word, then all, and the largest group's
  if (kMixed && a.second && !*a.left) {   // nothing to do
    if (tid == 0) out->u0 = out->u1 = 0;
    __syncthreads();
    return;
  }
  Plan p;
  p.t0 = 0;
  int longest = 0;
  if (n == 1) {
    Group g;
    const int s = a.tok_seq[0];
    g.pmin = g.pmax = usable_pos(a, s, a.tok_pos[0]);
    g.seq = g.pmin < 0 ? -1 : s;
    reach<kCells>(a, g);
    p.all = g.tiles;
  } else {
#pragma unroll 4
    for (int t = tid; t < n; t += blockDim.x) {
      const int s = a.tok_seq[t], x = a.tok_pos[t];
      seq[t] = s;
      pos[t] = usable_pos(a, s, x);
    }
    __syncthreads();
    for (int w = warp; w < words; w += warps) {
      const int t = 32 * w + lane;
      const unsigned f = __ballot_sync(kFull, (kMixed && t >= n) || (t < n && (t == 0 || new_run(seq[t], pos[t], seq[t - 1], pos[t - 1]))));
      if (lane == 0) starts[w] = f;
    }
    __syncthreads();
    // the 32 tokens from t on: which start a run
    auto starts_from = [&](int t) {
      const int w = t >> 5;
      return __funnelshift_r(w < words ? starts[w] : ~0u, w + 1 < words ? starts[w + 1] : ~0u, t & 31);
    };
    // whether a run that starts at t is this launch's
    auto takes = [&](int t) {
      const unsigned f = starts_from(t + 1);
      const int len = f ? __ffs((int)f) : 33;   // (or more)
      return len > a.run_lo && len <= a.run_hi;
    };
    constexpr int kEach = kPlanWords / 32;   // words of a lane
    if (warp == 0) {
      int at[kEach], x = -1;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        const int w = kEach * lane + i;
        const unsigned f = w < words ? starts[w] : 0u;
        at[i] = x;
        if (f) x = 32 * w + 31 - __clz((int)f);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x = max(x, y);
      }
      const int before = __shfl_up_sync(kFull, x, 1);
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (kEach * lane + i < words) last[kEach * lane + i] = lane > 0 ? max(at[i], before) : at[i];
    }
    __syncthreads();
    for (int w = warp; w < words; w += warps) {
      const int t = 32 * w + lane;
      int m = 0;
      bool left = false;   // to the other launch
      Group g;
      if constexpr (NT == 1) {
        if (kMixed && t < n)   // (runs of at most two tokens: the first, or the second)
          left = starts[w] >> lane & 1u ? !takes(t) : a.run_hi < 2 || (starts_from(t - 1) & 7u) != 5u;
        if (t < n && !left) {
          g.pmin = g.pmax = pos[t];
          g.seq = g.pmin < 0 ? -1 : seq[t];
          reach<kCells>(a, g);
          m = g.tiles;
        }
      } else {
        const unsigned f = starts[w] & ((2u << lane) - 1u);
        const int r = f ? 32 * w + 31 - __clz((int)f) : last[w];
        unsigned groups = __ballot_sync(kFull, t < n && (t - r) % NT == 0);
        while (groups) {   // a group: its first token's lane, and a lane a token
          const int b = __ffs((int)groups) - 1, t0 = 32 * w + b, x = t0 + lane;
          groups &= groups - 1u;
          const unsigned cut = __ballot_sync(kFull, lane > 0 && (x >= n || (starts[x >> 5] >> (x & 31) & 1u)));
          const int len = min(cut ? __ffs((int)cut) - 1 : 32, NT), q = lane < len ? pos[x] : 0;
          if (kMixed && (starts[w] >> b & 1u ? !takes(t0) : a.run_hi <= NT)) {   // (a group further on: a run of more than NT)
            left = true;
            continue;
          }
          g.pmin = __reduce_min_sync(kFull, lane < len ? q : 0x7fffffff);
          g.pmax = __reduce_max_sync(kFull, lane < len ? q : -1);
          g.seq = g.pmin < 0 ? -1 : seq[t0];
          reach<kCells>(a, g);
          if (lane == b) m = g.tiles;
        }
      }
      const int top = __reduce_max_sync(kFull, m);
      const unsigned firsts = kMixed ? __ballot_sync(kFull, m > 0) : 0u, leaves = kMixed ? __ballot_sync(kFull, left) : 0u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, m, o);
        if (lane >= o) m += y;
      }
      if (t < n) pre[t] = m;
      if (lane == 31) {
        sum[w] = m;
        last[w] = top | (kMixed && leaves ? kLeaves : 0);   // (by now this word's last start has been read)
        if constexpr (kMixed) out->firsts[w] = firsts;
      }
    }
    __syncthreads();
    if (warp == 0) {
      int at[kEach], x = 0, top = 0;
      unsigned leaves = 0u;
#pragma unroll
      for (int i = 0; i < kEach; ++i) {
        at[i] = x;
        x += kEach * lane + i < words ? sum[kEach * lane + i] : 0;
        const int y = kEach * lane + i < words ? last[kEach * lane + i] : 0;
        top = max(top, kMixed ? y & (kLeaves - 1) : y);
        if (kMixed) leaves |= y & kLeaves;
      }
      top = __reduce_max_sync(kFull, top);
      if (kMixed && !a.second) {
        leaves = __reduce_or_sync(kFull, leaves);
        if (blockIdx.x == 0 && lane == 0) *a.left = leaves;
      }
      const int own = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, x, o);
        if (lane >= o) x += y;
      }
#pragma unroll
      for (int i = 0; i < kEach; ++i)
        if (kEach * lane + i < words) sum[kEach * lane + i] = at[i] + x - own;
      if (lane == 31) {
        sum[kPlanWords] = x;
        sum[kPlanWords + 1] = top;
      }
    }
    __syncthreads();
    p.all = sum[kPlanWords];
    longest = sum[kPlanWords + 1];
  }
  // each has a tile; no fewer than tokens, whose runs would each wait for memory (12 tokens of 4 positions 24 -> 13 us)
  p.parts = min(max_parts, max(p.all / least, min(n, p.all)));
  if (kMixed) p.parts = max(p.parts, 1);
  const int enough = p.all / p.parts + more;
  if (longest <= more) {   // (a part gets less than a group more than its share)
    uncut = max(uncut, longest);
  } else if (longest > uncut && longest <= enough) {   // what the parts would have if each began with a group: a thread each
    int* begins = seq;                                 // (free by now)
    for (int i = tid; i <= p.parts; i += blockDim.x) {
      const int u = share_of(p.all, i, p.parts);
      int w = 0, l = 0;   // the last token with no more than u tiles before it
#pragma unroll
      for (int s = kPlanWords / 2; s >= 1; s >>= 1)
        if (w + s < words && sum[w + s] <= u) w += s;
#pragma unroll
      for (int s = 16; s >= 1; s >>= 1)
        if (32 * w + l + s < n && sum[w] + pre[32 * w + l + s - 1] <= u) l += s;
      begins[i] = i == p.parts ? u : sum[w] + (l > 0 ? pre[32 * w + l - 1] : 0);
    }
    __syncthreads();
    int largest = 0;
    for (int i = lane; i < p.parts; i += 32) largest = max(largest, begins[i + 1] - begins[i]);
    if ((int)__reduce_max_sync(kFull, largest) <= enough) uncut = longest;
  }
  p.u0 = p.u1 = p.first = 0;
  if (warp == 0 && part < p.parts) {
    // tile u's group: its first token, its first tile, its tiles
    auto group_of = [&](int u, int& begin, int& tiles) {
      begin = 0;
      tiles = p.all;
      if (n == 1) return 0;
      int w = -1;   // the last token with no more than u tiles before it: its word, then its lane
#pragma unroll
      for (int i = 0; i < kPlanWords / 32; ++i)
        if (32 * i < words) w += __popc(__ballot_sync(kFull, 32 * i + lane < words && sum[32 * i + lane] <= u));
      const int t = 32 * w + lane, before = sum[w] + (lane > 0 && t < n ? pre[t - 1] : 0);
      const int l = __popc(__ballot_sync(kFull, t < n && before <= u)) - 1;
      begin = __shfl_sync(kFull, before, l);
      tiles = sum[w] + pre[32 * w + l] - begin;
      return 32 * w + l;
    };
    auto bound = [&](int u) {
      if (u >= p.all) return u;
      int begin, tiles;
      group_of(u, begin, tiles);
      return tiles <= uncut ? begin : u;
    };
    p.u0 = bound(share_of(p.all, part, p.parts));
    p.u1 = bound(share_of(p.all, part + 1, p.parts));
    int begin = 0, tiles;
    if (p.u0 < p.u1) p.t0 = group_of(p.u0, begin, tiles);
    p.first = p.u0 - begin;
  }
  if (tid == 0) static_cast<Plan&>(*out) = p;
  __syncthreads();   // the scratch is free
}

// A run of tiles of one group.
struct Run {
  Group g;
  int first, n;            // tiles first .. first + n - 1 of the group
  int64_t list, list_n;    // the sequence's part of seq_blk_slots
  unsigned bad;            // this lane's token of the group: what is wrong with it
};
// By a whole warp: tiles `first` and on, at most `most`, of the group that starts at token t0.
template <int NT, int kCells>
__device__ __forceinline__ Run run_at(const PagedArgs& a, int t0, int first, int most) {
  static_assert(NT <= 32, "a lane a token");
  const int lane = threadIdx.x & 31;
  Run r;
  const int t = t0 + lane;
  const bool have = lane < NT && t < a.n_tokens;
  const int s = have ? a.tok_seq[t] : -1, raw = have ? a.tok_pos[t] : -1, p = have ? usable_pos(a, s, raw) : -1;
  const int sq = __shfl_up_sync(kFull, s, 1), q = __shfl_up_sync(kFull, p, 1);
  const unsigned cut = __ballot_sync(kFull, lane > 0 && (!have || new_run(s, p, sq, q)));
  r.g.t0 = t0;
  r.g.nt = cut ? __ffs((int)cut) - 1 : NT;
  const bool in = lane < r.g.nt;
  r.g.pmin = __reduce_min_sync(kFull, in ? p : 0x7fffffff);
  r.g.pmax = __reduce_max_sync(kFull, in ? p : -1);
  r.g.seq = r.g.pmin < 0 ? -1 : __shfl_sync(kFull, s, 0);
  r.bad = !in ? 0u : (unsigned)s >= (unsigned)a.n_seq || raw < 0 ? kErrToken : raw >= a.max_len ? kErrMaxBlocks : 0u;
  reach<kCells>(a, r.g);
  r.first = first;
  r.n = min(most, r.g.tiles - first);
  r.list = r.list_n = 0;
  if (r.g.seq >= 0) {
    r.list = a.seq_blk_off[r.g.seq];
    r.list_n = a.seq_blk_off[r.g.seq + 1] - r.list;
    if (r.list < 0 || r.list_n < 0 || r.list + r.list_n > a.n_list) r.list_n = 0;
  }
  return r;
}
// By one warp of the KV head that reports: what is wrong with the group's tokens, and which parts share it (said at each
// of the group's tokens by the part where it starts, or by each of the parts but the last for itself, see PagedArgs).
__device__ __forceinline__ void announce(const PagedArgs& a, const Plan& p, const Run& r, int part, int u, unsigned* err) {
  const int lane = threadIdx.x & 31;
  if (r.first == 0 && r.bad) atomicOr(err, r.bad);
  const bool goes_on = r.first + r.n < r.g.tiles;
  if (a.span_by_token ? r.first != 0 : !goes_on) return;
  if (!goes_on) {
    if (lane < r.g.nt) a.span[r.g.t0 + lane] = make_int4(0, 0, 0, 0);
    return;
  }
  auto part_of = [&](int64_t tile) {
    int x = min((int)((float)tile * (float)p.parts / (float)p.all), p.parts - 1);   // off by one at most
    while (share_of(p.all, x + 1, p.parts) <= tile) ++x;
    while (share_of(p.all, x, p.parts) > tile) --x;
    return x;
  };
  const int64_t begin = (int64_t)u - r.first;
  const int4 span = make_int4(r.g.t0, r.g.nt | (a.kind << 8), r.first == 0 ? part : part_of(begin), part_of(begin + r.g.tiles - 1));
  if (a.span_by_token ? lane < r.g.nt : lane == 0) a.span[a.span_by_token ? r.g.t0 + lane : part] = span;
}
// The slot of the block of the group's position v (in reading order), -1: not read.
__device__ __forceinline__ int slot_at(const PagedArgs& a, const Run& r, int v, int v_end, bool report, unsigned* err) {
  if (v >= v_end) return -1;
  const int p = pos_of(r.g, v);
  if (p > r.g.pmax || (p >= a.n_sink && p < r.g.lo)) return -1;
  const int j = p >> a.r_shift;
  if (j < r.list_n) return a.seq_blk_slots[r.list + j];
  if (report) atomicOr(err, kErrBlockList);
  return -1;
}
__device__ __forceinline__ int cell_at(const PagedArgs& a, const Run& r, int v, int slot, bool report, unsigned* err) {
  if (slot < 0) return -1;
  if (slot >= a.n_slots) {
    if (report) atomicOr(err, kErrSlot);
    return -1;
  }
  return a.blk_cells[((int64_t)slot << a.r_shift) + (pos_of(r.g, v) & ((1 << a.r_shift) - 1))];
}
__device__ __forceinline__ int checked_cell(const PagedArgs& a, int c, bool report, unsigned* err) {
  if (c < a.n_cells) return c;
  if (report) atomicOr(err, kErrCell);
  return -1;
}

// Adds those of two halves that are infinite or NaN to (x, y).
__device__ __forceinline__ void add_not_finite(float& x, float& y, uint32_t w) {
  const float2 v = __half22float2(half2_of(w));
  if (!isfinite(v.x)) x += v.x;
  if (!isfinite(v.y)) y += v.y;
}

}  // namespace
}  // namespace qsa
