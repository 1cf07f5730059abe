// Upkeep of a cache's cells and blocks: reading rows back as values
// (qsa_kv_read), copying cells (qsa_cells_copy), sharing a sequence's blocks
// (qsa_seq_fork), and finding what the sequences still hold (qsa_cache_sweep),
// which frees the rest and can plan the moves that make the cache dense.
//
// llama.cpp issue #28734, fix summary: lever2b keeps each block's member cells
// in a device table, and lever2 names the operations that change them behind
// the indexer's back (defragmentation, rollback, sequence operations).
//
// No kernel here lets its successor launch early except the inner ones of the
// sweep: what they write (rows, block lists, free cells) may be an input that
// the next call reads before its dependency wait, so the next kernel may start
// only after the last CTA, and every CTA ends with a fence.
#include <atomic>

#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// ------------------------------------------------------------- qsa_kv_read
// One warp per (entry, K or V, KV head): lane l takes dims 8l .. 8l+7.
__global__ void __launch_bounds__(kThreads)
k_kv_read(const ReadArgs a, unsigned* err) {
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int rows = 2 * a.G;
  const int64_t i = w / rows;
  const int kind = (int)(w - i * rows);
  if (i >= a.n) return;
  const int64_t c = a.cells[i];
  if (c < 0) return;
  if (c >= a.n_cells) {
    if (lane == 0) atomicOr(err, kErrCell);
    return;
  }
  const int g = kind < a.G ? kind : kind - a.G;
  const unsigned char* cache = kind < a.G ? a.k_cache : a.v_cache;
  const int64_t cg = c * a.G + g, ncg = a.n_cells * a.G;
  uint4 o;
  __half2* h = reinterpret_cast<__half2*>(&o);
  if (a.kv_type == QSA_KV_F16) {
    o = reinterpret_cast<const uint4*>(cache + cg * (kHeadDim * 2))[lane];
  } else if (a.kv_type == QSA_KV_Q8_0) {
    const uint2 q = reinterpret_cast<const uint2*>(cache + cg * kHeadDim)[lane];
    const float d = __half2float(reinterpret_cast<const __half*>(cache + ncg * kHeadDim)[cg * 8 + (lane >> 2)]);
    const signed char* b = reinterpret_cast<const signed char*>(&q);
#pragma unroll
    for (int k = 0; k < 4; ++k) h[k] = __floats2half2_rn(d * (float)b[2 * k], d * (float)b[2 * k + 1]);
  } else {
    // value i of a block in the low nibble of byte i, value i + 16 in its high
    // nibble: lanes 0, 1 of a block's four take the low nibbles
    const uint2 q = *reinterpret_cast<const uint2*>(cache + cg * (kHeadDim / 2) + (lane >> 2) * 16 + (lane & 1) * 8);
    const float d = __half2float(reinterpret_cast<const __half*>(cache + ncg * (kHeadDim / 2))[cg * 8 + (lane >> 2)]);
    const int sh = (lane & 2) ? 4 : 0;
    const unsigned char* b = reinterpret_cast<const unsigned char*>(&q);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      h[k] = __floats2half2_rn(d * (float)((int)((b[2 * k] >> sh) & 15) - 8),
                               d * (float)((int)((b[2 * k + 1] >> sh) & 15) - 8));
  }
  __half* out = (kind < a.G ? a.k_out : a.v_out) + (i * a.G + g) * kHeadDim;
  reinterpret_cast<uint4*>(out)[lane] = o;
  __threadfence();
}

// ----------------------------------------------------------- qsa_cells_copy
// A cell is up to five contiguous runs of 16-byte chunks (K and V codes, K and
// V scales, the indexer key).  A lane keeps the addresses of its chunks of cell
// 0, at most kCopyBatch (all of a cell's for two fp16 heads), and a warp walks
// the pairs: the batch's loads, the next pair's cells, then the stores.
constexpr int kCopyBatch = 5;
constexpr int kCopyPerSm = 4;   // CTAs that share an SM

__global__ void __launch_bounds__(kThreads, kCopyPerSm)
k_cells_copy(const CopyArgs a, unsigned* err) {
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * kWarps, first = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int64_t n = a.n_dev ? min((int64_t)max(*a.n_dev, 0), (int64_t)a.n) : (int64_t)a.n;
  for (int c0 = 0; c0 < a.chunks; c0 += 32 * kCopyBatch) {
    unsigned char* at[kCopyBatch];
    unsigned pitch[kCopyBatch];   // 0: no such chunk
#pragma unroll
    for (int b = 0; b < kCopyBatch; ++b) {
      int c = c0 + b * 32 + lane;
      at[b] = nullptr;
      pitch[b] = 0u;
#pragma unroll
      for (int k = 0; k < 5; ++k) {
        if (pitch[b] == 0u && c < a.len[k]) {
          at[b] = a.base[k] + c * 16;
          pitch[b] = (unsigned)a.len[k] * 16u;
        }
        c -= a.len[k];
      }
    }
    int s = -1, d = -1;
    if (first < n) s = a.src[first], d = a.dst[first];
    for (int64_t i = first; i < n; i += warps) {
      const bool in = (unsigned)s < (unsigned)a.n_cells && (unsigned)d < (unsigned)a.n_cells;
      if (!in && s >= 0 && d >= 0 && lane == 0) atomicOr(err, kErrCell);
      uint4 v[kCopyBatch];
#pragma unroll
      for (int b = 0; b < kCopyBatch; ++b)
        if (in && pitch[b]) v[b] = *reinterpret_cast<const uint4*>(at[b] + (uint64_t)(unsigned)s * pitch[b]);
      const unsigned to = (unsigned)d;
      if (i + warps < n) s = a.src[i + warps], d = a.dst[i + warps];
#pragma unroll
      for (int b = 0; b < kCopyBatch; ++b)
        if (in && pitch[b]) *reinterpret_cast<uint4*>(at[b] + (uint64_t)to * pitch[b]) = v[b];
    }
  }
  __threadfence();
}

// ------------------------------------------------------------- qsa_seq_fork
// grid.y: the forks; grid.x: kForkPer list entries a thread; CTA x = 0 also
// writes the private tail block.  Every CTA checks the whole fork (a bad one
// changes nothing) and loads its entries before the checks that need the
// tables have come back.
constexpr int kForkPer = 4;

__global__ void __launch_bounds__(kThreads)
k_seq_fork(const ForkArgs a, unsigned* err) {
  grid_dep_wait();
  const int tid = threadIdx.x, f = blockIdx.y, r = a.r;
  const int64_t j0 = (int64_t)blockIdx.x * (kThreads * kForkPer) + tid;
  const int s = a.src_seq[f], d = a.dst_seq[f], p = a.n_pos[f], ts = a.tail_slot[f];
  unsigned bad = 0u;
  int64_t so = 0, to = 0;
  int nb = 0, tail = 0, slot = -1;
  int64_t list = 0;            // entries of dst's list
  int v[kForkPer];
  float w[kForkPer];
  if (s < 0 || s >= a.n_seq || d < 0 || d >= a.n_seq || p < 0) {
    bad = kErrToken;
  } else {
    nb = p / r;
    tail = p - nb * r;
    so = a.seq_blk_off[s];
    to = a.seq_blk_off[d];
    const int64_t need = nb + (tail > 0 ? 1 : 0), sl = a.seq_blk_off[s + 1], tl = a.seq_blk_off[d + 1];
    list = tl - to;
    if (nb > a.max_blocks) bad |= kErrMaxBlocks;
    if (so < 0 || to < 0 || sl > a.n_list || tl > a.n_list || so + need > sl || to + need > tl) bad |= kErrBlockList;
    if (!bad) {
#pragma unroll
      for (int i = 0; i < kForkPer; ++i)
        if (j0 + i * kThreads < nb) {
          v[i] = a.seq_blk_slots[so + j0 + i * kThreads];
          w[i] = a.block_weight ? a.block_weight[so + j0 + i * kThreads] : 0.f;
        }
    }
    if (!bad && tail > 0) {
      slot = a.seq_blk_slots[so + nb];
      if (slot < 0 || slot >= a.n_slots || ts < 0 || ts >= a.n_slots || slot == ts) bad |= kErrSlot;
      for (int x = 0; x < tail && !(bad & kErrSlot); ++x) {
        const int c = a.tail_cells[(int64_t)f * r + x], o = a.blk_cells[(int64_t)slot * r + x];
        if (c < 0 || c >= a.n_cells || o < 0 || o >= a.n_cells) bad |= kErrCell;
      }
    }
  }
  if (blockIdx.x == 0) {
    // A sequence forked onto itself gets a tail of its own: the tail's list
    // entry is both read above and written below.  This CTA's threads have all
    // read it at the barrier; in the other CTAs either value leads to the same
    // whole blocks (copied onto themselves).
    __syncthreads();
    if (bad && tid == 0) atomicOr(err, bad);
    if (tid < r) {
      const bool has = !bad && tid < tail;
      const int from = has ? a.blk_cells[(int64_t)slot * r + tid] : -1;
      const int cell = has ? a.tail_cells[(int64_t)f * r + tid] : -1;
      a.copy_src[(int64_t)f * r + tid] = from;
      a.copy_dst[(int64_t)f * r + tid] = cell;
      if (!bad && tail > 0) {
        a.blk_cells[(int64_t)ts * r + tid] = cell;
        if (tid == 0) {
          a.slot_block_idx[ts] = max(nb, a.slot_block_idx[slot]);   // (after an eviction past its place in the list)
          a.seq_blk_slots[to + nb] = ts;
        }
      }
    }
  }
  if (!bad) {
#pragma unroll
    for (int i = 0; i < kForkPer; ++i)
      if (j0 + i * kThreads < nb) {
        a.seq_blk_slots[to + j0 + i * kThreads] = v[i];
        if (a.block_weight) a.block_weight[to + j0 + i * kThreads] = w[i];
      }
    // the whole blocks' weights go along; the tail's and those to come begin anew
    if (a.block_weight)
      for (int64_t j = nb + (int64_t)blockIdx.x * kThreads + tid; j < list; j += (int64_t)gridDim.x * kThreads) a.block_weight[to + j] = 0.f;
  }
  __threadfence();
}

// ---------------------------------------------------------- qsa_cache_sweep
// Five phases, each a loop over all threads (or, by tiles of 4,096 cells or
// slots, over all CTAs) of whatever runs it:
//   clear   a bit of every cell and slot
//   mark    a thread per list entry: the slot it names is held while the
//           sequence's positions reach its block, and with it the cells of
//           those positions
//   count   held cells and slots of each tile
//   apply   ranks: free lists, moves, cell_map
//   table   the block table under the new places (without compaction the bits
//           say all it needs, so it does not wait for the counts)
// A small cache is swept by one cluster with its hardware barrier between the
// phases, one launch in all; a large one by kernels of their own over the whole GPU.
constexpr int kSweepThreads = 1024, kSweepWarps = kSweepThreads / 32;
constexpr int kTile = 4 * kSweepThreads;        // a thread's four cells or slots of a tile
constexpr int kTileWords = kTile / 32;
// Threads of a CTA that walks list entries or table rows by itself: these wait on
// scattered accesses, and small CTAs leave no SM with a second wave of them
// (1.25M cells, 1,024 threads: 23.0 us, compacting 30.9; 256: 22.0 and 29.5).
// The ranks are faster with 1,024 (512: 22.9 and 32.4, as a thread's stores of
// eight cells spread over more lines).
constexpr int kSweepRows = 256;
constexpr int kSweepCluster = 16;
// A cluster sweeps caches of up to so many cells, list entries and slots.  The
// host makes one launch instead of four or five, which is what such a call waits
// for (us a call, cluster / kernels of their own, compacting: 11.1 / 21.1 at 5,000
// cells, 12.6 / 20.4 at 50,000, 14.9 / 20.1 at 65,536); in a graph the device
// takes 9.9 / 10.5, 12.3 / 13.8 and 14.7 / 13.9.
constexpr int64_t kSweepClusterCells = 65536;
constexpr int kSweepSeqs = 256;                 // sequences whose lists a CTA keeps in shared memory

struct SweepSmem {
  unsigned tmp[2][kSweepWarps];
  int64_t off[kSweepSeqs + 1];
  int len[kSweepSeqs];
};

__device__ __forceinline__ void sweep_clear(const SweepArgs& a, int64_t i0, int64_t n) {
  uint4* p = reinterpret_cast<uint4*>(a.cell_bits);   // the slots' bits follow
  const int64_t all = (a.cell_tiles + a.slot_tiles) * (kTileWords / 4);
  for (int64_t i = i0; i < all; i += n) p[i] = make_uint4(0u, 0u, 0u, 0u);
}

// The sequences' lists and lengths, from shared memory where they fit.
struct SweepSeqs {
  const int64_t* off;
  const int32_t* len;
  int64_t lists, end;   // list entries; the loop's end (every sequence is looked at, too)
};
__device__ __forceinline__ SweepSeqs sweep_seqs(const SweepArgs& a, SweepSmem& sm) {
  const bool near = a.n_seq <= kSweepSeqs;
  if (near) {
    for (int i = threadIdx.x; i <= a.n_seq; i += blockDim.x) {
      sm.off[i] = a.seq_blk_off[i];
      if (i < a.n_seq) sm.len[i] = a.seq_len[i];
    }
    __syncthreads();
  }
  SweepSeqs q;
  q.off = near ? sm.off : a.seq_blk_off;
  q.len = near ? sm.len : a.seq_len;
  q.lists = q.off[a.n_seq] < a.n_list ? q.off[a.n_seq] : a.n_list;
  q.end = q.lists > a.n_seq ? q.lists : a.n_seq;
  return q;
}

// What list entry e marks: its slot (-1: nothing) and the first `held` cells of
// the slot's row.  `slot` is the entry's, loaded by the caller.
struct SweepEntry {
  int slot;
  int64_t held;
  int c[8];   // compress_ratio is at most 8
};
__device__ __forceinline__ SweepEntry sweep_entry(const SweepArgs& a, const SweepSeqs& q, int64_t e, int slot, unsigned* err) {
  SweepEntry r;
  r.slot = -1;
  r.held = 0;
  if (e < a.n_seq) {   // a length that its list, as far as it is there, cannot hold
    const int64_t end = q.off[e + 1] < a.n_list ? q.off[e + 1] : a.n_list;
    if (q.len[e] > 0 && (q.len[e] + (int64_t)a.r - 1) / a.r > end - q.off[e]) atomicOr(err, kErrBlockList);
  }
  if (e >= q.lists || e < q.off[0]) return r;
  int lo = 0, hi = a.n_seq;                   // the last sequence whose list starts at or before e
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (q.off[mid] <= e) lo = mid;
    else hi = mid;
  }
  r.held = q.len[lo] - (e - q.off[lo]) * a.r;
  if (r.held <= 0) return r;
  if (slot < 0 || slot >= a.n_slots) {
    atomicOr(err, kErrSlot);
    return r;
  }
  r.slot = slot;
  const int32_t* row = a.blk_cells + (int64_t)slot * a.r;
  if (a.r == 4 && a.rows16) {
    const int4 v = *reinterpret_cast<const int4*>(row);
    r.c[0] = v.x, r.c[1] = v.y, r.c[2] = v.z, r.c[3] = v.w;
#pragma unroll
    for (int i = 4; i < 8; ++i) r.c[i] = -1;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.c[i] = i < a.r ? row[i] : -1;
  }
  return r;
}
__device__ __forceinline__ void sweep_flag(const SweepArgs& a, const SweepEntry& r, unsigned* cell_bits,
                                           unsigned* slot_bits, unsigned* err) {
  if (r.slot < 0) return;
  atomicOr(&slot_bits[r.slot >> 5], 1u << (r.slot & 31));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (i >= r.held || r.c[i] < 0) continue;
    if (r.c[i] >= a.n_cells) atomicOr(err, kErrCell);
    else atomicOr(&cell_bits[r.c[i] >> 5], 1u << (r.c[i] & 31));
  }
}
__device__ __forceinline__ void sweep_mark(const SweepArgs& a, const SweepSeqs& q, int64_t i0, int64_t n,
                                           unsigned* cell_bits, unsigned* slot_bits, unsigned* err) {
  for (int64_t e = i0; e < q.end; e += n)
    sweep_flag(a, sweep_entry(a, q, e, e < q.lists ? a.seq_blk_slots[e] : -1, err), cell_bits, slot_bits, err);
}

// This thread's four bits of a tile.
__device__ __forceinline__ unsigned sweep_bits(const SweepArgs& a, int64_t tile) {
  return (__ldcg(a.cell_bits + tile * kTileWords + (threadIdx.x >> 3)) >> (4 * (threadIdx.x & 7))) & 15u;
}

// Sums of x and of y over the CTA, in every thread.
__device__ __forceinline__ uint2 block_sums(unsigned x, unsigned y, SweepSmem& sm) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  x = __reduce_add_sync(kFull, x);
  y = __reduce_add_sync(kFull, y);
  __syncthreads();
  if (lane == 0) sm.tmp[0][warp] = x, sm.tmp[1][warp] = y;
  __syncthreads();
  static_assert(kSweepWarps == 32, "one partial per lane");
  return make_uint2(__reduce_add_sync(kFull, sm.tmp[0][lane]), __reduce_add_sync(kFull, sm.tmp[1][lane]));
}

// Tiles [0, cell_tiles) are cells', the others slots' (whose bits follow).
// Ranks of tile t, of which this thread's bits are w; all_sums: every tile's sum, in global
// memory or (kNear) shared.  In a compaction a held cell at or past n_held is
// written to cell_map as -2 - (its move's number); sweep_table resolves it.
template <bool kNear>
__device__ __forceinline__ void sweep_apply(const SweepArgs& a, int64_t t, unsigned w, const unsigned* all_sums,
                                            SweepSmem& sm) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto sum_of = [&](const unsigned* p) { return kNear ? *p : __ldcg(p); };
  {
    const bool cells = t < a.cell_tiles;
    const int64_t tile = cells ? t : t - a.cell_tiles, tiles = cells ? a.cell_tiles : a.slot_tiles;
    const unsigned* sums = all_sums + (cells ? 0 : a.cell_tiles);
    unsigned before = 0, all = 0;
    for (int64_t k = tid; k < tiles; k += kSweepThreads) {
      const unsigned v = sum_of(sums + k);
      all += v;
      if (k < tile) before += v;
    }
    const uint2 s2 = block_sums(before, all, sm);
    const int64_t n_held = s2.y;
    // held cells below n_held: the movers' ranks start there
    unsigned below = 0;
    if (cells && a.compact) {
      const int64_t cut = n_held / kTile;
      for (int64_t k = tid; k < cut; k += kSweepThreads) below += sum_of(sums + k);
      if (cut < tiles) {
        const unsigned v = sweep_bits(a, cut);
        const int in = (int)(n_held - cut * kTile) - 4 * tid;   // of this thread's four cells
        if (in > 0) below += __popc(in >= 4 ? v : v & ((1u << in) - 1u));
      }
    }
    // this thread's rank: the tiles before, the warps before, the lanes before
    unsigned incl = __popc(w);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += y;
    }
    below = __reduce_add_sync(kFull, below);
    __syncthreads();
    if (lane == 31) sm.tmp[0][warp] = incl;
    if (lane == 0) sm.tmp[1][warp] = below;
    __syncthreads();
    below = __reduce_add_sync(kFull, sm.tmp[1][lane]);
    int64_t rk = s2.x + __reduce_add_sync(kFull, lane < warp ? sm.tmp[0][lane] : 0u) + incl - __popc(w);
    if (tid == 0 && tile == 0) {
      if (cells) {
        a.counts[0] = (int)n_held;
        a.counts[1] = (int)(a.n_cells - n_held);
        a.counts[3] = a.compact ? (int)(n_held - below) : 0;
      } else {
        a.counts[2] = (int)(a.n_slots - n_held);
      }
    }
    const int64_t c0 = tile * kTile + 4 * tid, n_of = cells ? a.n_cells : a.n_slots;
    int map[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t c = c0 + i;
      const bool held = (w >> i) & 1u;
      map[i] = held ? (int)c : -1;
      if (c >= n_of) continue;
      if (!cells) {
        if (!held && a.free_slots) a.free_slots[c - rk] = (int)c;
      } else if (a.compact) {
        if (held && c >= n_held) {
          const int64_t k = rk - below;
          a.move_src[k] = (int)c;
          map[i] = (int)(-2 - k);
        }
        if (!held && c < n_held) a.move_dst[c - rk] = (int)c;
        if (c >= n_held && a.free_cells) a.free_cells[c - n_held] = (int)c;
      } else if (!held && a.free_cells) {
        a.free_cells[c - rk] = (int)c;
      }
      rk += held;
    }
    if (cells && a.cell_map) {
      if (a.map16 && c0 + 4 <= n_of) {
        *reinterpret_cast<int4*>(a.cell_map + c0) = make_int4(map[0], map[1], map[2], map[3]);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (c0 + i < n_of) a.cell_map[c0 + i] = map[i];
      }
    }
  }
}

// The block table without what nobody holds, under the cells' new places; and
// the movers' entries of cell_map (either form of an entry gives its place, so
// the two may meet).
__device__ __forceinline__ void sweep_table(const SweepArgs& a, int64_t i0, int64_t n) {
  const int64_t moves = a.compact ? __ldcg(a.counts + 3) : 0;
  auto place = [&](int c) -> int {
    if (c < 0 || c >= a.n_cells) return -1;
    if (!a.compact) return (__ldcg(a.cell_bits + (c >> 5)) >> (c & 31)) & 1u ? c : -1;
    const int v = *reinterpret_cast<volatile const int32_t*>(a.cell_map + c);
    return v < -1 ? __ldcg(a.move_dst + (-2 - v)) : v;
  };
  for (int64_t slot = i0; slot < a.n_slots; slot += n) {
    const bool held = (__ldcg(a.slot_bits + (slot >> 5)) >> (slot & 31)) & 1u;
    const int32_t* row = a.blk_cells + slot * a.r;
    int32_t* out = a.blk_cells_out + slot * a.r;
    if (a.r == 4 && a.rows16) {
      const int4 v = *reinterpret_cast<const int4*>(row);
      int4 o = make_int4(-1, -1, -1, -1);
      if (held) o = make_int4(place(v.x), place(v.y), place(v.z), place(v.w));
      *reinterpret_cast<int4*>(out) = o;
    } else {
      for (int i = 0; i < a.r; ++i) out[i] = held ? place(row[i]) : -1;
    }
  }
  for (int64_t k = i0; k < moves; k += n)
    *reinterpret_cast<volatile int32_t*>(a.cell_map + __ldcg(a.move_src + k)) = __ldcg(a.move_dst + k);
}

__device__ __forceinline__ int64_t grid_thread() { return (int64_t)blockIdx.x * blockDim.x + threadIdx.x; }
__device__ __forceinline__ int64_t grid_threads() { return (int64_t)gridDim.x * blockDim.x; }

__global__ void __launch_bounds__(kSweepThreads) k_sweep_clear(const SweepArgs a) {
  grid_dep_wait();
  grid_dep_launch();
  sweep_clear(a, grid_thread(), grid_threads());
}
__global__ void __launch_bounds__(kSweepRows) k_sweep_mark(const SweepArgs a, unsigned* err) {
  __shared__ SweepSmem sm;
  grid_dep_wait();
  grid_dep_launch();
  sweep_mark(a, sweep_seqs(a, sm), grid_thread(), grid_threads(), a.cell_bits, a.slot_bits, err);
}
__global__ void __launch_bounds__(kSweepThreads) k_sweep_count(const SweepArgs a) {
  __shared__ SweepSmem sm;
  grid_dep_wait();
  grid_dep_launch();
  const uint2 sum = block_sums(__popc(sweep_bits(a, blockIdx.x)), 0u, sm);
  if (threadIdx.x == 0) a.sums[blockIdx.x] = sum.x;
}
__global__ void __launch_bounds__(kSweepThreads) k_sweep_apply(const SweepArgs a) {
  __shared__ SweepSmem sm;
  grid_dep_wait();
  if (a.compact) grid_dep_launch();   // else this is the last kernel
  else sweep_table(a, grid_thread(), grid_threads());
  sweep_apply<false>(a, blockIdx.x, sweep_bits(a, blockIdx.x), a.sums, sm);
  __threadfence();
}
__global__ void __launch_bounds__(kSweepRows) k_sweep_table(const SweepArgs a) {
  grid_dep_wait();
  sweep_table(a, grid_thread(), grid_threads());
  __threadfence();
}
// All of it by one cluster.  Every CTA marks its entries in bits of its own, in
// shared memory (50,000 cells: 62,500 atomics that cross no network); the CTA of
// a tile (each has at most kNearTiles) joins the 16 CTAs' bits of it, keeps them
// in registers, writes them out for the table, and puts the tile's sum straight
// into every CTA's shared memory.
constexpr int kNearTiles = (int)(2 * (kSweepClusterCells / kTile) / kSweepCluster);
__global__ void __launch_bounds__(kSweepThreads) k_sweep_cluster(const SweepArgs a, unsigned* err) {
  __shared__ SweepSmem sm;
  __shared__ unsigned s_sums[kNearTiles * kSweepCluster];
  __shared__ alignas(16) unsigned s_bits[kNearTiles * kSweepCluster * kTileWords];   // cells, then slots, as in the workspace
  static_assert(kNearTiles * kSweepCluster * (int64_t)kTile >= 2 * kSweepClusterCells, "every tile has a CTA");
  static_assert(sizeof(s_bits) == 16 * kSweepThreads, "a thread clears 16 bytes");
  static_assert(kSweepCluster == 16 && kTileWords * 8 == kSweepThreads, "eight threads a word join two CTAs' each");
  grid_dep_wait();
  // warps dealt to the CTAs in turn: a small cache keeps all 16 SMs busy
  const int64_t n = grid_threads();
  const int64_t i0 = ((int64_t)(threadIdx.x >> 5) * kSweepCluster + blockIdx.x) * 32 + (threadIdx.x & 31);
  const int slot0 = i0 < a.n_list ? a.seq_blk_slots[i0] : -1;
  reinterpret_cast<uint4*>(s_bits)[threadIdx.x] = make_uint4(0u, 0u, 0u, 0u);
  const SweepSeqs q = sweep_seqs(a, sm);
  SweepEntry first;
  first.slot = -1;
  if (i0 < q.end) first = sweep_entry(a, q, i0, slot0, err);
  __syncthreads();
  unsigned* slot_bits = s_bits + a.cell_tiles * kTileWords;
  sweep_flag(a, first, s_bits, slot_bits, err);
  sweep_mark(a, q, i0 + n, n, s_bits, slot_bits, err);
  __syncwarp();
  cluster_sync();
  unsigned w[kNearTiles];
  const int tiles = (int)(a.cell_tiles + a.slot_tiles), part = threadIdx.x & 7;
#pragma unroll
  for (int k = 0; k < kNearTiles; ++k) {
    const int t = (int)blockIdx.x + k * kSweepCluster;
    const unsigned* word = s_bits + t * kTileWords + (threadIdx.x >> 3);
    w[k] = t < tiles ? ld_dsmem_u32v(dsmem_addr(word, 2 * part)) | ld_dsmem_u32v(dsmem_addr(word, 2 * part + 1)) : 0u;
  }
#pragma unroll
  for (int k = 0; k < kNearTiles; ++k) {
    const int t = (int)blockIdx.x + k * kSweepCluster;
#pragma unroll
    for (int o = 1; o <= 4; o <<= 1) w[k] |= __shfl_xor_sync(kFull, w[k], o);
    if (t < tiles && part == 0) a.cell_bits[t * kTileWords + (threadIdx.x >> 3)] = w[k];
    w[k] = (w[k] >> (4 * part)) & 15u;
    const uint2 sum = block_sums(__popc(w[k]), 0u, sm);
    if (t < tiles && threadIdx.x < kSweepCluster) st_dsmem_u32(dsmem_addr(&s_sums[t], threadIdx.x), sum.x);
  }
  cluster_sync();   // also: nobody touches a peer after this
  if (!a.compact) sweep_table(a, i0, n);
#pragma unroll
  for (int k = 0; k < kNearTiles; ++k) {
    const int t = (int)blockIdx.x + k * kSweepCluster;
    if (t < tiles) sweep_apply<true>(a, t, w[k], s_sums, sm);
  }
  if (a.compact) {
    __syncwarp();
    cluster_sync();
    sweep_table(a, i0, n);
  }
  __threadfence();
}

}  // namespace

cudaError_t launch_kv_read(const ReadArgs& a, unsigned* err, cudaStream_t stream) {
  if (a.n <= 0) return cudaSuccess;
  const int64_t warps = (int64_t)a.n * 2 * a.G;
  prof_before(kKRead, stream);
  cudaError_t e = launch_pdl(k_kv_read, dim3((unsigned)ceil_div(warps, kWarps)), dim3(kThreads), 0, stream, 1, a, err);
  prof_after(kKRead, stream);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_cells_copy(const CopyArgs& a, unsigned* err, cudaStream_t stream) {
  if (a.n <= 0) return cudaSuccess;
  prof_before(kKCopy, stream);
  const int64_t ctas = ceil_div(a.n, kWarps);
  constexpr int64_t kResident = 152 * kCopyPerSm;
  cudaError_t e = launch_pdl(k_cells_copy, dim3((unsigned)(ctas < kResident ? ctas : kResident)), dim3(kThreads), 0,
                             stream, 1, a, err);
  prof_after(kKCopy, stream);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

cudaError_t launch_seq_fork(const ForkArgs& a, unsigned* err, cudaStream_t stream) {
  if (a.n <= 0) return cudaSuccess;
  const int64_t x = ceil_div(a.max_blocks > 0 ? a.max_blocks : 1, kThreads * kForkPer);
  prof_before(kKFork, stream);
  cudaError_t e = launch_pdl(k_seq_fork, dim3((unsigned)x, (unsigned)a.n), dim3(kThreads), 0, stream, 1, a, err);
  prof_after(kKFork, stream);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// A CTA a sequence: the weights of the entries behind its blocks.
__global__ void __launch_bounds__(kThreads) k_weight_trim(const int32_t* seq_len, const int64_t* seq_blk_off, int r, int64_t n_list,
                                                          float* block_weight, unsigned* err) {
  grid_dep_wait();
  const int s = blockIdx.x, len = seq_len[s];
  const int64_t off = seq_blk_off[s], end = seq_blk_off[s + 1];
  if (off < 0 || end < off || end > n_list) {
    if (threadIdx.x == 0) atomicOr(err, kErrBlockList);
    return;
  }
  const int64_t held = len > 0 ? ((int64_t)len + r - 1) / r : 0;
  for (int64_t j = off + held + threadIdx.x; j < end; j += kThreads) block_weight[j] = 0.f;
}
cudaError_t launch_weight_trim(const int32_t* seq_len, const int64_t* seq_blk_off, int n_seq, int r, int64_t n_list, float* block_weight,
                               unsigned* err, cudaStream_t stream) {
  return launch_pdl(k_weight_trim, dim3((unsigned)n_seq), dim3(kThreads), 0, stream, 1, seq_len, seq_blk_off, r, n_list, block_weight,
                    err);
}

// Workspace: the cells' bits and the slots', in whole tiles, then the tiles' sums.
static int64_t sweep_tiles(int64_t n) { return ceil_div(n > 0 ? n : 1, kTile); }
size_t sweep_workspace_bytes(int64_t n_cells, int64_t n_slots) {
  const int64_t tiles = sweep_tiles(n_cells) + sweep_tiles(n_slots);
  return (size_t)round_up(tiles * (kTileWords * 4) + tiles * 4, 256);
}

// Clusters of kSweepCluster CTAs can run on the current device (asked once per device).
static cudaError_t sweep_cluster_ok(bool* ok) {
  constexpr int kMaxDevices = 64;
  static std::atomic<int> known[kMaxDevices];   // 0: not asked, 1: no, 2: yes
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  int k = known[dev].load(std::memory_order_acquire);
  if (k == 0) {
    k = 1;
    if (cudaFuncSetAttribute(k_sweep_cluster, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess) {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(kSweepCluster);
      cfg.blockDim = dim3(kSweepThreads);
      cudaLaunchAttribute attr;
      attr.id = cudaLaunchAttributeClusterDimension;
      attr.val.clusterDim.x = kSweepCluster;
      attr.val.clusterDim.y = 1;
      attr.val.clusterDim.z = 1;
      cfg.attrs = &attr;
      cfg.numAttrs = 1;
      int n = 0;
      if (cudaOccupancyMaxActiveClusters(&n, k_sweep_cluster, &cfg) == cudaSuccess && n > 0) k = 2;
    }
    (void)cudaGetLastError();
    known[dev].store(k, std::memory_order_release);
  }
  *ok = k == 2;
  return cudaSuccess;
}

cudaError_t launch_cache_sweep(const SweepArgs& args, void* ws, unsigned* err, cudaStream_t stream) {
  SweepArgs a = args;
  a.cell_tiles = sweep_tiles(a.n_cells);
  a.slot_tiles = sweep_tiles(a.n_slots);
  a.cell_bits = static_cast<unsigned*>(ws);
  a.slot_bits = a.cell_bits + a.cell_tiles * kTileWords;
  const int64_t tiles = a.cell_tiles + a.slot_tiles;
  a.sums = a.cell_bits + tiles * kTileWords;
  a.rows16 = ((reinterpret_cast<uintptr_t>(a.blk_cells) | reinterpret_cast<uintptr_t>(a.blk_cells_out)) & 15u) == 0u;
  a.map16 = (reinterpret_cast<uintptr_t>(a.cell_map) & 15u) == 0u;
  const dim3 block(kSweepThreads);
  const dim3 rows(kSweepRows);
  auto grid = [](int64_t n, int threads) { return dim3((unsigned)ceil_div(n > 0 ? n : 1, threads)); };
  bool cluster = false;
  if (a.n_cells <= kSweepClusterCells && a.n_list <= kSweepClusterCells && a.n_slots <= kSweepClusterCells) {
    const cudaError_t e = sweep_cluster_ok(&cluster);
    if (e != cudaSuccess) return e;
  }
  const int64_t entries = a.n_list > a.n_seq ? a.n_list : a.n_seq;
  prof_before(kKSweep, stream);
  cudaError_t e;
  if (cluster) {
    e = launch_pdl(k_sweep_cluster, dim3(kSweepCluster), block, 0, stream, kSweepCluster, a, err);
  } else {
    e = launch_pdl(k_sweep_clear, grid(tiles * (kTileWords / 4), kSweepThreads), block, 0, stream, 1, a);
    if (e == cudaSuccess) e = launch_pdl(k_sweep_mark, grid(entries, kSweepRows), rows, 0, stream, 1, a, err);
    if (e == cudaSuccess) e = launch_pdl(k_sweep_count, dim3((unsigned)tiles), block, 0, stream, 1, a);
    if (e == cudaSuccess) e = launch_pdl(k_sweep_apply, dim3((unsigned)tiles), block, 0, stream, 1, a);
    if (e == cudaSuccess && a.compact) e = launch_pdl(k_sweep_table, grid(a.n_slots, kSweepRows), rows, 0, stream, 1, a);
  }
  prof_after(kKSweep, stream);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace qsa
