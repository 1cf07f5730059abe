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
// grid.y: the forks; grid.x: 256 list entries each; CTA x = 0 also writes the
// private tail block.
__global__ void __launch_bounds__(kThreads)
k_seq_fork(const ForkArgs a, unsigned* err) {
  grid_dep_wait();
  const int tid = threadIdx.x, f = blockIdx.y, r = a.r;
  const int64_t j = (int64_t)blockIdx.x * kThreads + tid;
  const int s = a.src_seq[f], d = a.dst_seq[f], p = a.n_pos[f];
  unsigned bad = 0u;
  int64_t so = 0, to = 0;
  int nb = 0, tail = 0, slot = -1, ts = -1;
  if (s < 0 || s >= a.n_seq || d < 0 || d >= a.n_seq || p < 0) {
    bad = kErrToken;
  } else {
    nb = p / r;
    tail = p - nb * r;
    so = a.seq_blk_off[s];
    to = a.seq_blk_off[d];
    const int64_t need = nb + (tail > 0 ? 1 : 0), sl = a.seq_blk_off[s + 1], tl = a.seq_blk_off[d + 1];
    if (nb > a.max_blocks) bad |= kErrMaxBlocks;
    if (so < 0 || to < 0 || sl > a.n_list || tl > a.n_list || so + need > sl || to + need > tl) bad |= kErrBlockList;
    if (!bad && tail > 0) {
      slot = a.seq_blk_slots[so + nb];
      ts = a.tail_slot[f];
      if (slot < 0 || slot >= a.n_slots || ts < 0 || ts >= a.n_slots || slot == ts) bad |= kErrSlot;
      for (int x = 0; x < tail && !bad; ++x) {
        const int c = a.tail_cells[(int64_t)f * r + x], o = a.blk_cells[(int64_t)slot * r + x];
        if (c < 0 || c >= a.n_cells || o < 0 || o >= a.n_cells) bad |= kErrCell;
      }
    }
  }
  // A sequence forked onto itself gets a tail of its own: the tail's list entry
  // is both read above and written below.  This CTA's threads have all read it
  // at the barrier; in the other CTAs either value leads to the same whole
  // blocks (copied onto themselves).
  __syncthreads();
  if (bad && blockIdx.x == 0 && tid == 0) atomicOr(err, bad);
  if (blockIdx.x == 0 && tid < r) {
    const bool has = !bad && tid < tail;
    const int from = has ? a.blk_cells[(int64_t)slot * r + tid] : -1;
    const int cell = has ? a.tail_cells[(int64_t)f * r + tid] : -1;
    a.copy_src[(int64_t)f * r + tid] = from;
    a.copy_dst[(int64_t)f * r + tid] = cell;
    if (!bad && tail > 0) {
      a.blk_cells[(int64_t)ts * r + tid] = cell;
      if (tid == 0) a.slot_block_idx[ts] = nb;
    }
  }
  if (bad) return;
  if (j < nb) a.seq_blk_slots[to + j] = a.seq_blk_slots[so + j];
  if (tail > 0 && blockIdx.x == 0 && tid == 0) a.seq_blk_slots[to + nb] = ts;
  __threadfence();
}

// ---------------------------------------------------------- qsa_cache_sweep
constexpr int kTileWords = 256;              // bitmap words of one CTA: 8,192 cells or slots

__global__ void __launch_bounds__(kThreads) k_sweep_clear(uint4* bits, int64_t n16) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < n16) bits[i] = make_uint4(0u, 0u, 0u, 0u);
}

// One thread per list entry: the slot it names is held while the sequence's
// positions reach its block, and with it the cells of those positions.
__global__ void __launch_bounds__(kThreads) k_sweep_mark(const SweepArgs a, unsigned* err) {
  grid_dep_wait();
  grid_dep_launch();
  const int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (e < a.n_seq) {   // a length that its list cannot hold
    const int64_t cap = a.seq_blk_off[e + 1] - a.seq_blk_off[e];
    if (a.seq_len[e] > 0 && (a.seq_len[e] + (int64_t)a.r - 1) / a.r > cap) atomicOr(err, kErrBlockList);
  }
  if (e >= a.n_list || e < a.seq_blk_off[0] || e >= a.seq_blk_off[a.n_seq]) return;
  int lo = 0, hi = a.n_seq;                   // the last sequence whose list starts at or before e
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.seq_blk_off[mid] <= e) lo = mid;
    else hi = mid;
  }
  const int64_t first = (e - a.seq_blk_off[lo]) * a.r;
  const int64_t held = min((int64_t)a.seq_len[lo] - first, (int64_t)a.r);
  if (held <= 0) return;
  const int slot = a.seq_blk_slots[e];
  if (slot < 0 || slot >= a.n_slots) {
    atomicOr(err, kErrSlot);
    return;
  }
  atomicOr(&a.slot_bits[slot >> 5], 1u << (slot & 31));
  for (int i = 0; i < (int)held; ++i) {
    const int c = a.blk_cells[(int64_t)slot * a.r + i];
    if (c >= a.n_cells) atomicOr(err, kErrCell);
    else if (c >= 0) atomicOr(&a.cell_bits[c >> 5], 1u << (c & 31));
  }
}

__device__ __forceinline__ unsigned block_sum(unsigned v, unsigned* s_tmp) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  __syncthreads();
  if (lane == 0) s_tmp[warp] = v;
  __syncthreads();
  unsigned t = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) t += s_tmp[w];
  return t;
}

// Live cells (then slots) of each tile.
__global__ void __launch_bounds__(kThreads) k_sweep_count(const SweepArgs a) {
  __shared__ unsigned s_tmp[kWarps];
  grid_dep_wait();
  grid_dep_launch();
  const bool cells = blockIdx.x < (unsigned)a.cell_tiles;
  const int64_t tile = cells ? blockIdx.x : blockIdx.x - a.cell_tiles;
  const unsigned* bits = (cells ? a.cell_bits : a.slot_bits) + tile * kTileWords;
  const unsigned sum = block_sum(__popc(bits[threadIdx.x]), s_tmp);
  if (threadIdx.x == 0) (cells ? a.cell_sums : a.slot_sums)[tile] = sum;
}

// Ranks, free lists and moves of one tile's cells or slots.  In a compaction
// a live cell at or past n_live is written to cell_map as -2 - (its move's
// number); k_sweep_table resolves it.
__global__ void __launch_bounds__(kThreads) k_sweep_apply(const SweepArgs a) {
  __shared__ unsigned s_tmp[kWarps];
  __shared__ unsigned s_bits[kTileWords], s_rank[kTileWords];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool cells = blockIdx.x < (unsigned)a.cell_tiles;
  const int64_t tile = cells ? blockIdx.x : blockIdx.x - a.cell_tiles;
  const unsigned* sums = cells ? a.cell_sums : a.slot_sums;
  const int64_t n_tiles = cells ? a.cell_tiles : a.slot_tiles;
  unsigned before = 0, all = 0;
  for (int64_t k = tid; k < n_tiles; k += kThreads) {
    const unsigned v = sums[k];
    all += v;
    if (k < tile) before += v;
  }
  before = block_sum(before, s_tmp);
  all = block_sum(all, s_tmp);
  const unsigned w = ((cells ? a.cell_bits : a.slot_bits) + tile * kTileWords)[tid];
  unsigned incl = __popc(w);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(kFull, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) s_tmp[warp] = incl;
  s_bits[tid] = w;
  __syncthreads();
  unsigned rank = before + incl - __popc(w);
  for (int k = 0; k < warp; ++k) rank += s_tmp[k];
  s_rank[tid] = rank;
  __syncthreads();
  // live cells below n_live: the movers' ranks start there
  unsigned below = 0;
  const int64_t n_live = all;
  if (cells && a.compact) {
    const int64_t cut = n_live / (32 * kTileWords);
    for (int64_t k = tid; k < cut; k += kThreads) below += sums[k];
    const int64_t cw = n_live >> 5;
    if (cut < n_tiles) {
      const int64_t word = cut * kTileWords + tid;
      const unsigned v = a.cell_bits[word];
      if (word < cw) below += __popc(v);
      if (word == cw) below += __popc(v & ((1u << (n_live & 31)) - 1u));
    }
    below = block_sum(below, s_tmp);
  }
  if (tid == 0 && tile == 0) {
    if (cells) {
      a.counts[0] = (int)all;
      a.counts[1] = (int)(a.n_cells - n_live);
      a.counts[3] = a.compact ? (int)(all - below) : 0;
    } else {
      a.counts[2] = (int)(a.n_slots - (int64_t)all);
    }
  }
  const int64_t n = cells ? a.n_cells : a.n_slots;
  for (int i = tid; i < 32 * kTileWords; i += kThreads) {
    const int64_t c = tile * (32 * kTileWords) + i;
    if (c >= n) break;
    const unsigned word = s_bits[i >> 5];
    const bool live = (word >> (i & 31)) & 1u;
    const int64_t rk = (int64_t)s_rank[i >> 5] + __popc(word & ((1u << (i & 31)) - 1u));
    if (!cells) {
      if (!live && a.free_slots) a.free_slots[c - rk] = (int)c;
      continue;
    }
    int map = live ? (int)c : -1;
    if (a.compact) {
      if (live && c >= n_live) {
        const int64_t k = rk - below;
        a.move_src[k] = (int)c;
        map = (int)(-2 - k);
      }
      if (!live && c < n_live) a.move_dst[c - rk] = (int)c;
      if (c >= n_live && a.free_cells) a.free_cells[c - n_live] = (int)c;
    } else if (!live && a.free_cells) {
      a.free_cells[c - rk] = (int)c;
    }
    if (a.cell_map) a.cell_map[c] = map;
  }
}

// The block table without what nobody holds, under the cells' new places; and
// the movers' entries of cell_map.
__global__ void __launch_bounds__(kThreads) k_sweep_table(const SweepArgs a) {
  grid_dep_wait();
  const int64_t i = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (i < a.n_slots * a.r) {
    const int64_t slot = i / a.r;
    const int c = a.blk_cells[i];
    int v = -1;
    if (c >= 0 && c < a.n_cells && ((a.slot_bits[slot >> 5] >> (slot & 31)) & 1u)) {
      if (a.compact) {
        // the entry of a mover may already be resolved by its own thread
        v = *reinterpret_cast<volatile const int32_t*>(a.cell_map + c);
        if (v < -1) v = a.move_dst[-2 - v];
      } else {
        v = ((a.cell_bits[c >> 5] >> (c & 31)) & 1u) ? c : -1;
      }
    }
    a.blk_cells_out[i] = v;
  }
  if (a.compact && i < a.counts[3]) {
    *reinterpret_cast<volatile int32_t*>(a.cell_map + a.move_src[i]) = a.move_dst[i];
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
  const int64_t x = ceil_div(a.max_blocks > 0 ? a.max_blocks : 1, kThreads);
  prof_before(kKFork, stream);
  cudaError_t e = launch_pdl(k_seq_fork, dim3((unsigned)x, (unsigned)a.n), dim3(kThreads), 0, stream, 1, a, err);
  prof_after(kKFork, stream);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// Workspace: the two bitmaps in whole tiles, then the tiles' sums.
static int64_t sweep_tiles(int64_t n) { return ceil_div(n > 0 ? n : 1, 32 * kTileWords); }
size_t sweep_workspace_bytes(int64_t n_cells, int64_t n_slots) {
  const int64_t tc = sweep_tiles(n_cells), ts = sweep_tiles(n_slots);
  return (size_t)round_up((tc + ts) * kTileWords * 4 + (tc + ts) * 4, 256);
}

cudaError_t launch_cache_sweep(const SweepArgs& args, void* ws, unsigned* err, cudaStream_t stream) {
  SweepArgs a = args;
  a.cell_tiles = sweep_tiles(a.n_cells);
  a.slot_tiles = sweep_tiles(a.n_slots);
  const int64_t tiles = a.cell_tiles + a.slot_tiles;
  a.cell_bits = static_cast<unsigned*>(ws);
  a.slot_bits = a.cell_bits + a.cell_tiles * kTileWords;
  a.cell_sums = a.slot_bits + a.slot_tiles * kTileWords;
  a.slot_sums = a.cell_sums + a.cell_tiles;
  const int64_t n16 = tiles * kTileWords / 4;
  const int64_t entries = a.n_list > a.n_seq ? a.n_list : a.n_seq;
  int64_t table = a.n_slots * a.r;
  if (a.compact && a.n_cells / 2 > table) table = a.n_cells / 2;
  const dim3 block(kThreads);
  auto grid = [](int64_t n) { return dim3((unsigned)ceil_div(n > 0 ? n : 1, kThreads)); };
  prof_before(kKSweep, stream);
  cudaError_t e = launch_pdl(k_sweep_clear, grid(n16), block, 0, stream, 1, reinterpret_cast<uint4*>(ws), n16);
  if (e == cudaSuccess) e = launch_pdl(k_sweep_mark, grid(entries), block, 0, stream, 1, a, err);
  if (e == cudaSuccess) e = launch_pdl(k_sweep_count, dim3((unsigned)tiles), block, 0, stream, 1, a);
  if (e == cudaSuccess) e = launch_pdl(k_sweep_apply, dim3((unsigned)tiles), block, 0, stream, 1, a);
  if (e == cudaSuccess) e = launch_pdl(k_sweep_table, grid(table), block, 0, stream, 1, a);
  prof_after(kKSweep, stream);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

}  // namespace qsa
