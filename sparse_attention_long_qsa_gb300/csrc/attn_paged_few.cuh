// Attention over a paged cache for two and more tokens of a sequence, of any cache
// type, on the 5th-generation tensor cores.  (Prompts over fp16 rows go to
// attn_paged_tc.cu, single tokens to attn_paged_one.cu.)
//
// A group is 16 tokens: 16 tokens x 8 heads are the 128 rows of a CTA's products.
// Fewer tokens leave rows empty.  Per tile of 64 cells (a CTA walks runs of tiles):
//   S = Q K^T     M 128, N 64, K 256; Q in tensor memory, so that only K is read
//                 from shared memory (an operand A there costs 36 cycles more a
//                 product of any N)
//   P             exp2 of S relative to a reference of each row, in two fp16 parts
//                 (22 bits), over S in tensor memory (attn_paged_tmem.cuh)
//   O += P V      M 128, N 256, K 64, in place
// 256 columns of tensor memory hold O, 128 Q, and 2 x 64 S and P of two tiles: all
// 512.  The tensor cores form tile i + 1's scores while the softmax warps work on
// tile i, and add P V of tile i while they work on tile i + 1.
//
// A code times its block's scale has 19 bits at most and is a multiple of 2^-24, so
// two fp16 parts hold it exactly, for every scale that is finite and leaves the
// block within fp16's range.  Scores are then two products (Q K_lo, Q K_hi), sums
// three (P_lo V_hi, P_hi V_lo, P_hi V_hi: what is left out is 2^-22 of a term); the
// small ones come first, so that their roundings are small.
//
// Warps 0-7: softmax, two threads a row, 32 columns each.  Warps 16-19 (fp16: 16-23):
// rows by cp.async, three to seven loads (a tile's K or V rows) ahead.  Warps 8-15: rows to
// operands in stages of 64 KB (32 KB of fp16); a quarter-warp writes 8 cells' chunks,
// which the swizzle spreads over all banks.  The last warp issues the products.  Waits are
// bounded (kErrTimeout).
//
// A V value that is not finite (a block whose scale is not, or leaves fp16's range)
// must reach the rows that see its cell and no others, which a probability of zero
// would not keep out: it is replaced by zero, and what it does to the rows that see
// it is added when the run's result is written.
//
// What bounds it: a tile of codes takes some 4,200 cycles, its products 2,560 (1,024
// and 1,536), its operands 2 x 1,250; they alternate in two stages, which is all that
// shared memory holds of 64 KB each, so neither is ever alone (tensor pipe 52 %).  Five
// tokens over 250k q8_0 cells: 128 us with their join, 0.31 of the row bandwidth (the
// kernel before, on mma.sync, took 310); with block weights 160 us.  512 tokens in a
// window of 1,024 over q8_0: 47 us (157); over all of 50k: 0.70 ms.  With half of the
// products left out the five tokens take 10 % less: it is the chain, not a unit, that
// is full.
#pragma once

#include <atomic>
#include <mutex>

#include "attn_paged_tmem.cuh"

namespace qsa {
namespace {

constexpr int kNT = 16;                      // tokens of a group
constexpr int kCells = 64;                   // cells of a tile
constexpr int kUncut = 4;                    // tiles (see plan): 2 us each
constexpr int kSoft = 256, kConv = 256;
constexpr int kSuper = 512;                  // cells whose ids are looked up together
constexpr int kTiles = kSuper / kCells;
constexpr uint32_t kColQ = 256, kColS = 384;
constexpr uint32_t kPartBytes = 64 * 512;    // 64 cells, 256 dims

// Code bytes of a row, fp16 parts of a value, tiles of operands and loads under way, threads that copy rows (a warp's copy
// of 512 bytes takes it some 80 cycles), and the bits of a scale from which on it counts as infinite.
template <int KV> struct Row;
template <> struct Row<QSA_KV_F16> {
  static constexpr int kCodes = 512, kParts = 1, kStages = 3, kAhead = 3, kGather = 256;
  static constexpr uint32_t kLimit = 0x7c00u;
};
template <> struct Row<QSA_KV_Q8_0> {
  static constexpr int kCodes = 256, kParts = 2, kStages = 2, kAhead = 4, kGather = 128;
  static constexpr uint32_t kLimit = 0x6000u;   // 512
};
template <> struct Row<QSA_KV_Q4_0> {
  static constexpr int kCodes = 128, kParts = 2, kStages = 2, kAhead = 7, kGather = 128;
  static constexpr uint32_t kLimit = 0x7000u;   // 8192
};

template <int KV>
constexpr int kThreads = kSoft + kConv + Row<KV>::kGather + 32;

template <int KV, bool kMixed>
struct Smem {
  static constexpr int kStages = Row<KV>::kStages, kAhead = Row<KV>::kAhead;
  static constexpr int kPieces = Row<KV>::kCodes / 64, kPitch = Row<KV>::kCodes + 16;
  alignas(1024) unsigned char stage[kStages][Row<KV>::kParts * kPartBytes];
  alignas(16) unsigned char raw[kAhead][kCells * kPitch];   // rows as they come, codes then scales
  float max[2][2][128];                      // of half a row, by tile parity
  bool alone[2][2][128];                     // (see tile_top)
  float sum[2][128];
  alignas(16) float out[kSoft / 32][32][kOutPitch];   // see write_rows
  int ids[2][kSuper];
  uint32_t ok[8][kSuper / 32];               // which of them exist
  uint64_t landed[kAhead], taken[kAhead], full[kStages], empty[kStages], s_full[2], p_full[2], pv_done[2], q_full;
  uint32_t tmem;
  PlanOf<kMixed> plan;
  unsigned stray[8];                         // of a run: V values that are not finite were met
};
template <int KV, bool kMixed>
constexpr size_t kSmemBytes = sizeof(Smem<KV, kMixed>) + 1024;
static_assert(kSmemBytes<QSA_KV_F16, true> <= 227 * 1024 && kSmemBytes<QSA_KV_Q8_0, true> <= 227 * 1024 &&
                  kSmemBytes<QSA_KV_Q4_0, true> <= 227 * 1024, "shared memory of an SM");
static_assert(sizeof(Smem<QSA_KV_F16, false>::stage) >= kPlanScratch, "the plan's scratch");

// kind::f16, fp32 accumulators, M = 128; B K-major (scores) or MN-major (P V)
constexpr uint32_t kIdescS = (1u << 4) | (((uint32_t)kCells >> 3) << 17) | ((128u >> 4) << 24);
constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((256u >> 3) << 17) | ((128u >> 4) << 24);

// D += A B, A in tensor memory.  By a whole warp, of which one lane issues: a branch to a lane chosen by number would cost
// some 120 cycles a product (256 products of N = 64: 122 cycles each, 33 like this).
__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrives when the warp's products so far are done (the same lane).
__device__ __forceinline__ void commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(bar)
      : "memory");
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// The halves of x whose magnitude is limit (bits of a half) or more, or NaN: all their bits set.
__device__ __forceinline__ uint32_t halves_from(uint32_t x, uint32_t limit) {
  return ((x & 0x7fffu) >= limit ? 0xffffu : 0u) | (((x >> 16) & 0x7fffu) >= limit ? 0xffff0000u : 0u);
}
__device__ __forceinline__ uint4 ld_smem(uint32_t p) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(p) : "memory");
  return x;
}
// The sums of blocks of R of 32 values, at a multiple of 16 bytes.
template <int R>
__device__ __forceinline__ void block_sums(float* e, const float (&s)[32]) {
#pragma unroll
  for (int j = 0; j < 32 / R; j += 4) {
    float x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = s[(j + k) * R];
#pragma unroll
      for (int c = 1; c < R; ++c) x[k] += s[(j + k) * R + c];
    }
    *reinterpret_cast<float4*>(e + j) = make_float4(x[0], x[1], x[2], x[3]);
  }
}
// (bounds of 768 or 896 threads: 80 or 72 registers, so that the six or seven warps of one sub-partition fit)
template <int KV, bool kWeigh, bool kMixed>
__global__ void __launch_bounds__(KV == QSA_KV_F16 ? 896 : 768, 1) k_paged_few(const PagedArgs a, unsigned* err) {
  using S = Smem<KV, kMixed>;
  constexpr int kStages = S::kStages, kAhead = S::kAhead, kPieces = S::kPieces, kPitch = S::kPitch, kCodes = Row<KV>::kCodes, kParts = Row<KV>::kParts;
  constexpr uint32_t kStageBytes = kParts * kPartBytes;
  constexpr bool kF16 = KV == QSA_KV_F16;
  constexpr int kGather = Row<KV>::kGather;
  constexpr int kAdditions = 4 * (kParts + 1);   // to O, of a tile
  extern __shared__ unsigned char raw[];
  S& sm = *reinterpret_cast<S*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
  const int G = a.n_kv_heads, g = blockIdx.x % G, part = blockIdx.x / G;
  const bool reports = g == 0;
  // scores in the log2 domain; a negative scale turns the queries' signs instead, and one of zero stays above it (-inf times
  // zero would be NaN)
  const float scale2 = fmaxf(fabsf(a.attn_scale) * 1.4426950408889634f, 1e-37f);
  const uint32_t flip = a.attn_scale < 0.f ? 0x80008000u : 0u;
  const uint32_t stage0 = smem_u32(sm.stage[0]);
  const uint32_t bland = smem_u32(sm.landed), btaken = smem_u32(sm.taken), bfull = smem_u32(sm.full), bempty = smem_u32(sm.empty), bs = smem_u32(sm.s_full), bp = smem_u32(sm.p_full),
                 bpv = smem_u32(sm.pv_done), bq = smem_u32(&sm.q_full);

  if constexpr (kMixed) {   // nothing to do: before anything is set up
    if (a.second) {
      grid_dep_wait();
      if (!*a.left) {
        if (tid == 0 && reports && !a.span_by_token) a.span[part] = make_int4(0, 0, 0, 0);
        return;
      }
    }
  }
  if (warp == 0) tmem_alloc(smem_u32(&sm.tmem), 512);
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bfull + 8 * i, kConv / 32);
      mbar_init(bempty + 8 * i, 1);
    }
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(bland + 8 * i, kGather);
      mbar_init(btaken + 8 * i, kConv / 32);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bs + 8 * i, 1);
      mbar_init(bp + 8 * i, kSoft / 32);
      mbar_init(bpv + 8 * i, 1);
    }
    mbar_init(bq, kSoft / 32);
    for (int i = 0; i < 8; ++i) sm.stray[i] = 0u;
  }
  grid_dep_wait();
  grid_dep_launch();
  plan<kNT, kCells, kMixed>(a, reinterpret_cast<int*>(sm.stage[0]), &sm.plan, tid, part, gridDim.x / G, 1, kUncut,
                    a.n_tokens > (int)gridDim.x / G ? 6 + a.n_tokens / 64 : kUncut);
  const PlanOf<kMixed>& pl = sm.plan;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  bool timed_out = false;
  // The CTA's runs, each role in a loop of its own that goes on to the next run by itself.  base, chunks: tiles of the runs
  // before, and groups of kSuper ids, from which stages, barriers and buffers go on.
  auto for_runs = [&](auto body) {
    int base = 0, runs = 0, chunks = 0, t0 = pl.t0, first = pl.first;
    for (int u = pl.u0; u < pl.u1; ++runs) {
      const Run run = run_at<kNT, kCells>(a, t0, first, pl.u1 - u);
      body(run, base, runs, chunks, u);
      u += run.n;
      base += run.n;
      chunks += (run.n + kTiles - 1) / kTiles;
      t0 = next_group<kMixed>(a, pl, run.g.t0 + run.g.nt);
      first = 0;
    }
  };
  // loads in the order of the products: K of tile 0, then K of tile j + 1 and V of tile j, V of the last
  auto load_of_k = [](int i) { return i == 0 ? 0 : 2 * i - 1; };
  auto load_of_v = [](int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; };

  if (warp < 8) {
    // 2 x 104 + 2 x 64 + 64 of a sub-partition's 5 x 80; fp16: 2 x 104 + 2 x 56 + 2 x 56 of 6 x 72
    asm volatile("setmaxnreg.inc.sync.aligned.u32 104;\n");
    // ---- softmax: row 32 (warp % 4) + lane, columns 32 half .. + 31
    const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane, tok = row >> 3, head = row & 7;
    const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
    auto load_q = [&](const Group& gr) {   // 128 dims of the row
      const bool mine = tok < gr.nt;
      const __half* src = a.q + (((int64_t)(gr.t0 + tok) * G + g) * kGqa + head) * kHeadDim + 128 * half;
      if (4 * quarter < gr.nt) {
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          uint4 y[8];
          const uint4* q = reinterpret_cast<const uint4*>(src + 64 * k);
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = mine ? q[j] : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t x[16];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint4 z = y[4 * c + j];
              x[4 * j] = z.x ^ flip, x[4 * j + 1] = z.y ^ flip, x[4 * j + 2] = z.z ^ flip, x[4 * j + 3] = z.w ^ flip;
            }
            tmem_st16(tl + kColQ + 64 * half + 32 * k + 16 * c, x);
          }
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) arrive(bq);
    };
    for_runs([&](const Run& run, int base, int runs, int chunks, int u) {
      const Group& gr = run.g;
      const int n = run.n, v_first = run.first * kCells;
      const bool idle = 4 * quarter >= gr.nt, mine = tok < gr.nt;   // rows of no token
      const int64_t out_row = ((int64_t)(gr.t0 + tok) * G + g) * kGqa + head;
      if (runs == 0) load_q(gr);
      if (tid == 0) sm.stray[(runs + 4) & 7] = 0u;   // every warp has left run `runs` - 4; rows come three runs ahead at most
      const int pos = mine ? token_pos(a, gr.t0 + tok) : -1;
      // the reading-order range that the token sees, and its sinks
      const int vhi = pos - gr.lo_al + gr.ns_al + 1;
      const int vlo = a.window > 0 ? max(pos - a.window + 1 - gr.lo_al + gr.ns_al, gr.ns_al) : 0;
      const int vsink = gr.lo_al == 0 || gr.ns_al > 0 ? min(min(a.n_sink, pos + 1), gr.nv) : 0;
      const bool whole = n == gr.tiles;
      const int64_t ps = ((int64_t)(2 * part + (run.first == 0 ? 1 : 0)) * G + g) * (a.of.tokens * kGqa);   // the run's rows
      float* sums = a.of.o + ps * kHeadDim + 128 * half;
      const int stretch = stretch_of(n, kAdditions);
      int next = stretch;   // where the next one begins
      float fs = 0.f;       // of the stretches' sums so far
      float m = mine ? kNoMax : 0.f, high = kNoMax, l = 0.f;   // the row's reference, the highest, this half's sum relative to it
      bool big = false;   // (see is_big)
      for (int i = 0; i < n; ++i) {
        const int b = (base + i) & 1;
        const uint32_t ts = tl + kColS + kCells * b + 32 * half;
        const int v0 = v_first + i * kCells + 32 * half;
        if (!mbar_wait(bs + 8 * b, (uint32_t)((base + i) >> 1) & 1u)) timed_out = true;
        if (!idle) {
          tc_fence_after();
          const bool begins = i == next;
          float raised = 1.f;
          float s[32];
          tmem_ld16_nowait(ts, reinterpret_cast<uint32_t*>(s));
          tmem_ld16_nowait(ts + 16, reinterpret_cast<uint32_t*>(s + 16));
          uint32_t see = sm.ok[(chunks + i / kTiles) & 7][(i % kTiles) * 2 + half] & below(vhi - v0) &
                         (~below(vlo - v0) | below(vsink - v0));
          if (!mine) see = 0xffffffffu;   // (no mask for the others' sake)
          const bool all_seen = __all_sync(kFull, see == 0xffffffffu);
          tmem_wait_ld();
          if (!all_seen) {
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] = (see >> j) & 1u ? s[j] : -INFINITY;
          }
          float t4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
          for (int j = 4; j < 32; ++j) t4[j & 3] = fmaxf(t4[j & 3], s[j]);
          bool alone;
          const float top = tile_top(t4, scale2, alone);
          sm.max[b][half][row] = top;
          sm.alone[b][half][row] = alone;
          bar_named(2 + quarter, 64);   // the row's two threads
          const float nm = mine ? next_reference(m, high, top, sm.max[b][half ^ 1][row], alone || sm.alone[b][half ^ 1][row], big, scale2) : m;
          if (__any_sync(kFull, nm != m)) {
            const float f = ex2(m - nm);
            l *= f;
            m = nm;
            big = is_big(m);
            raised = f;
            if (i > 0 && !begins) {   // O holds the tiles before
              if (!mbar_wait(bpv + 8 * (b ^ 1), (uint32_t)((base + i - 1) >> 1) & 1u)) timed_out = true;
              tc_fence_after();
#pragma unroll 1
              for (int k = 0; k < 8; ++k) {
                uint32_t o[16];
                tmem_ld16_nowait(tl + 128 * half + 16 * k, o);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_st16(tl + 128 * half + 16 * k, o);
              }
            }
          }
          // probabilities, in place: of 16 cells first parts in 8 columns, second parts in the next 8
          float ref = kUp - m, by = scale2;
          if (big) {
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] = __fsub_rn(__fmul_rn(s[j], scale2), m);
            ref = kUp, by = 1.f;
          }
          float sx = 0.f, sy = 0.f;
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t w[16];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int c = 16 * k + 2 * j;
              float x = s[c], y = s[c + 1];
              fma2(x, y, by, ref);
              x = ex2(x), y = ex2(y);
              add2(sx, sy, x, y);
              if constexpr (kWeigh) s[c] = x, s[c + 1] = y;
              float2 h;
              w[j] = first_part(x, y, h);
              add2(x, y, -h.x, -h.y);
              w[8 + j] = bits(__floats2half2_rn(x, y));
            }
            tmem_st16(ts + 16 * k, w);
          }
          l += sx + sy;
          tmem_wait_st();
          if (begins) {   // the sums of the stretch before, of the reference before
            if (!mbar_wait(bpv + 8 * (b ^ 1), (uint32_t)((base + i - 1) >> 1) & 1u)) timed_out = true;
            tc_fence_after();
            write_rows<false>(tl + 128 * half, sm.out[warp], 1.f, sums, kGqa * kHeadDim, i > stretch ? sums : nullptr, fs, 32 * quarter, gr.nt);
            fs = 1.f;
            next += stretch;
          }
          fs *= raised;
          tc_fence_before();
          __syncwarp();
          if (lane == 0) arrive(bp + 8 * b);
          if constexpr (kWeigh) {   // the sums of whole blocks, relative to the row's reference
            if (!all_seen) {   // (of a row that is NaN, only what it sees)
#pragma unroll
              for (int j = 0; j < 32; ++j) s[j] = (see >> j) & 1u ? s[j] : 0.f;
            }
            if (mine) {
              if (half == 0) a.em[out_row * a.e_tiles + run.first + i] = m;
              float* e = a.e + out_row * a.e_blocks + (v0 >> a.r_shift);
              if (a.r_shift == 0) block_sums<1>(e, s);
              else if (a.r_shift == 1) block_sums<2>(e, s);
              else if (a.r_shift == 2) block_sums<4>(e, s);
              else block_sums<8>(e, s);
            }
          }
        } else if (lane == 0) {
          arrive(bp + 8 * b);
        }
      }
      // ---- the run's result: a row of 256 values, 128 a thread
      if (!mbar_wait(bpv + 8 * ((base + n - 1) & 1), (uint32_t)((base + n - 1) >> 1) & 1u)) timed_out = true;
      tc_fence_after();
      if (u + n < pl.u1) load_q(run_at<kNT, kCells>(a, next_group<kMixed>(a, pl, gr.t0 + gr.nt), 0, 1).g);   // scores of the next run form meanwhile
      if (idle) return;
      sm.sum[half][row] = l;
      bar_named(2 + quarter, 64);
      l = sm.sum[0][row] + sm.sum[1][row];
      if (mine && half == 0) {
        if (!whole) *reinterpret_cast<float2*>(a.of.ml + 2 * (ps + row)) = make_float2(m, l);
        else if (kWeigh) a.lse[out_row] = make_float2(m, l != 0.f ? 1.f / l : 0.f);
        if (kWeigh && g == 0 && head == 0 && run.first == 0) a.geo[gr.t0 + tok] = make_int4(gr.ns_al, gr.lo_al, gr.nv, kCells);
      }
      const float w = whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
      float* rows = whole ? a.out + ((int64_t)gr.t0 * G + g) * kGqa * kHeadDim + 128 * half : sums;
      const bool stray = *reinterpret_cast<volatile unsigned*>(&sm.stray[runs & 7]) != 0u;   // (one value for the warp)
      const int64_t stride = (whole ? G : 1) * (kGqa * kHeadDim);
      write_rows<false>(tl + 128 * half, sm.out[warp], w, rows, stride, stretch < n ? sums : nullptr, fs, 32 * quarter, gr.nt);
      if (stray) {   // (a row whose sum is not finite is NaN throughout)
        put_not_finite(
            a, run, v_first, min(gr.nv, v_first + n * kCells),
            mine && l - l == 0.f ? rows + tok * stride + head * kHeadDim : nullptr,
            [&](int p) { return p <= pos && (a.window == 0 || p > pos - a.window || p < a.n_sink); },
            [&](int c, int k, uint32_t (&x)[8]) {
              if constexpr (kF16) {
                const uint4* from = reinterpret_cast<const uint4*>(static_cast<const __half*>(a.v_cache) +
                                                                   ((int64_t)c * G + g) * kHeadDim + 128 * half + 16 * k);
                const uint4 lo = from[0], hi = from[1];
                x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
              } else {
                const unsigned short* d = reinterpret_cast<const unsigned short*>(static_cast<const unsigned char*>(a.v_cache) +
                                                                                  a.n_cells * (int64_t)(G * kCodes));
                if ((d[((int64_t)c * G + g) * 8 + 4 * half + (k >> 1)] & 0x7fffu) >= Row<KV>::kLimit) {
#pragma unroll
                  for (int j = 0; j < 8; ++j) x[j] = 0x7fff7fffu;
                }
              }
            });
      }
      tc_fence_before();
    });
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kF16 ? 56 : 64));
    for_runs([&](const Run& run, int base, int runs, int, int) {
      const int n = run.n;
      // ---- operands: this thread's cell of a tile is 8 w8 + lane % 8, of each 64 bytes of its row 16
      const int w8 = warp - 8, own = 8 * w8 + (lane & 7);
#pragma unroll 1
      for (int L = 0; L < 2 * n; ++L) {
        const int use = 2 * base + L, st = use % kStages, rs = use % kAhead;
        if (!mbar_wait(bland + 8 * rs, (uint32_t)(use / kAhead) & 1u)) timed_out = true;
        const uint32_t from = smem_u32(sm.raw[0]) + rs * (kCells * kPitch) + own * kPitch;
        uint4 x[kPieces], scales;
#pragma unroll
        for (int p = 0; p < kPieces; ++p) x[p] = ld_smem(from + 64 * p + (lane >> 3) * 16);
        if constexpr (!kF16) scales = ld_smem(from + kCodes);
        if (use >= kStages && !mbar_wait(bempty + 8 * st, (uint32_t)(use / kStages - 1) & 1u)) timed_out = true;
        const bool k = L == 0 || ((L & 1) && L != 2 * n - 1);
        const uint32_t dst = stage0 + st * kStageBytes + own * 128;
        // chunk c16 (of 8 dims) of atom column `col` (64 dims)
        auto put = [&](uint32_t col, uint32_t c16, uint32_t part, const uint32_t (&w)[4]) {
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(dst + part * kPartBytes + col * 8192 + ((c16 ^ (lane & 7)) << 4)),
                       "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]) : "memory");
        };
        if constexpr (kF16) {
          if (!k) {
            __half2 z = half2_of(0u);   // NaN if some value is not finite
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {
              z = __hfma2(half2_of(x[p].x), half2_of(0u), z), z = __hfma2(half2_of(x[p].y), half2_of(0u), z);
              z = __hfma2(half2_of(x[p].z), half2_of(0u), z), z = __hfma2(half2_of(x[p].w), half2_of(0u), z);
            }
            if (halves_from(bits(z), Row<KV>::kLimit)) {
#pragma unroll
              for (int p = 0; p < kPieces; ++p) {
                x[p].x &= ~halves_from(x[p].x, Row<KV>::kLimit), x[p].y &= ~halves_from(x[p].y, Row<KV>::kLimit);
                x[p].z &= ~halves_from(x[p].z, Row<KV>::kLimit), x[p].w &= ~halves_from(x[p].w, Row<KV>::kLimit);
              }
              sm.stray[runs & 7] = 1u;
            }
          }
#pragma unroll
          for (int p = 0; p < kPieces; ++p) {
            const uint32_t w[4] = {x[p].x, x[p].y, x[p].z, x[p].w};
            put(p >> 1, 4 * (p & 1) + (lane >> 3), 0, w);
          }
        } else {
          uint32_t d[4] = {scales.x, scales.y, scales.z, scales.w};
          uint32_t top = 0u;
#pragma unroll
          for (int j = 0; j < 4; ++j) top = __vmaxu2(top, d[j] & 0x7fff7fffu);
          if (max(top & 0xffffu, top >> 16) >= Row<KV>::kLimit) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t out = halves_from(d[j], Row<KV>::kLimit);
              d[j] = k ? d[j] | out : d[j] & ~out;   // NaN, or zero
            }
            if (!k) sm.stray[runs & 7] = 1u;
          }
          // two words of codes to a chunk's two parts
          auto split = [&](uint32_t col, uint32_t c16, uint32_t x0, uint32_t x1, uint32_t off, uint32_t scale) {
            const __half2 s = half2_of(scale);
            const __half2 c[4] = {bytes2<0x4140>(x0, off), bytes2<0x4342>(x0, off), bytes2<0x4140>(x1, off), bytes2<0x4342>(x1, off)};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const __half2 h = __hmul2(c[j], s);
              hi[j] = bits(h);
              lo[j] = bits(__hfma2(c[j], s, __hneg2(h)));
            }
            put(col, c16, 0, hi);
            put(col, c16, 1, lo);
          };
          if constexpr (KV == QSA_KV_Q8_0) {
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {   // 64 dims, 16 of them here: of block 2 p or 2 p + 1
              const uint32_t s = __byte_perm(d[p], 0u, lane & 16 ? 0x3232 : 0x1010), c16 = 2 * (lane >> 3);
              split(p, c16, x[p].x ^ 0x80808080u, x[p].y ^ 0x80808080u, 0x64806480u, s);
              split(p, c16 + 1, x[p].z ^ 0x80808080u, x[p].w ^ 0x80808080u, 0x64806480u, s);
            }
          } else {
#pragma unroll
            for (int p = 0; p < kPieces; ++p) {   // block 4 p + lane / 8: its first 16 dims, then the others
              const uint32_t s = __byte_perm(lane & 16 ? d[2 * p + 1] : d[2 * p], 0u, lane & 8 ? 0x3232 : 0x1010);
              const uint32_t col = 2 * p + (lane >> 4), c16 = (lane >> 1) & 4;
              constexpr uint32_t kLow = 0x0f0f0f0fu, kOff = 0x64086408u;
              split(col, c16, x[p].x & kLow, x[p].y & kLow, kOff, s);
              split(col, c16 + 1, x[p].z & kLow, x[p].w & kLow, kOff, s);
              split(col, c16 + 2, (x[p].x >> 4) & kLow, (x[p].y >> 4) & kLow, kOff, s);
              split(col, c16 + 3, (x[p].z >> 4) & kLow, (x[p].w >> 4) & kLow, kOff, s);
            }
          }
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          arrive(bfull + 8 * st);
          arrive(btaken + 8 * rs);
        }
      }
    });
  } else if (warp < 16 + kGather / 32) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(kF16 ? 56 : 64));
    for_runs([&](const Run& run, int base, int, int chunks, int) {
      const int n = run.n, v_first = run.first * kCells, v_end = min(run.g.nv, (run.first + n) * kCells);
      // ---- rows
      const int tx = tid - kSoft - kConv, w4 = warp - 16;
      constexpr int kLanes = kCodes / 16, kRows = 32 / kLanes;   // lanes a row, rows of a warp's copy
      const int64_t codes = a.n_cells * (int64_t)(G * kCodes);
      const uint32_t pitch = (uint32_t)(G * kCodes);
      const unsigned char* kc = static_cast<const unsigned char*>(a.k_cache) + g * kCodes + (lane % kLanes) * 16;
      const unsigned char* vc = static_cast<const unsigned char*>(a.v_cache) + g * kCodes + (lane % kLanes) * 16;
      const unsigned char* ks = static_cast<const unsigned char*>(a.k_cache) + codes + g * 16;
      const unsigned char* vs = static_cast<const unsigned char*>(a.v_cache) + codes + g * 16;
      constexpr int kPer = kSuper / kGather;
      int slot[kPer], cell[kPer];
      auto find_slots = [&](int sc) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) slot[i] = slot_at(a, run, v_first + sc * kSuper + i * kGather + tx, v_end, reports, err);
      };
      auto find_cells = [&](int sc) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) cell[i] = cell_at(a, run, v_first + sc * kSuper + i * kGather + tx, slot[i], reports, err);
      };
      auto keep_cells = [&](int sc) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const int c = checked_cell(a, cell[i], reports, err);
          sm.ids[(chunks + sc) & 1][i * kGather + tx] = c;
          const uint32_t ok = __ballot_sync(kFull, c >= 0);
          if (lane == 0) sm.ok[(chunks + sc) & 7][i * (kGather / 32) + w4] = ok;
        }
      };
      find_slots(0);
      find_cells(0);
      find_slots(1);
      bar_named(1, kGather);   // the ids of the run before have been read
      keep_cells(0);
      bar_named(1, kGather);
      int next_k = 0, next_v = 0;   // tiles
#pragma unroll 1
      for (int L = 0; L < 2 * n; ++L) {
        const int use = 2 * base + L, rs = use % kAhead;
        const bool k = L == 0 || ((L & 1) && L != 2 * n - 1);
        const int i = k ? next_k : next_v;
        next_k += k, next_v += !k;
        if (k && i % kTiles == 0) {   // the next 512 ids
          if (i > 0) {
            bar_named(1, kGather);   // the ids two groups before have been read
            keep_cells(i / kTiles);
            bar_named(1, kGather);
          }
        } else if (k && i % kTiles == 1) {
          find_cells(i / kTiles + 1);
          find_slots(i / kTiles + 2);
        }
        if (use >= kAhead && !mbar_wait(btaken + 8 * rs, (uint32_t)(use / kAhead - 1) & 1u)) timed_out = true;
        const int* id = &sm.ids[0][0] + ((chunks * kTiles + i) & (2 * kTiles - 1)) * kCells;
        const uint32_t to = smem_u32(sm.raw[0]) + rs * (kCells * kPitch);
        const unsigned char* x = k ? kc : vc;
#pragma unroll
        for (int r = 0; r < kCells; r += kGather / 32 * kRows) {
          const int row = r + w4 * kRows + lane / kLanes, c = id[row];
          cp_async16(to + row * kPitch + (lane % kLanes) * 16, x + (uint64_t)(uint32_t)max(c, 0) * pitch, c >= 0);
        }
        if (!kF16 && lane < kCells / 4) {
          const int row = w4 * (kCells / 4) + lane, c = id[row];
          cp_async16(to + row * kPitch + kCodes, (k ? ks : vs) + (uint64_t)(uint32_t)max(c, 0) * (uint32_t)(G * 16), c >= 0);
        }
        // arrives when this thread's copies so far have landed
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bland + 8 * rs) : "memory");
      }
    });
    asm volatile("cp.async.wait_all;\n" ::: "memory");
  } else {
    // ---- the products, in the order in which the tensor cores take them: scores of tile i + 2 behind P V of tile i,
    // whose columns they take
    if (lane == 0 && reports && !a.span_by_token) a.span[part] = make_int4(0, 0, 0, 0);
    for_runs([&](const Run& run, int base, int runs, int, int u) {
      if (reports) announce(a, pl, run, part, u, err);
      const int n = run.n;
      if (!mbar_wait(bq, (uint32_t)runs & 1u)) timed_out = true;
      auto loaded = [&](int L) {
        const int use = 2 * base + L;
        if (!mbar_wait(bfull + 8 * (use % kStages), (uint32_t)(use / kStages) & 1u)) timed_out = true;
      };
      auto scores = [&](int i) {
        const int b = (base + i) & 1, st = (2 * base + load_of_k(i)) % kStages;
        const uint32_t k = stage0 + st * kStageBytes;
#pragma unroll
        for (int p = kParts - 1; p >= 0; --p)
#pragma unroll
          for (int kk = 0; kk < 16; ++kk)
            mma_ts(tmem + kColS + kCells * b, tmem + kColQ + 8 * kk,
                   smem_desc(k + p * kPartBytes + (kk >> 2) * 8192 + (kk & 3) * 32, 16, 1024), kIdescS, p < kParts - 1 || kk > 0);
        commit(bs + 8 * b);
        commit(bempty + 8 * st);
      };
      loaded(load_of_k(0));
      tc_fence_after();
      scores(0);
      if (n > 1) {
        loaded(load_of_k(1));
        scores(1);
      }
      const int stretch = stretch_of(n, kAdditions);
      int first = 0;   // of the stretch
      loaded(load_of_v(0, n));
      for (int i = 0; i < n; ++i) {
        const int b = (base + i) & 1, st = (2 * base + load_of_v(i, n)) % kStages;
        if (i == first + stretch) first = i;
        if (!mbar_wait(bp + 8 * b, (uint32_t)((base + i) >> 1) & 1u)) timed_out = true;
        tc_fence_after();
        const uint32_t v = stage0 + st * kStageBytes;
        // P's second part with V's first, P's first with V's parts, the smaller first
#pragma unroll
        for (int term = 0; term <= kParts; ++term) {
          const uint32_t p_part = term == 0 ? 8u : 0u, v_part = term == 1 && kParts == 2 ? kPartBytes : 0u;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(tmem, tmem + kColS + kCells * b + 16 * kk + p_part,
                   smem_desc(v + v_part + kk * 2048, 8192, 1024), kIdescO, i > first || term > 0 || kk > 0);
        }
        commit(bpv + 8 * b);
        commit(bempty + 8 * st);
        if (i + 2 < n) {
          loaded(load_of_k(i + 2));
          scores(i + 2);
        }
        if (i + 1 < n) loaded(load_of_v(i + 1, n));
      }
    });
  }
  if (timed_out) atomicOr(err, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

constexpr int kMaxDevices = 64;

template <int KV, bool kWeigh, bool kMixed>
cudaError_t launch(const PagedArgs& a, unsigned* err, cudaStream_t stream) {
  static std::atomic<bool> known[kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!known[dev].load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(mu);
    e = cudaFuncSetAttribute(k_paged_few<KV, kWeigh, kMixed>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<KV, kMixed>);
    if (e != cudaSuccess) return e;
    known[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(k_paged_few<KV, kWeigh, kMixed>, dim3((unsigned)(a.of.parts * a.n_kv_heads)), dim3(kThreads<KV>), kSmemBytes<KV, kMixed>, stream, 1,
                    a, err);
}

template <int KV, bool kMixed>
cudaError_t launch_kv(const PagedArgs& a, unsigned* err, cudaStream_t stream) {
  return a.weigh ? launch<KV, true, kMixed>(a, err, stream) : launch<KV, false, kMixed>(a, err, stream);
}
template <bool kMixed>
cudaError_t launch_few(const PagedArgs& a, int kv_type, unsigned* err, cudaStream_t stream) {
  return kv_type == QSA_KV_F16    ? launch_kv<QSA_KV_F16, kMixed>(a, err, stream)
         : kv_type == QSA_KV_Q8_0 ? launch_kv<QSA_KV_Q8_0, kMixed>(a, err, stream)
                                  : launch_kv<QSA_KV_Q4_0, kMixed>(a, err, stream);
}

}  // namespace
}  // namespace qsa
