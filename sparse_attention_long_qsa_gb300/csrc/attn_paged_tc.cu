// Attention over a paged fp16 cache for many tokens of a sequence (a prompt, a
// chunk of one), on the 5th-generation tensor cores.
//
// A group is 32 tokens.  A pair of CTAs (a cluster) takes it for one KV head: 16
// tokens x 8 heads are the 128 rows of each CTA, 256 rows of a product that both
// SMs' tensor cores form (cta_group::2).  Each CTA holds half of the product's other
// operand, so it gathers half the bytes: an SM reads some 37 bytes a cycle from L2,
// and a CTA alone would need 43.  Per tile of 128 cells (a pair walks a run of
// tiles, see attn_paged.cu):
//   S = Q K^T     M 256, N 128 (each CTA holds 64 cells' rows), K 256
//   P             exp2 of S relative to a reference of each row, in two fp16 parts
//                 (22 bits), over S in tensor memory (attn_paged_tmem.cuh)
//   O += P V      M 256, N 256 (each CTA holds 128 dims), K 128, twice (the two
//                 parts), in place
// 2 x 128 columns of tensor memory hold S and P of two tiles, 256 hold O: all 512.
// So the tensor cores form tile i + 1's scores while the softmax warps work on tile
// i, and add P V of tile i while they work on tile i + 1.
//
// Warps 0-7: softmax, two threads a row, 64 columns each.  Warps 8-15: gather the
// rows by cp.async into four stages of 32 KB, in the order in which the products
// take them (a warp's copy of 512 bytes takes it some 80 cycles to issue, so four
// warps would not keep up; the registers they do not need go to the softmax).
// Warp 16 tells the even CTA of the rows that have landed; there warp 17 issues the
// products.  Waits are bounded (kErrTimeout).
//
// A cell that some tokens of the group do not see may hold infinities or NaN, and a
// probability of zero would not keep them out.  In tiles at the edge of what the
// group sees, V values that are not finite are therefore taken out of shared memory
// before the product.  Where a run's result is not finite, or such values were taken
// out, those that the row sees are added up in its place.
//
// The two parts of P cost a half more than one would (3,072 instead of 2,048 tensor
// cycles a tile): the output is fp32, and one part would leave it 2e-4 off.
//
// What bounds it: the tensor pipe is 75 % busy (512 tokens over 50k cells, 0.455 ms,
// 915 TFLOP/s of the definition's products, 1.37 PFLOP/s of those that are made).  The
// rest is Q's reading from shared memory (36 cycles of each score product; tensor
// memory has no room for it) and 4 us for each stretch of sums that leaves.  8,192
// tokens in a window of 4,096: 0.62 ms, of which a run's beginning and end take a
// sixth and the plan of each 4,096 tokens 10 us.
#include <atomic>
#include <mutex>

#include "attn_paged_tmem.cuh"

namespace qsa {
namespace {

constexpr int kNT = 32;                      // tokens of a pair, half of them a CTA
constexpr int kCells = 128;                  // cells of a tile
constexpr int kUncut = 3;                    // tiles (see plan): 2 us each
constexpr int kSoft = 256, kGather = 256, kThreads = kSoft + kGather + 64;
constexpr int kStages = 4;
constexpr uint32_t kStageBytes = 32768;      // 64 cells' K rows, or 128 dims of 128 cells' V rows
constexpr int kSuper = 512;                  // cells whose ids are looked up together
constexpr uint32_t kColS = 256;
constexpr int kAdditions = 16;               // to O, of a tile

template <bool kMixed>
struct Smem {
  alignas(1024) unsigned char q[128 * 512];
  alignas(1024) unsigned char stage[kStages][kStageBytes];
  float max[2][2][128];                      // of half a row, by tile parity
  bool alone[2][2][128];                     // (see tile_top)
  float sum[2][128];
  alignas(16) float out[kSoft / 32][32][kOutPitch];   // see write_rows
  int ids[2][kSuper];
  uint32_t ok[4][kSuper / 32];               // which of them exist
  uint64_t landed[kStages], full[kStages], s_full[2], p_full[2], pv_done[2], q_full;
  uint32_t tmem;
  PlanOf<kMixed> plan;
  unsigned stray[4];                         // of a run: such V values were met (see above)
};
static_assert(kStages * kStageBytes >= kPlanScratch, "the plan's scratch");
template <bool kMixed>
constexpr size_t kSmemBytes = sizeof(Smem<kMixed>) + 1024;
static_assert(kSmemBytes<true> <= 227 * 1024, "shared memory of an SM");

// kind::f16, fp32 accumulators, M = 256 over the pair; B K-major (scores) or MN-major (P V)
constexpr uint32_t kIdescS = (1u << 4) | (((uint32_t)kCells >> 3) << 17) | ((256u >> 4) << 24);
constexpr uint32_t kIdescO = (1u << 4) | (1u << 16) | ((256u >> 3) << 17) | ((256u >> 4) << 24);

__device__ __forceinline__ void pair_alloc(uint32_t dst_smem) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(dst_smem), "r"(512) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
}
__device__ __forceinline__ void pair_dealloc(uint32_t taddr) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;\n" ::"r"(taddr), "r"(512) : "memory");
}
// D += A B over the pair: A from both CTAs' shared memory, or (ts) their tensor memory, B half in each.  By a whole warp, of
// which one lane issues: a branch to a lane chosen by number would cost some 120 cycles a product.
__device__ __forceinline__ void pair_mma(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void pair_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Arrives at this barrier in both CTAs when the warp's products so far are done (the same lane).
__device__ __forceinline__ void pair_commit(uint32_t bar) {
  asm volatile(
      "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(bar),
               "h"((uint16_t)3)
               : "memory");
}
// Arrives at the even CTA's barrier (an address of its shared memory).
__device__ __forceinline__ void lead_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
// The halves of x that are infinite or NaN, all their bits set.
__device__ __forceinline__ uint32_t stray_halves(uint32_t x) {
  return ((x & 0x7c00u) == 0x7c00u ? 0xffffu : 0u) | ((x & 0x7c000000u) == 0x7c000000u ? 0xffff0000u : 0u);
}
// Whether some token of the group does not see some cell of the tile at v0.
__device__ __forceinline__ bool edge_tile(const Group& g, int window, int v0) {
  return g.nt > 1 && (pos_of(g, v0 + kCells - 1) > g.pmin || (window > 0 && pos_of(g, max(v0, g.ns_al)) <= g.pmax - window));
}
// (bounds of 640 threads: 96 registers, so that the five warps of one sub-partition fit)
template <bool kMixed>
__global__ void __launch_bounds__(640, 1) k_paged_prompt(const PagedArgs a, unsigned* err) {
  extern __shared__ unsigned char raw[];
  Smem<kMixed>& sm = *reinterpret_cast<Smem<kMixed>*>(raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u));
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(kFull, tid >> 5, 0);
  const int G = a.n_kv_heads, rank = (int)cluster_rank(), g = (blockIdx.x >> 1) % G, part = (blockIdx.x >> 1) / G;
  const bool reports = g == 0 && rank == 0;
  // scores in the log2 domain; a negative scale turns the queries' signs instead
  const float scale2 = fabsf(a.attn_scale) * 1.4426950408889634f;
  const uint32_t flip = a.attn_scale < 0.f ? 0x80008000u : 0u;
  const uint32_t stage0 = smem_u32(sm.stage[0]);
  const uint32_t bland = smem_u32(sm.landed), bfull = smem_u32(sm.full), bs = smem_u32(sm.s_full),
                 bp = smem_u32(sm.p_full), bpv = smem_u32(sm.pv_done), bq = smem_u32(&sm.q_full);
  // the even CTA's, where the products are issued
  const uint32_t lfull = dsmem_addr(sm.full, 0), lp = dsmem_addr(sm.p_full, 0), lq = dsmem_addr(&sm.q_full, 0);

  if constexpr (kMixed) {   // nothing to do: before anything is set up
    if (a.second) {
      grid_dep_wait();
      if (!*a.left) {
        if (tid == 0 && reports && !a.span_by_token) a.span[part] = make_int4(0, 0, 0, 0);
        return;
      }
    }
  }
  if (warp == 0) pair_alloc(smem_u32(&sm.tmem));
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bland + 8 * i, kGather);
      mbar_init(bfull + 8 * i, 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bs + 8 * i, 1);
      mbar_init(bp + 8 * i, 2 * kSoft / 32);
      mbar_init(bpv + 8 * i, 1);
    }
    mbar_init(bq, 2 * kSoft / 32);
    for (int i = 0; i < 4; ++i) sm.stray[i] = 0u;
  }
  grid_dep_wait();
  grid_dep_launch();
  plan<kNT, kCells, kMixed>(a, reinterpret_cast<int*>(sm.stage[0]), &sm.plan, tid, part, (int)(gridDim.x >> 1) / G, 1, kUncut,
                    a.n_tokens > (int)(gridDim.x >> 1) / G ? 6 + a.n_tokens / 128 : kUncut);
  const PlanOf<kMixed>& pl = sm.plan;
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist
  tc_fence_after();
  const uint32_t tmem = sm.tmem;
  bool timed_out = false;
  // The pair's runs, each role in a loop of its own that goes on to the next run by itself: the rows of its first tiles are
  // gathered while the sums of this one are still formed and written.  base, chunks: tiles of the runs before, and groups
  // of kSuper ids, from which stages, barriers and buffers go on.
  auto for_runs = [&](auto body) {
    int base = 0, runs = 0, chunks = 0, t0 = pl.t0, first = pl.first;
    for (int u = pl.u0; u < pl.u1; ++runs) {
      const Run run = run_at<kNT, kCells>(a, t0, first, pl.u1 - u);
      body(run, base, runs, chunks, u);
      u += run.n;
      base += run.n;
      chunks += (run.n + kSuper / kCells - 1) / (kSuper / kCells);
      t0 = next_group<kMixed>(a, pl, run.g.t0 + run.g.nt);
      first = 0;
    }
  };
  // loads in the order of the products: K of tile 0, then K of tile j + 1 and V of tile j, V of the last
  auto load_of_k = [](int i) { return i == 0 ? 0 : 2 * i - 1; };
  auto load_of_v = [](int i, int n) { return i == n - 1 ? 2 * n - 1 : 2 * i + 2; };

  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 136;\n");   // 2 x 136 + 2 x 56 of a sub-partition's 4 x 96
    auto load_q = [&](const Group& gr) {
#pragma unroll 8
      for (int i = tid; i < 128 * 32; i += kSoft) {   // piece i % 32 of row i / 32
        const int r = i >> 5, c16 = i & 31, t = 16 * rank + (r >> 3);
        uint4 x = make_uint4(0, 0, 0, 0);
        if (t < gr.nt)
          x = *reinterpret_cast<const uint4*>(a.q + ((int64_t)(gr.t0 + t) * G * kGqa + g * kGqa + (r & 7)) * kHeadDim + c16 * 8);
        x.x ^= flip, x.y ^= flip, x.z ^= flip, x.w ^= flip;
        *reinterpret_cast<uint4*>(sm.q + sw128(128, r, c16)) = x;
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) lead_arrive(lq);
    };
    for_runs([&](const Run& run, int base, int runs, int chunks, int u) {
      const Group& gr = run.g;
      const int n = run.n, v_first = run.first * kCells;
      // ---- softmax: row 32 (warp % 4) + lane, columns 64 half .. + 63
      const int quarter = warp & 3, half = warp >> 2, row = 32 * quarter + lane, tok = 16 * rank + (row >> 3), head = row & 7;
      const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
      if (runs == 0) load_q(gr);
      if (tid == 0) sm.stray[(runs + 2) & 3] = 0u;   // last read at the end of run `runs` - 2, which every warp has left
      const int pos = tok < gr.nt ? token_pos(a, gr.t0 + tok) : -1;
      // the reading-order range that the token sees, and its sinks
      const int vhi = pos - gr.lo_al + gr.ns_al + 1;
      const int vlo = a.window > 0 ? max(pos - a.window + 1 - gr.lo_al + gr.ns_al, gr.ns_al) : 0;
      const int vsink = gr.lo_al == 0 || gr.ns_al > 0 ? min(min(a.n_sink, pos + 1), gr.nv) : 0;
      const bool whole = n == gr.tiles;
      const int64_t ps = ((int64_t)(2 * part + (run.first == 0 ? 1 : 0)) * G + g) * (kNT * kGqa);   // the run's rows
      float* sums = a.of.o + ps * kHeadDim + 128 * half;
      const int stretch = stretch_of(n, kAdditions);
      int next = stretch;   // where the next one begins
      float fs = 0.f;       // of the stretches' sums so far
      bool odd = false;     // some of them are not finite
      float m = kNoMax, high = kNoMax, l = 0.f;   // the row's reference, the highest, this half's sum relative to it
      bool big = false;   // (see is_big)
      for (int i = 0; i < n; ++i) {
        const int b = (base + i) & 1;
        const uint32_t ts = tl + kColS + kCells * b + 64 * half;
        const int v0 = v_first + i * kCells + 64 * half;
        if (!mbar_wait(bs + 8 * b, (uint32_t)((base + i) >> 1) & 1u)) timed_out = true;
        tc_fence_after();
        const bool begins = i == next;
        float raised = 1.f;
        float s[64];
#pragma unroll
        for (int k = 0; k < 4; ++k) tmem_ld16_nowait(ts + 16 * k, reinterpret_cast<uint32_t*>(s + 16 * k));
        uint32_t see[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          see[k] = sm.ok[(chunks + (i >> 2)) & 3][(i & 3) * 4 + 2 * half + k] & below(vhi - v0 - 32 * k) &
                   (~below(vlo - v0 - 32 * k) | below(vsink - v0 - 32 * k));
        const bool all_seen = __all_sync(kFull, (see[0] & see[1]) == 0xffffffffu);
        tmem_wait_ld();
        if (!all_seen) {
#pragma unroll
          for (int j = 0; j < 64; ++j) s[j] = (see[j >> 5] >> (j & 31)) & 1u ? s[j] : -INFINITY;
        }
        float t4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
        for (int j = 4; j < 64; ++j) t4[j & 3] = fmaxf(t4[j & 3], s[j]);
        bool alone;
        const float top = tile_top(t4, scale2, alone);
        sm.max[b][half][row] = top;
        sm.alone[b][half][row] = alone;
        bar_named(2 + quarter, 64);   // the row's two threads
        const float nm = next_reference(m, high, top, sm.max[b][half ^ 1][row], alone || sm.alone[b][half ^ 1][row], big, scale2);
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
        // probabilities, in place: of 32 cells first parts in 16 columns, second parts in the next 16
        float ref = kUp - m, by = scale2;
        if (big) {
#pragma unroll
          for (int j = 0; j < 64; ++j) s[j] = __fsub_rn(__fmul_rn(s[j], scale2), m);
          ref = kUp, by = 1.f;
        }
        float sx = 0.f, sy = 0.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float x = s[32 * k + 2 * j], y = s[32 * k + 2 * j + 1];
            fma2(x, y, by, ref);
            if (!all_seen) {   // (times a scale of zero, -inf would be NaN)
              x = (see[k] >> (2 * j)) & 1u ? x : -INFINITY;
              y = (see[k] >> (2 * j + 1)) & 1u ? y : -INFINITY;
            }
            x = ex2(x), y = ex2(y);
            add2(sx, sy, x, y);
            float2 h;
            hi[j] = first_part(x, y, h);
            add2(x, y, -h.x, -h.y);
            lo[j] = bits(__floats2half2_rn(x, y));
          }
          tmem_st16(ts + 32 * k, hi);
          tmem_st16(ts + 32 * k + 16, lo);
        }
        l += sx + sy;
        if (edge_tile(gr, a.window, v_first + i * kCells)) {
          const int use = 2 * base + load_of_v(i, n);
          if (!mbar_wait(bland + 8 * (use % kStages), (uint32_t)(use / kStages) & 1u)) timed_out = true;
          uint4* v = reinterpret_cast<uint4*>(sm.stage[use % kStages]);
          bool found = false;
#pragma unroll 4
          for (int k = tid; k < (int)kStageBytes / 16; k += kSoft) {
            uint4 x = v[k];
            if (stray_halves(x.x) | stray_halves(x.y) | stray_halves(x.z) | stray_halves(x.w)) {
              x.x &= ~stray_halves(x.x), x.y &= ~stray_halves(x.y), x.z &= ~stray_halves(x.z), x.w &= ~stray_halves(x.w);
              v[k] = x;
              found = true;
            }
          }
          if (__any_sync(kFull, found)) {
            if (lane == 0) {
              st_dsmem_u32(dsmem_addr(&sm.stray[runs & 3], 0), 1u);
              st_dsmem_u32(dsmem_addr(&sm.stray[runs & 3], 1), 1u);
            }
            asm volatile("fence.acq_rel.cluster;\n" ::: "memory");
            fence_async_smem();
          }
        }
        tmem_wait_st();
        if (begins) {   // the sums of the stretch before, of the reference before
          if (!mbar_wait(bpv + 8 * (b ^ 1), (uint32_t)((base + i - 1) >> 1) & 1u)) timed_out = true;
          tc_fence_after();
          odd |= write_rows<true>(tl + 128 * half, sm.out[warp], 1.f, sums, kGqa * kHeadDim, i > stretch ? sums : nullptr, fs,
                                  128 * rank + 32 * quarter, gr.nt);
          fs = 1.f;
          next += stretch;
        }
        fs *= raised;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) lead_arrive(lp + 8 * b);
      }
      // ---- the run's result: a row of 256 values, 128 a thread
      if (!mbar_wait(bpv + 8 * ((base + n - 1) & 1), (uint32_t)((base + n - 1) >> 1) & 1u)) timed_out = true;
      tc_fence_after();
      if (u + n < pl.u1) load_q(run_at<kNT, kCells>(a, next_group<kMixed>(a, pl, gr.t0 + gr.nt), 0, 1).g);   // scores of the next run form meanwhile
      sm.sum[half][row] = l;
      bar_named(2 + quarter, 64);
      l = sm.sum[0][row] + sm.sum[1][row];
      if (tok < gr.nt && !whole && half == 0) *reinterpret_cast<float2*>(a.of.ml + 2 * (ps + tok * kGqa + head)) = make_float2(m, l);
      const float w = whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
      float* rows = whole ? a.out + ((int64_t)gr.t0 * G + g) * kGqa * kHeadDim + 128 * half : sums;
      const int64_t stride = (whole ? G : 1) * (kGqa * kHeadDim);
      odd |= write_rows<true>(tl + 128 * half, sm.out[warp], w, rows, stride, stretch < n ? sums : nullptr, fs,
                              128 * rank + 32 * quarter, gr.nt);
      // (the products of infinite values with a weight's second part, of zero or below it, are NaN; a row whose sum is not
      // finite is NaN throughout)
      odd = odd || *reinterpret_cast<volatile unsigned*>(&sm.stray[runs & 3]) != 0u;
      if (__any_sync(kFull, odd && tok < gr.nt && l - l == 0.f)) {
        put_not_finite(
            a, run, v_first, min(gr.nv, v_first + n * kCells),
            tok < gr.nt && l - l == 0.f ? rows + tok * stride + head * kHeadDim : nullptr,
            [&](int p) { return p <= pos && (a.window == 0 || p > pos - a.window || p < a.n_sink); },
            [&](int c, int k, uint32_t (&x)[8]) {
              const uint4* from = reinterpret_cast<const uint4*>(static_cast<const __half*>(a.v_cache) +
                                                                 ((int64_t)c * G + g) * kHeadDim + 128 * half + 16 * k);
              const uint4 lo = from[0], hi = from[1];
              x[0] = lo.x, x[1] = lo.y, x[2] = lo.z, x[3] = lo.w, x[4] = hi.x, x[5] = hi.y, x[6] = hi.z, x[7] = hi.w;
            });
      }
      tc_fence_before();
    });
  } else if (warp < 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 56;\n");
    for_runs([&](const Run& run, int base, int, int chunks, int) {
      const int n = run.n, v_first = run.first * kCells, v_end = min(run.g.nv, (run.first + n) * kCells);
      // ---- gather: of K the rows of cells 64 rank .. + 63 of a tile, of V dims 128 rank .. + 127 of all its cells
      const int tx = tid - kSoft, w8 = warp - 8;
      const unsigned char* kc = static_cast<const unsigned char*>(a.k_cache) + g * 512 + lane * 16;
      const unsigned char* vc = static_cast<const unsigned char*>(a.v_cache) + g * 512 + rank * 256 + (lane & 15) * 16;
      const uint32_t pitch = (uint32_t)G * 512u;
      constexpr int kPer = kSuper / kGather, kTiles = kSuper / kCells;
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
          if (lane == 0) sm.ok[(chunks + sc) & 3][i * 8 + w8] = ok;
        }
      };
      find_slots(0);
      find_cells(0);
      bar_named(1, kGather);   // the ids of the run before have been read
      keep_cells(0);
      find_slots(1);
      find_cells(1);
      find_slots(2);
      bar_named(1, kGather);
      for (int L = 0; L < 2 * n; ++L) {
        const int use = 2 * base + L, st = use % kStages;
        const bool is_k = L == 0 || (L & 1 && L != 2 * n - 1);
        const int i = L == 0 ? 0 : L == 2 * n - 1 ? n - 1 : is_k ? (L + 1) >> 1 : (L >> 1) - 1;
        // the ids of tiles kTiles * sc .. are kept before the first K load of the group before
        if (is_k && i % kTiles == 0) {
          const int sc = i / kTiles;
          bar_named(1, kGather);   // the ids two groups before have been read
          if (sc > 0) {
            keep_cells(sc);
            find_cells(sc + 1);
            find_slots(sc + 2);
            bar_named(1, kGather);
          }
        }
        // A tile's K rows follow the scores, its V rows the sums, of the tile two before.  That frees their stage, also where
        // a run ends: products end in the order in which they take their rows.  (And each phase is waited for in turn.)
        const int x = base + i;
        if (x >= 2 && !mbar_wait((is_k ? bs : bpv) + 8 * (x & 1), (uint32_t)((x - 2) >> 1) & 1u)) timed_out = true;
        const int* id = &sm.ids[(chunks + i / kTiles) & 1][(i % kTiles) * kCells];
        const uint32_t stage = stage0 + st * kStageBytes;
        if (is_k) {
          const uint32_t dst = stage + (lane >> 3) * 8192;
#pragma unroll 8
          for (int k = 0; k < 8; ++k) {   // a warp a row, its 32 pieces of 16 bytes
            const int row = 8 * k + w8, c = id[64 * rank + row];
            cp_async16(dst + row * 128 + (((lane & 7) ^ (row & 7)) << 4), kc + (uint64_t)(uint32_t)max(c, 0) * pitch, c >= 0);
          }
        } else {
          const uint32_t dst = stage + ((lane >> 3) & 1) * 16384;
#pragma unroll 8
          for (int k = 0; k < 8; ++k) {   // a warp two rows
            const int row = 16 * k + 2 * w8 + (lane >> 4), c = id[row];
            cp_async16(dst + row * 128 + (((lane & 7) ^ (row & 7)) << 4), vc + (uint64_t)(uint32_t)max(c, 0) * pitch, c >= 0);
          }
        }
        // arrives when this thread's copies so far have landed
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];\n" ::"r"(bland + 8 * st) : "memory");
      }
    });
    asm volatile("cp.async.wait_all;\n" ::: "memory");
  } else if (warp == 16) {
    // ---- what has landed here becomes visible to the products
    if (lane == 0 && reports && !a.span_by_token) a.span[part] = make_int4(0, 0, 0, 0);
    for_runs([&](const Run& run, int base, int, int, int u) {
      if (reports) announce(a, pl, run, part, u, err);
      for (int use = 2 * base; use < 2 * (base + run.n); ++use) {
        const int st = use % kStages;
        if (!mbar_wait(bland + 8 * st, (uint32_t)(use / kStages) & 1u)) timed_out = true;
        fence_async_smem();
        __syncwarp();
        if (lane == 0) lead_arrive(lfull + 8 * st);
      }
    });
  } else {
    // ---- the products, in the order in which the tensor cores take them: scores of tile i + 2 behind P V of tile i,
    // whose columns they take
    for_runs([&](const Run& run, int base, int runs, int, int) {
      if (rank != 0) return;
      const int n = run.n;
      const uint32_t q = smem_u32(sm.q);
      if (!mbar_wait(bq, (uint32_t)runs & 1u)) timed_out = true;
      auto loaded = [&](int L) {
        const int use = 2 * base + L;
        if (!mbar_wait(bfull + 8 * (use % kStages), (uint32_t)(use / kStages) & 1u)) timed_out = true;
      };
      auto scores = [&](int i) {
        const int b = (base + i) & 1;
        const uint32_t k = stage0 + (2 * base + load_of_k(i)) % kStages * kStageBytes;
#pragma unroll
        for (int kk = 0; kk < 16; ++kk)
          pair_mma(tmem + kColS + kCells * b, smem_desc(q + (kk >> 2) * 16384 + (kk & 3) * 32, 16, 1024),
                   smem_desc(k + (kk >> 2) * 8192 + (kk & 3) * 32, 16, 1024), kIdescS, kk > 0);
        pair_commit(bs + 8 * b);
      };
      loaded(load_of_k(0));
      tc_fence_after();
      scores(0);
      if (n > 1) {
        loaded(load_of_k(1));
        scores(1);
      }
      loaded(load_of_v(0, n));
      const int stretch = stretch_of(n, kAdditions);
      int first = 0;   // of the stretch
      for (int i = 0; i < n; ++i) {   // (an issue ends some 500 cycles before its products: waits that pass at once cost nothing)
        const int b = (base + i) & 1;
        if (i == first + stretch) first = i;
        if (i + 2 < n) loaded(load_of_k(i + 2));
        if (!mbar_wait(bp + 8 * b, (uint32_t)((base + i) >> 1) & 1u)) timed_out = true;
        tc_fence_after();
        const uint32_t v = stage0 + (2 * base + load_of_v(i, n)) % kStages * kStageBytes;
#pragma unroll
        for (int second = 0; second < 2; ++second)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            pair_mma_ts(tmem, tmem + kColS + kCells * b + 32 * (kk >> 1) + 16 * second + 8 * (kk & 1),
                        smem_desc(v + kk * 2048, 16384, 1024), kIdescO, i > first || second > 0 || kk > 0);
        pair_commit(bpv + 8 * b);
        if (i + 2 < n) scores(i + 2);
        if (i + 1 < n) loaded(load_of_v(i + 1, n));
      }
    });
  }
  if (timed_out) atomicOr(err, kErrTimeout);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  if (warp == 0) pair_dealloc(tmem);
}

constexpr int kMaxDevices = 64;

template <bool kMixed>
cudaError_t launch(const PagedArgs& a, unsigned* err, cudaStream_t stream) {
  static std::atomic<bool> known[kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!known[dev].load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(mu);
    e = cudaFuncSetAttribute(k_paged_prompt<kMixed>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes<kMixed>);
    if (e != cudaSuccess) return e;
    known[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(k_paged_prompt<kMixed>, dim3((unsigned)(2 * a.of.parts * a.n_kv_heads)), dim3(kThreads), kSmemBytes<kMixed>, stream, 2,
                    a, err);
}

}  // namespace

cudaError_t launch_paged_prompt(const PagedArgs& a, bool mixed, unsigned* err, cudaStream_t stream) {
  return mixed ? launch<true>(a, err, stream) : launch<false>(a, err, stream);
}

}  // namespace qsa
