// Attention over a paged cache for single tokens of their sequences (decoding).
//
// One token's 8 heads of a KV head are too few for warps to share the work on a
// tile: the exchange of maxima and probabilities would cost more than the products.
// So a warp takes 16 cells at a time for itself: it copies their rows with
// cp.async, two chunks ahead, each half of a chunk (K rows, V rows) refilled as soon
// as it is read; forms the scores of 16 cells x 8 heads (mma.sync, cells as rows);
// and adds P.V for all 256 dims, V^T as the operand with 16 rows, the probabilities
// transposed in registers.  Warps share nothing until a run of chunks ends.  Chunks
// of all tokens, laid end to end, are dealt in equal runs to the CTAs of a KV head,
// one CTA an SM.
//
// Codes enter the products as
// integers, K scales apply to a block's sum, V scales to the probabilities, which go
// in as two fp16 parts (22 bits); sums are fp32.  A half keeps its bits 30 binary places below the
// largest only, so the weights p * d_V are relative to the chunk's largest
// probability (2^15) and largest scale ([1/4, 1/2)): they are off by 2^-22 of
// themselves or by 2^-39 of that largest product.  Where a chunk's scales of V lie
// more than 2^10 apart they are relative to the block's largest, and where those of a
// block do, or are infinite or NaN, its cells are added one by one, each relative to
// its own.
//
// What bounds it: fp16 rows the gather (64 sequences of up to 8,000 cells: 134 us,
// 5.2 TB/s; a gather of rows reaches 5.7 to 6.3), codes the warps' chains of dependent
// instructions (250k q8_0: 63 us, 4.3 TB/s, 50 % of the issue slots; 5 x 250k q4_0:
// 144 us, 63 %), as shared memory holds rows for 12 warps and registers sums for 16.
// One token over 50k fp16 cells takes 30 us, of which the rows take 17: the plan 1, the
// ids 2, the merge and the join 7.
#include <atomic>
#include <mutex>

#include "attn_paged.cuh"
#include "tc_util.cuh"

namespace qsa {
namespace {

constexpr int kChunk = 16;                       // cells of one warp step
constexpr int kBlocks = kHeadDim / 32;
constexpr float kUp = 15.f;                      // probabilities are held as 2^(s - m + kUp)
constexpr unsigned kSpread = 10u << 10;          // (bits of a half) of a chunk's V scales
constexpr int kPitchO = kHeadDim + 4;            // floats between two heads of a warp's o: its stores do not conflict
constexpr int kMinChunks = 4;                    // of a part

// A row: codes then scales.  Warps: as many as two chunks of each fit shared memory
// with (fp16), or as the registers allow with 128 each.
template <int KV> struct Row;
template <> struct Row<QSA_KV_F16> { static constexpr int kCodes = 512, kPitch = 528, kWarps = 6; };
template <> struct Row<QSA_KV_Q8_0> { static constexpr int kCodes = 256, kPitch = 272, kWarps = 12; };
template <> struct Row<QSA_KV_Q4_0> { static constexpr int kCodes = 128, kPitch = 144, kWarps = 16; };

template <int KV, bool kMixed>
struct Smem {
  using R = Row<KV>;
  static constexpr int kHalf = kChunk * R::kPitch;
  alignas(16) unsigned char stage[R::kWarps][2][2][kHalf];   // K rows, V rows; after a run: each warp's o, fp32 [8][kPitchO]
  uint4 q[kBlocks][32];                          // a lane's query fragments of 32 dims
  uint2 vd[R::kWarps][kBlocks][4];               // a chunk's V scales: block, l4 -> cells 2 l4 + {0, 1, 8, 9}
  float m[R::kWarps][kGqa], l[R::kWarps][kGqa];
  float ml[2][kGqa];                             // the run's (max, sum)
  PlanOf<kMixed> plan;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm2t(uint32_t addr, uint32_t (&r)[2]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];\n" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma0(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// An 8 x 8 tile of halves, two of a row per lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// (sx, sy) += (dx, dy) * (cx, cy)
__device__ __forceinline__ void add_products2(float& sx, float& sy, float dx, float dy, float cx, float cy) {
  asm("{\n .reg .b64 s, d, c;\n mov.b64 s, {%0, %1};\n mov.b64 d, {%2, %3};\n mov.b64 c, {%4, %5};\n"
      " fma.rn.f32x2 s, d, c, s;\n mov.b64 {%0, %1}, s;\n}\n"
      : "+f"(sx), "+f"(sy)
      : "f"(dx), "f"(dy), "f"(cx), "f"(cy));
}
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t o) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;\n" : "=r"(r) : "r"(x), "r"(m), "r"(o));
  return r;
}
// Signed bytes (i, j) of x ^ 0x80808080 as halves.
template <int kSel>
__device__ __forceinline__ uint32_t signed2(uint32_t x) {
  return bits(bytes2<kSel>(x, 0x64806480u));
}
// Codes less 8 in bits 0..3 of x's two halves.
__device__ __forceinline__ uint32_t nibbles2(uint32_t x) {
  return bits(__hsub2(half2_of(and_or(x, 0x000f000fu, 0x64006400u)), half2_of(0x64086408u)));
}
// Those in bits 4..7, without a shift: 1024 + 16 c, a sixteenth of which is 64 + c, both exact.
__device__ __forceinline__ uint32_t high_nibbles2(uint32_t x) {
  return bits(__hfma2(half2_of(and_or(x, 0x00f000f0u, 0x64006400u)), half2_of(0x2c002c00u), half2_of(0xd480d480u)));
}
// x, infinities as NaN: a block of such values holds infinities of both signs and NaN
__device__ __forceinline__ __half2 nan_of_inf(__half2 x) { return __hfma2(x, half2_of(0u), x); }
// 2^k as a half, k in [-24, 15]
__device__ __forceinline__ __half2 pow2h(int k) {
  const uint32_t e = k >= -14 ? (uint32_t)(k + 15) << 10 : 1u << (k + 24);
  return half2_of(e | (e << 16));
}

template <int KV, bool kMixed>
__global__ void __launch_bounds__(Row<KV>::kWarps * 32, 1) k_paged_one(const PagedArgs a, unsigned* err) {
  extern __shared__ unsigned char smem_raw[];
  using R = Row<KV>;
  using S = Smem<KV, kMixed>;
  S& sm = *reinterpret_cast<S*>(smem_raw);
  constexpr int kWarps = R::kWarps, kThreads = 32 * kWarps, kCodes = R::kCodes, kPitch = R::kPitch;
  constexpr bool kF16 = KV == QSA_KV_F16;
  static_assert(sizeof(sm.stage[0]) >= kGqa * kPitchO * 4 && sizeof(sm.stage) >= kPlanScratch, "what the stages hold besides rows");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gid = lane >> 2, l4 = lane & 3;
  const int G = a.n_kv_heads, g = blockIdx.x % G, part = blockIdx.x / G;
  const float scale2 = a.attn_scale * 1.4426950408889634f;   // scores in the log2 domain

  grid_dep_wait();
  grid_dep_launch();
  plan<1, kChunk, kMixed>(a, reinterpret_cast<int*>(sm.stage), &sm.plan, tid, part, gridDim.x / G, kMinChunks, kWarps, 2 * kWarps);   // (a chunk a warp)
  const PlanOf<kMixed>& pl = sm.plan;
  if (tid == 0 && g == 0 && !a.span_by_token) a.span[part] = make_int4(0, 0, 0, 0);

  const unsigned char* kc = static_cast<const unsigned char*>(a.k_cache) + g * kCodes;
  const unsigned char* vc = static_cast<const unsigned char*>(a.v_cache) + g * kCodes;
  const uint32_t pitch = (uint32_t)G * kCodes;                                 // code bytes of a cell
  const unsigned char* ks = static_cast<const unsigned char*>(a.k_cache) + a.n_cells * (int64_t)pitch + g * 16;
  const unsigned char* vs = static_cast<const unsigned char*>(a.v_cache) + a.n_cells * (int64_t)pitch + g * 16;
  const uint32_t ring = smem_u32(sm.stage[warp]);
  constexpr uint32_t kHalf = S::kHalf;

  int t_next = pl.t0, first_next = pl.first;
  for (int u = pl.u0; u < pl.u1;) {
    const Run run = run_at<1, kChunk>(a, t_next, first_next, pl.u1 - u);
    const Group& gr = run.g;
    const int t0 = gr.t0, n = run.n, v_end = min(gr.nv, (run.first + n) * kChunk);
    if (warp == 0 && g == 0) announce(a, pl, run, part, u, err);
    u += n;
    t_next = next_group<kMixed>(a, pl, t0 + 1);
    first_next = 0;

    // ---- ids: position -> slot -> cell, a step of the warp's chunks apart; lanes i and i + 16 hold cell i
    auto find_slot = [&](int k) -> int {
      return k < n ? slot_at(a, run, (run.first + k) * kChunk + (lane & 15), v_end, g == 0 && lane < 16, err) : -1;
    };
    auto find_cell = [&](int k, int slot) -> int {
      return cell_at(a, run, (run.first + k) * kChunk + (lane & 15), slot, g == 0 && lane < 16, err);
    };
    // copies a chunk's rows; missing cells become zeros
    auto fetch = [&](int cell, uint32_t dst, const unsigned char* codes, const unsigned char* scales) {
      constexpr int kLanes = kCodes / 16, kRows = 32 / kLanes;
      const uint32_t to = dst + (lane / kLanes) * kPitch + (lane % kLanes) * 16;
      const unsigned char* from = codes + (lane % kLanes) * 16;
      if (__all_sync(kFull, cell >= 0)) {
#pragma unroll
        for (int k = 0; k < kChunk; k += kRows) {
          const int c = __shfl_sync(kFull, cell, k + lane / kLanes);
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"(to + k * kPitch), "l"(from + (uint64_t)(uint32_t)c * pitch)
                       : "memory");
        }
      } else {
#pragma unroll
        for (int k = 0; k < kChunk; k += kRows) {
          const int c = __shfl_sync(kFull, cell, k + lane / kLanes);
          cp_async16(to + k * kPitch, from + (uint64_t)(uint32_t)max(c, 0) * pitch, c >= 0);
        }
      }
      if constexpr (!kF16) {
        if (lane < kChunk) cp_async16(dst + lane * kPitch + kCodes, scales + (uint64_t)(uint32_t)max(cell, 0) * (uint32_t)(G * 16), cell >= 0);
      }
    };
    int cell[2];   // of the chunks in flight
    int ahead, slot;
    {
      const int s0 = find_slot(warp), s1 = find_slot(warp + kWarps), s2 = find_slot(warp + 2 * kWarps);
      slot = find_slot(warp + 3 * kWarps);
      const int c0 = find_cell(warp, s0), c1 = find_cell(warp + kWarps, s1);
      ahead = find_cell(warp + 2 * kWarps, s2);
      cell[0] = checked_cell(a, c0, g == 0 && lane < 16, err);
      cell[1] = checked_cell(a, c1, g == 0 && lane < 16, err);
    }
    __syncthreads();   // the run before is done with shared memory
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (warp + s * kWarps < n) fetch(cell[s], ring + 2 * s * kHalf, kc, ks);
      asm volatile("cp.async.commit_group;\n" ::: "memory");
      if (warp + s * kWarps < n) fetch(cell[s], ring + (2 * s + 1) * kHalf, vc, vs);
      asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
    // ---- the queries, as fragments of 32 dims: those of a lane's k indices, in the order of the rows' bytes
    for (int i = tid; i < kBlocks * 32; i += kThreads) {
      const int ln = i & 31, b = i >> 5, h = ln >> 2, q4 = ln & 3;
      const __half* q = a.q + ((int64_t)t0 * G * kGqa + g * kGqa + h) * kHeadDim + 32 * b;
      auto two = [&](int d) { return *reinterpret_cast<const uint32_t*>(q + d); };
      uint4 x;
      if constexpr (KV == QSA_KV_F16) {
        x = make_uint4(two(2 * q4), two(8 + 2 * q4), two(16 + 2 * q4), two(24 + 2 * q4));
      } else if constexpr (KV == QSA_KV_Q8_0) {
        x = make_uint4(two(4 * q4), two(4 * q4 + 2), two(16 + 4 * q4), two(18 + 4 * q4));
      } else {   // dims 4 l4 + {0, 2}, 4 l4 + {1, 3}, and the 16 further
        const uint2 lo = *reinterpret_cast<const uint2*>(q + 4 * q4), hi = *reinterpret_cast<const uint2*>(q + 16 + 4 * q4);
        x = make_uint4(__byte_perm(lo.x, lo.y, 0x5410), __byte_perm(lo.x, lo.y, 0x7632), __byte_perm(hi.x, hi.y, 0x5410),
                       __byte_perm(hi.x, hi.y, 0x7632));
      }
      sm.q[b][ln] = x;
    }
    __syncthreads();

    float acc[kBlocks][2][4];
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[b][i][j] = 0.f;
    float run_m[2] = {kNoMax, kNoMax}, run_l[2] = {0.f, 0.f};   // of heads 2 l4, 2 l4 + 1; run_l: this lane's cells only

    int st = 0;
#pragma unroll 1
    for (int k = warp; k < n; k += kWarps, st ^= 1) {
      const uint32_t sk = ring + 2 * st * kHalf, sv = sk + kHalf;
      const unsigned ok = __ballot_sync(kFull, cell[0] >= 0);   // bits i and i + 16: cell i
      cell[0] = cell[1];
      cell[1] = k + 2 * kWarps < n ? checked_cell(a, ahead, g == 0 && lane < 16, err) : -1;
      ahead = find_cell(k + 3 * kWarps, slot);
      slot = find_slot(k + 4 * kWarps);
      asm volatile("cp.async.wait_group 3;\n" ::: "memory");
      __syncwarp();   // every lane's copies of the K rows are in

      // ---- scores: s[j] of cell gid + 8 j with heads 2 l4, 2 l4 + 1
      float2 s[2] = {};
      float dk[2][8];
      if constexpr (!kF16) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint4 d;
          asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                       : "=r"(d.x), "=r"(d.y), "=r"(d.z), "=r"(d.w) : "r"(sk + (gid + 8 * j) * kPitch + kCodes) : "memory");
          const uint32_t x[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const float2 f = __half22float2(nan_of_inf(half2_of(x[b])));
            dk[j][2 * b] = f.x, dk[j][2 * b + 1] = f.y;
          }
        }
      }
      const uint32_t arow = sk + (lane & 15) * kPitch + (lane >> 4) * 16;   // of the four 8 x 16-byte pieces: rows 0-7, 8-15, then 16 bytes on
      if constexpr (KV == QSA_KV_F16) {
        float c[2][4];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const uint4 q = sm.q[b][lane];
          uint32_t w[4];
          ldsm4(arow + 64 * b, w);
          if (b == 0) mma0(c[0], w, q.x, q.y); else mma(c[0], w, q.x, q.y);
          ldsm4(arow + 64 * b + 32, w);
          if (b == 0) mma0(c[1], w, q.z, q.w); else mma(c[1], w, q.z, q.w);
        }
        s[0] = make_float2(c[0][0] + c[1][0], c[0][1] + c[1][1]);
        s[1] = make_float2(c[0][2] + c[1][2], c[0][3] + c[1][3]);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) {
          const uint4 q = sm.q[b][lane];
          uint32_t x0[4], x1[4];
          if constexpr (KV == QSA_KV_Q8_0) {
            ldsm4(arow + 32 * b, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] ^= 0x80808080u;
            x0[0] = signed2<0x4140>(w[0]), x0[1] = signed2<0x4140>(w[1]), x0[2] = signed2<0x4342>(w[0]), x0[3] = signed2<0x4342>(w[1]);
            x1[0] = signed2<0x4140>(w[2]), x1[1] = signed2<0x4140>(w[3]), x1[2] = signed2<0x4342>(w[2]), x1[3] = signed2<0x4342>(w[3]);
          } else {
            if ((b & 1) == 0) ldsm4(arow + 16 * b, w);
            const uint32_t w0 = w[2 * (b & 1)], w1 = w[2 * (b & 1) + 1];
            const uint32_t v0 = w0 >> 8, v1 = w1 >> 8;
            x0[0] = nibbles2(w0), x0[1] = nibbles2(w1), x0[2] = nibbles2(v0), x0[3] = nibbles2(v1);
            x1[0] = high_nibbles2(w0), x1[1] = high_nibbles2(w1), x1[2] = high_nibbles2(v0), x1[3] = high_nibbles2(v1);
          }
          float c[4];
          mma0(c, x0, q.x, q.y);
          mma(c, x1, q.z, q.w);
          s[0].x = fmaf(dk[0][b], c[0], s[0].x), s[0].y = fmaf(dk[0][b], c[1], s[0].y);
          s[1].x = fmaf(dk[1][b], c[2], s[1].x), s[1].y = fmaf(dk[1][b], c[3], s[1].y);
        }
      }
      __syncwarp();   // the K rows have been read
      if (k + 2 * kWarps < n) fetch(cell[1], sk, kc, ks);
      asm volatile("cp.async.commit_group;\n" ::: "memory");

      // ---- softmax of the two heads over the 16 cells (8 lanes hold them)
      s[0].x *= scale2, s[0].y *= scale2, s[1].x *= scale2, s[1].y *= scale2;
      if (ok != kFull) {   // missing cells: p = 0
        if (!((ok >> gid) & 1u)) s[0].x = s[0].y = -INFINITY;
        if (!((ok >> (gid + 8)) & 1u)) s[1].x = s[1].y = -INFINITY;
      }
      float m[2] = {fmaxf(s[0].x, s[1].x), fmaxf(s[0].y, s[1].y)};
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1)
#pragma unroll
        for (int h = 0; h < 2; ++h) m[h] = fmaxf(m[h], __shfl_xor_sync(kFull, m[h], o));
      float f[2], fac[2];   // of the sums so far, of the chunk
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        m[h] = fmaxf(m[h], kNoMax);
        const float nm = fmaxf(run_m[h], m[h]);
        f[h] = ex2(run_m[h] - nm);
        fac[h] = ex2(m[h] - nm);
        run_m[h] = nm;
      }
      float p[2][2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        p[j][0] = ex2(s[j].x - m[0] + kUp);
        p[j][1] = ex2(s[j].y - m[1] + kUp);
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) run_l[h] = fmaf(p[0][h] + p[1][h], fac[h], run_l[h] * f[h]);
      if (a.weigh) {   // the sums of whole blocks: cells gid + 8 j are 4 lanes apart
        const int per = kChunk >> a.r_shift;
        const int64_t row = ((int64_t)t0 * G + g) * kGqa + 2 * l4;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float e = p[j][h];
            for (int o = 0; o < a.r_shift; ++o) e += __shfl_xor_sync(kFull, e, 4 << o);
            if ((gid & ((1 << a.r_shift) - 1)) == 0)
              a.e[(row + h) * a.e_blocks + (int64_t)(run.first + k) * per + ((gid + 8 * j) >> a.r_shift)] = e;
          }
        if (gid == 0) {
          a.em[row * a.e_tiles + run.first + k] = m[0];
          a.em[(row + 1) * a.e_tiles + run.first + k] = m[1];
        }
      }
      // the probabilities in two parts, from (cell, heads) to (head, cells)
      uint32_t ph[2], pw[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const __half2 hi = __floats2half2_rn(p[j][0], p[j][1]);
        const float2 x = __half22float2(hi);
        ph[j] = transposed(bits(hi));
        pw[j] = transposed(bits(__floats2half2_rn(p[j][0] - x.x, p[j][1] - x.y)));
      }
      if (__any_sync(kFull, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[b][i][j] *= f[j & 1];
      }

      asm volatile("cp.async.wait_group 3;\n" ::: "memory");
      __syncwarp();   // the V rows
      // tile i of a block, rows gid and gid + 8: dims 16 i + gid and 8 more (fp16); 2 gid + i and 16 more (codes)
      const uint32_t vrow = sv + ((lane & 7) + ((lane >> 4) << 3)) * kPitch + ((lane >> 3) & 1) * 16;
      if constexpr (kF16) {
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t x[4];
            float c[4];
            ldsm4t(vrow + 64 * b + 32 * i, x);
            mma0(c, x, ph[0], ph[1]);
            mma(c, x, pw[0], pw[1]);
            add_products2(acc[b][i][0], acc[b][i][1], fac[0], fac[1], c[0], c[1]);
            add_products2(acc[b][i][2], acc[b][i][3], fac[0], fac[1], c[2], c[3]);
          }
      } else {
        // the chunk's scales: this lane those of cells 2 l4 + {0, 1, 8, 9} in block gid
        __half2 dv[2];
        uint32_t top, least;
        {
          uint32_t d[2];
          ldsm2t(sv + (lane & 15) * kPitch + kCodes, d);
          dv[0] = nan_of_inf(half2_of(d[0])), dv[1] = nan_of_inf(half2_of(d[1]));
          const uint32_t a0 = d[0] & 0x7fff7fffu, a1 = d[1] & 0x7fff7fffu;
          top = max(max(a0 & 0xffffu, a0 >> 16), max(a1 & 0xffffu, a1 >> 16));
          // the smallest of those that are not zero
          auto not0 = [](uint32_t x) { return x == 0u ? 0x7fffu : x; };
          least = min(min(not0(a0 & 0xffffu), not0(a0 >> 16)), min(not0(a1 & 0xffffu), not0(a1 >> 16)));
        }
        // one exponent for the chunk brings its largest scale to [1/4, 1/2), if all lie close together; else each block its own
        const uint32_t top_all = __reduce_max_sync(kFull, top), least_all = __reduce_min_sync(kFull, least);
        const bool close = top_all < 0x7c00u && (top_all == 0u || (least_all >= 0x0400u && top_all <= least_all + kSpread));
        bool plain = close;
        int ve = top_all == 0u ? 0 : 13 - min(max((int)(top_all >> 10), 1), 30);
        if (!close) {
          top = max(top, __shfl_xor_sync(kFull, top, 1));
          top = max(top, __shfl_xor_sync(kFull, top, 2));
          least = min(least, __shfl_xor_sync(kFull, least, 1));
          least = min(least, __shfl_xor_sync(kFull, least, 2));
          plain = __all_sync(kFull, top < 0x7c00u && (top == 0u || (least >= 0x0400u && top <= least + kSpread)));
          ve = top == 0u ? 0 : 13 - min(max((int)(top >> 10), 1), 30);
        }
        if (plain) {
          const __half2 up = pow2h(ve);
          sm.vd[warp][gid][l4] = make_uint2(bits(__hmul2(dv[0], up)), bits(__hmul2(dv[1], up)));
          __syncwarp();
        }
        // adds the chunk's products of block b, with weights of the scales d0, d1 (scaled by 2^e)
        auto add = [&](int b, const uint32_t (&w)[4], __half2 d0, __half2 d1, uint32_t h0, uint32_t h1, uint32_t l0, uint32_t l1,
                       float f0, float f1) {
          const __half2 a0 = half2_of(h0), a1 = half2_of(h1);
          const __half2 x0 = __hmul2(a0, d0), x1 = __hmul2(a1, d1);
          const uint32_t y0 = bits(__hfma2(half2_of(l0), d0, __hfma2(a0, d0, __hneg2(x0))));
          const uint32_t y1 = bits(__hfma2(half2_of(l1), d1, __hfma2(a1, d1, __hneg2(x1))));
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t x[4];
            if constexpr (KV == QSA_KV_Q8_0) {
#pragma unroll
              for (int j = 0; j < 4; ++j) x[j] = i == 0 ? signed2<0x4240>(w[j]) : signed2<0x4341>(w[j]);
            } else {   // w[0], w[1]: the block's bytes of cells 0-7, 8-15
              const uint32_t v0 = w[0] >> (8 * i), v1 = w[1] >> (8 * i);
              x[0] = nibbles2(v0), x[1] = high_nibbles2(v0), x[2] = nibbles2(v1), x[3] = high_nibbles2(v1);
            }
            float c[4];
            mma0(c, x, bits(x0), bits(x1));
            mma(c, x, y0, y1);
            add_products2(acc[b][i][0], acc[b][i][1], f0, f1, c[0], c[1]);
            add_products2(acc[b][i][2], acc[b][i][3], f0, f1, c[2], c[3]);
          }
        };
        // the block's codes: q8_0 four pieces (dims 0-15, 16-31 of cells 0-7, then 8-15); q4_0 two blocks at a time
        auto codes = [&](int b, uint32_t (&w)[4], uint32_t (&two)[4]) {
          if constexpr (KV == QSA_KV_Q8_0) {
            ldsm4t(vrow + 32 * b, w);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] ^= 0x80808080u;
          } else {
            if ((b & 1) == 0) ldsm4t(sv + (lane & 15) * kPitch + 16 * b + (lane >> 4) * 16, two);
            w[0] = two[2 * (b & 1)], w[1] = two[2 * (b & 1) + 1], w[2] = w[3] = 0u;
          }
        };
        if (close) {
          uint32_t w[4], two[4];
          const float back = __uint_as_float((uint32_t)(127 - ve) << 23), f0 = fac[0] * back, f1 = fac[1] * back;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            codes(b, w, two);
            const uint2 d = sm.vd[warp][b][l4];
            add(b, w, half2_of(d.x), half2_of(d.y), ph[0], ph[1], pw[0], pw[1], f0, f1);
          }
        } else if (plain) {
          uint32_t w[4], two[4];
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            codes(b, w, two);
            const uint2 d = sm.vd[warp][b][l4];
            const float back = __uint_as_float((uint32_t)(127 - __shfl_sync(kFull, ve, 4 * b)) << 23);
            add(b, w, half2_of(d.x), half2_of(d.y), ph[0], ph[1], pw[0], pw[1], fac[0] * back, fac[1] * back);
          }
        } else {
          // cell by cell (this lane's weights of all other cells are zero), each block relative to the cell's scale
#pragma unroll 1
          for (int cellno = 0; cellno < kChunk; ++cellno) {
            const bool mine = ((cellno >> 1) & 3) == l4;
            const uint32_t keep = mine ? 0xffffu << (16 * (cellno & 1)) : 0u;
            const uint32_t k0 = cellno < 8 ? keep : 0u, k1 = cellno < 8 ? 0u : keep;
            uint32_t w[4], two[4];
#pragma unroll
            for (int b = 0; b < kBlocks; ++b) {
              codes(b, w, two);
              const uint32_t pair = __shfl_sync(kFull, bits(cellno < 8 ? dv[0] : dv[1]), 4 * b + ((cellno >> 1) & 3));
              const uint32_t d = (pair >> (16 * (cellno & 1))) & 0xffffu;
              const int e = 13 - min(max((int)((d & 0x7fffu) >> 10), 1), 30);
              const __half2 both = __hmul2(half2_of(d * 0x00010001u), pow2h(e));
              const __half2 z = half2_of(0u);
              add(b, w, k0 ? both : z, k1 ? both : z, ph[0] & k0, ph[1] & k1, pw[0] & k0, pw[1] & k1,
                  fac[0] * __uint_as_float((uint32_t)(127 - e) << 23), fac[1] * __uint_as_float((uint32_t)(127 - e) << 23));
            }
          }
        }
      }
      __syncwarp();   // the V rows have been read
      if (k + 2 * kWarps < n) fetch(cell[1], sv, vc, vs);
      asm volatile("cp.async.commit_group;\n" ::: "memory");
    }
    asm volatile("cp.async.wait_all;\n" ::: "memory");

    // ---- the run's result: the warps' (max, sum, o) in warp order
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) run_l[h] += __shfl_xor_sync(kFull, run_l[h], o);
      if (gid == 0) {
        sm.m[warp][2 * l4 + h] = run_m[h];
        sm.l[warp][2 * l4 + h] = run_l[h];
      }
    }
    __syncthreads();   // also: every warp is done with its stages
    {
      float* o = reinterpret_cast<float*>(sm.stage[warp]);
      float f[2];   // of heads 2 l4, 2 l4 + 1
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float m = kNoMax;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][2 * l4 + h]);
        f[h] = ex2(run_m[h] - m);
      }
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float* x = o + (2 * l4 + h) * kPitchO + 32 * b;
          if constexpr (kF16) {
#pragma unroll
            for (int i = 0; i < 2; ++i) x[16 * i + gid] = acc[b][i][h] * f[h], x[16 * i + 8 + gid] = acc[b][i][2 + h] * f[h];
          } else {
            *reinterpret_cast<float2*>(x + 2 * gid) = make_float2(acc[b][0][h] * f[h], acc[b][1][h] * f[h]);
            *reinterpret_cast<float2*>(x + 16 + 2 * gid) = make_float2(acc[b][0][2 + h] * f[h], acc[b][1][2 + h] * f[h]);
          }
        }
    }
    if (tid < kGqa) {
      float m = kNoMax, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][tid]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) l = fmaf(sm.l[w][tid], ex2(sm.m[w][tid] - m), l);
      sm.ml[0][tid] = m;
      sm.ml[1][tid] = l;
    }
    __syncthreads();
    const bool whole = n == gr.tiles;
    const int64_t ps = ((int64_t)(2 * part + (run.first == 0 ? 1 : 0)) * G + g) * kGqa;   // the run's rows in the workspace
    float* out = whole ? a.out + ((int64_t)t0 * G + g) * kGqa * kHeadDim : a.of.o + ps * kHeadDim;
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 15u) == 0u;
    float odd = 0.f;   // zero, or NaN
    for (int i = tid; i < kGqa * kHeadDim / 4; i += kThreads) {
      const int h = i >> 6, d = (i & 63) * 4;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 y = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.stage[w]) + h * kPitchO + d);
        x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
      }
      if constexpr (kF16) odd = fmaf((x.x + x.y) + (x.z + x.w), 0.f, odd);
      const float l = sm.ml[1][h], s = whole ? (l != 0.f ? 1.f / l : 0.f) : 1.f;
      if (wide) {
        *reinterpret_cast<float4*>(out + 4 * i) = make_float4(x.x * s, x.y * s, x.z * s, x.w * s);
      } else {
        out[4 * i] = x.x * s, out[4 * i + 1] = x.y * s, out[4 * i + 2] = x.z * s, out[4 * i + 3] = x.w * s;
      }
    }
    // infinite values of V and NaN make the sum of their dim (times a weight's second part, of zero or below it, infinity was
    // NaN): those of the run's cells, added up, take its place
    if (kF16 && __any_sync(kFull, odd != 0.f)) {
#pragma unroll 1
      for (int i = tid; i < kGqa * kHeadDim / 4; i += kThreads) {
        const int h = i >> 6, d = (i & 63) * 4;   // (one head for a warp)
        if (!isfinite(sm.ml[1][h])) continue;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int v = run.first * kChunk; v < v_end; v += 32) {
          const int mine = checked_cell(a, cell_at(a, run, v + lane, slot_at(a, run, v + lane, v_end, false, err), false, err), false, err);
#pragma unroll 8
          for (int j = 0; j < 32; ++j) {
            const int c = __shfl_sync(kFull, mine, j);
            const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __half*>(a.v_cache) + ((int64_t)max(c, 0) * G + g) * kHeadDim + d);
            if (c >= 0) add_not_finite(y[0], y[1], w.x), add_not_finite(y[2], y[3], w.y);
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (y[j] != 0.f) out[4 * i + j] = y[j];
      }
    }
    if (tid < kGqa) {
      const float m = sm.ml[0][tid], l = sm.ml[1][tid];
      if (!whole) *reinterpret_cast<float2*>(a.of.ml + 2 * (ps + tid)) = make_float2(m, l);
      else if (a.weigh) a.lse[((int64_t)t0 * G + g) * kGqa + tid] = make_float2(m, l != 0.f ? 1.f / l : 0.f);
    }
    if (a.weigh && tid == 0 && g == 0 && run.first == 0) a.geo[t0] = make_int4(gr.ns_al, gr.lo_al, gr.nv, kChunk);
  }
}

constexpr int kMaxDevices = 64;

template <int KV, bool kMixed>
cudaError_t launch(const PagedArgs& a, unsigned* err, cudaStream_t stream) {
  static std::atomic<bool> known[kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!known[dev].load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(mu);
    e = cudaFuncSetAttribute(k_paged_one<KV, kMixed>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(Smem<KV, kMixed>));
    if (e != cudaSuccess) return e;
    known[dev].store(true, std::memory_order_release);
  }
  return launch_pdl(k_paged_one<KV, kMixed>, dim3((unsigned)(a.of.parts * a.n_kv_heads)), dim3(Row<KV>::kWarps * 32), sizeof(Smem<KV, kMixed>), stream, 1,
                    a, err);
}

template <int KV>
cudaError_t launch_kv(const PagedArgs& a, bool mixed, unsigned* err, cudaStream_t stream) {
  return mixed ? launch<KV, true>(a, err, stream) : launch<KV, false>(a, err, stream);
}

}  // namespace

cudaError_t launch_paged_one(const PagedArgs& a, int kv_type, bool mixed, unsigned* err, cudaStream_t stream) {
  return kv_type == QSA_KV_F16    ? launch_kv<QSA_KV_F16>(a, mixed, err, stream)
         : kv_type == QSA_KV_Q8_0 ? launch_kv<QSA_KV_Q8_0>(a, mixed, err, stream)
                                  : launch_kv<QSA_KV_Q4_0>(a, mixed, err, stream);
}

}  // namespace qsa
