// Sparse attention over the selected cells of a q4_0 cache: one thread-block
// cluster per (token, KV head), as for the other cache types, but the codes
// never become an fp16 tile in shared memory.
//
//   out[h] = sum_c softmax_c(scale * q_h . K_c) V_c,   K_c[i] = d_K[c][i/32] (n_K[c][i] - 8)
//
// A row is 128 bytes of codes and 16 bytes of scales, a quarter of its fp16
// form.  mma.sync takes its operands from registers: ldmatrix hands each thread
// exactly the nibbles of its fragment, and two instructions make two of them fp16
// operands.  (A code put under the exponent of 1024 is 1024 + code: published for
// int4 weights by Kim et al., "Who Says Elephants Can't Run", 2022.)  A tcgen05
// operand in shared memory would be written and read back expanded, 1 KB each a
// cell and head, some 2,000 cycles per 128 cells on an SM, where all of this
// kernel takes 2,550.  Codes stored to tensor memory as the A operand would not
// pay that; such a form is not built.
//
// Both products are exact in their codes; no K or V value is ever rounded:
//   Q.K  per 32-value block with integer codes, the block's sum then scaled by
//        d_K in fp32.  Codes in bits 4..7 of a half weigh 16 times more: their
//        queries are divided by 16.  (Masked codes without the offset of 8 are
//        subnormals, n * 2^-24, and would save the subtraction, but the tensor
//        core then drops low bits of the queries: scores off by 1e-6.)
//   P.V  d_V is folded into the probabilities: w = p * d_V, split into two
//        fp16 parts (22 bits), two products into fp32.  A half keeps its bits
//        only 30 binary places below the largest, so three forms, chosen by what
//        a chunk of 16 cells holds, keep what is lost small beside what the chunk
//        itself adds to a block of dims, however little that is beside other
//        chunks and other blocks:
//          near   the chunk's probabilities and scales lie close to the warp's
//                 largest: weights relative to those, summed in place (2^-18 of
//                 the chunk's part lost at most, with all 16 cells at the edges)
//          apart  weights relative to the chunk's own largest, summed in an
//                 accumulator of its own, which is added with the chunk's factor
//                 in fp32 (2^-22)
//          wild   scales of V in the chunk more than 2^10 apart, subnormal, zero
//                 for some of the cells only, or infinite: products in fp32, cell
//                 by cell
//        512 tokens at 250k cells take 147 us so (156 to 158 with scales or scores
//        that set most chunks apart, 606 with all of them wild), and 151 with the
//        apart form for every chunk that is not wild.  Weights relative to the
//        warp's largest throughout take 140, but one cell or block of large
//        values, however unlikely, then costs all others their bits (5e-4 of a
//        block's norm at a ratio of 3,000, a tenth of it at 1e6).
//
// Work split.  A warp takes 16 cells at a time: it copies their rows with
// cp.async into its own ring of stages (kStages - 1 chunks in flight), forms
// the scores of 8 heads x 16 cells and adds P.V relative to a reference score a
// head, which is raised, and the accumulator rescaled, when a chunk exceeds it.
// Warps of a CTA and CTAs of a cluster share nothing until the end, when their
// (reference, sum, o) are merged in a fixed order through shared and distributed
// shared memory.
#include <atomic>
#include <mutex>
#include <type_traits>

#include "qsa_internal.cuh"
#include "tc_util.cuh"

namespace qsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kChunk = 16;                       // cells of one warp step
constexpr int kRow = 144;                        // 128 B codes + 16 B scales: ldmatrix rows 144 B apart do not conflict
constexpr int kStageBytes = 2 * kChunk * kRow;   // K rows, then V rows
constexpr int kStages = 2;
constexpr int kMaxCluster = 16;
constexpr float kUp = 15.f;                      // probabilities are held as 2^(s - m + kUp), m a whole number, at least s
constexpr float kSlack = 2.f;                    // a raised reference lies so far above the chunk's largest score
constexpr float kNear = 7.f;                     // "near": the chunk's largest scores at most so far below the reference,
constexpr int kNearExp = 2;                      // its largest scale of V within 2^-kNearExp of the warp's,
constexpr unsigned kNearSpread = 5u << 10;       // its smallest (as bits) at most so far below its largest
constexpr unsigned kSpread = 10u << 10;          // the same for "apart"
constexpr int kNoExp = 64;                       // no scale of V seen yet
constexpr float kNoMax = -3.0e38f;               // no cell seen yet (below every score, and finite)
constexpr int kBlocks = kHeadDim / 32;           // q4_0 blocks of a row

constexpr int kPitch = kHeadDim + 4;             // floats between two heads of a warp's o: its stores do not conflict

template <int kWarps>
struct Smem {
  alignas(16) unsigned char stage[kWarps][kStages][kStageBytes];   // after the loop: each warp's o, fp32 [8][kPitch]
  uint4 q[kBlocks][32];                          // a lane's query fragments of a block: step 0, step 1
  float4 kd[kWarps][kBlocks][9];                 // a chunk's K scales: block, gid -> cells gid, gid + 8, each twice
                                                 // (blocks 144 B apart: their stores do not conflict)
  uint2 vd[kWarps][kBlocks][4];                  // its V scales times a power of two: block, l4 -> cells 2 l4 + {0, 1, 8, 9}
  float m[kWarps][kGqa], l[kWarps][kGqa];
  float cta[2 * kGqa];                           // the CTA's (max, sum)
  alignas(16) float po[kGqa * kHeadDim];         // the cluster's partials of this CTA's dims: [NC][8][256 / NC]
  alignas(16) float pm[kMaxCluster][2 * kGqa];   // their (max, sum)
  float w[kMaxCluster][kGqa];
};
static_assert(kStages * kStageBytes >= kGqa * kPitch * 4, "a warp's o fits in its stages");

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];\n"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix2_trans(uint32_t addr, uint32_t (&r)[2]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];\n"
               : "=r"(r[0]), "=r"(r[1])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same from zero.
__device__ __forceinline__ void mma0(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                     uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};\n"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
// An 8 x 8 tile of halves, two of a row per lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(y) : "r"(x));
  return y;
}
// 2^x; results below the normal range are zero
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
// (x & m) | o in one instruction
__device__ __forceinline__ uint32_t and_or(uint32_t x, uint32_t m, uint32_t o) {
  uint32_t r;
  asm("lop3.b32 %0, %1, %2, %3, 0xea;\n" : "=r"(r) : "r"(x), "r"(m), "r"(o));
  return r;
}
// (sx, sy) += (dx, dy) * (cx, cy)
__device__ __forceinline__ void fma2(float& sx, float& sy, float dx, float dy, float cx, float cy) {
  asm("{\n .reg .b64 s, d, c;\n mov.b64 s, {%0, %1};\n mov.b64 d, {%2, %3};\n mov.b64 c, {%4, %5};\n"
      " fma.rn.f32x2 s, d, c, s;\n mov.b64 {%0, %1}, s;\n}\n"
      : "+f"(sx), "+f"(sy)
      : "f"(dx), "f"(dy), "f"(cx), "f"(cy));
}
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
// Codes less 8 as halves: those in bits 0..3 of x's two halves, and 16 times
// those in bits 4..7.  A code put under the exponent of 1024 is 1024 + code (or
// + 16 codes); taking off 1024 + 8 (or + 128) is exact.
__device__ __forceinline__ uint32_t low_codes(uint32_t x) {
  return bits(__hsub2(half2_of(and_or(x, 0x000f000fu, 0x64006400u)), half2_of(0x64086408u)));
}
__device__ __forceinline__ uint32_t high_codes(uint32_t x) {
  return bits(__hsub2(half2_of(and_or(x, 0x00f000f0u, 0x64006400u)), half2_of(0x64806480u)));
}
// x, infinities as NaN
__device__ __forceinline__ __half2 nan_of_inf(__half2 x) { return __hfma2(x, half2_of(0u), x); }
// 2^k as a half, k in [-24, 15]
__device__ __forceinline__ __half2 pow2h(int k) {
  const uint32_t e = k >= -14 ? (uint32_t)(k + 15) << 10 : 1u << (k + 24);
  return half2_of(e | (e << 16));
}

template <int kWarps>
__global__ void __launch_bounds__(kWarps * 32, kWarps == 4 ? 4 : 1)
k_attn_q4(const AttnArgs a, unsigned* err) {
  extern __shared__ unsigned char smem_raw[];
  Smem<kWarps>& sm = *reinterpret_cast<Smem<kWarps>*>(smem_raw);
  constexpr int kThreads = kWarps * 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, l4 = lane & 3;
  const int g = blockIdx.y, t = blockIdx.z;
  const uint32_t rank = cluster_rank(), NC = cluster_size();
  const int G = a.n_kv_heads, Hq = G * kGqa;

  // ---- the query fragments, column gid = head gid (an input: read before the
  // wait).  Block b, step s: k index 2 l4 + {0, 1} is dim 32 b + 4 l4 + s + {0, 2},
  // k index 8 + 2 l4 + {0, 1} the dim 16 further (divided by 16).  A power of
  // two per head brings its largest query to [2^14, 2^15) first, so that the
  // others keep their bits through that division down to 2^-24 of it.
  float scale[2];   // of heads 2 l4, 2 l4 + 1's scores, to the log2 domain: without the queries' power of two
  {
    const __half* q = a.q + ((int64_t)t * Hq + g * kGqa + gid) * kHeadDim;
    uint32_t x[kBlocks][2][2];
    __half2 qmax = __float2half2_rn(0.f);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const uint2 lo = *reinterpret_cast<const uint2*>(q + 32 * b + 4 * l4);
      const uint2 hi = *reinterpret_cast<const uint2*>(q + 32 * b + 16 + 4 * l4);
      x[b][0][0] = __byte_perm(lo.x, lo.y, 0x5410);
      x[b][1][0] = __byte_perm(lo.x, lo.y, 0x7632);
      x[b][0][1] = __byte_perm(hi.x, hi.y, 0x5410);
      x[b][1][1] = __byte_perm(hi.x, hi.y, 0x7632);
      qmax = __hmax2(qmax, __hmax2(__habs2(half2_of(lo.x)), __habs2(half2_of(lo.y))));
      qmax = __hmax2(qmax, __hmax2(__habs2(half2_of(hi.x)), __habs2(half2_of(hi.y))));
    }
    qmax = __hmax2(qmax, half2_of(__shfl_xor_sync(kFull, bits(qmax), 1)));
    qmax = __hmax2(qmax, half2_of(__shfl_xor_sync(kFull, bits(qmax), 2)));
    const int e = 29 - (int)((bits(__hmax2(qmax, __lowhigh2highlow(qmax))) & 0x7fffu) >> 10);   // -2 .. 29
    const int e0 = min(e, 15);
    const __half2 up0 = pow2h(e0), up1 = pow2h(e - e0), sixteenth = __float2half2_rn(0.0625f);
    const float mine = a.attn_scale * 1.4426950408889634f * exp2f((float)-e);
    scale[0] = __shfl_sync(kFull, mine, 8 * l4);
    scale[1] = __shfl_sync(kFull, mine, 8 * l4 + 4);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const __half2 y = __hmul2(__hmul2(half2_of(x[b][i][j]), up0), up1);
          x[b][i][j] = bits(j ? __hmul2(y, sixteenth) : y);
        }
      if (b % kWarps == warp) sm.q[b][lane] = make_uint4(x[b][0][0], x[b][0][1], x[b][1][0], x[b][1][1]);
    }
  }
  cluster_arrive();   // waited for before anything is pushed to a peer
  grid_dep_wait();
  grid_dep_launch();
  const int32_t* crow = a.cells + (int64_t)t * a.cells_pitch;
  // chunks go round the cluster's CTAs first, so a short list uses all of them
  const int first = warp * (int)NC + (int)rank, step = kWarps * (int)NC;
  // the first chunk's ids and the count load together
  const int i_first = first * kChunk + (lane & 15);
  const int id_first = i_first < a.cells_pitch ? crow[i_first] : 0;
  int cnt = a.count[t];
  cnt = cnt < 0 ? 0 : (cnt > a.cells_pitch ? a.cells_pitch : cnt);
  const int n_chunks = (cnt + kChunk - 1) / kChunk;

  const uint32_t ring = smem_u32(sm.stage[warp]);
  const unsigned char* kc = static_cast<const unsigned char*>(a.k_cache);
  const unsigned char* vc = static_cast<const unsigned char*>(a.v_cache);
  const uint32_t pitch = (uint32_t)G * (kHeadDim / 2);                          // code bytes of a cell
  // Eight lanes copy a row's codes: a copy of whole 128-byte lines costs the
  // load unit a quarter of one that touches 16 lines in part.
  const unsigned char* kcodes = kc + g * (kHeadDim / 2) + (lane & 7) * 16;
  const unsigned char* vcodes = vc + g * (kHeadDim / 2) + (lane & 7) * 16;
  const unsigned char* scales = (lane < 16 ? kc : vc) + a.n_cells * (int64_t)pitch + g * (2 * kBlocks);

  // the ids of a chunk as listed, lanes i and i + 16 holding cell i (past the
  // list: kPast); looked at only a step later, so that nothing waits on the load
  constexpr int kPast = (int)0x80000000u;
  auto listed = [&](int chunk) -> int {
    const int i = chunk * kChunk + (lane & 15);
    return i < cnt ? crow[i] : kPast;
  };
  auto checked = [&](int c) -> int {
    if ((unsigned)c < (unsigned)a.n_cells) return c;
    if (c != kPast) atomicOr(err, kErrCell);
    return -1;
  };
  // copies a chunk's rows into a stage; missing cells become zeros
  auto fetch = [&](int cell, unsigned ok, int st) {
    const uint32_t dst = ring + (uint32_t)st * kStageBytes;
    const uint32_t at = dst + (lane >> 3) * kRow + (lane & 7) * 16;
    const uint32_t id = (uint32_t)max(cell, 0);
    cp_async16(dst + lane * kRow + 128, scales + (uint64_t)id * (pitch >> 3), cell >= 0);
    if (ok == kFull) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t off = (uint64_t)__shfl_sync(kFull, id, 4 * i + (lane >> 3)) * pitch;
        cp_async16(at + 4 * i * kRow, kcodes + off, true);
        cp_async16(at + (4 * i + kChunk) * kRow, vcodes + off, true);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t off = (uint64_t)__shfl_sync(kFull, id, 4 * i + (lane >> 3)) * pitch;
        const bool have = (ok >> (4 * i + (lane >> 3))) & 1u;
        cp_async16(at + 4 * i * kRow, kcodes + off, have);
        cp_async16(at + (4 * i + kChunk) * kRow, vcodes + off, have);
      }
    }
  };

  float acc[kBlocks][2][4];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[b][i][j] = 0.f;
  // of heads 2 l4, 2 l4 + 1; run_m: the reference (a whole number), run_l: this thread's cells only;
  // acc and run_l carry 2^kUp, acc 2^wexp too
  float run_m[2] = {kNoMax, kNoMax}, run_l[2] = {0.f, 0.f};
  int wexp = kNoExp;
  unsigned valid[kStages - 1] = {};       // of the chunks in flight, oldest first: which of the 16 cells exist

  int ahead = i_first < cnt ? id_first : kPast;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    const int chunk = first + s * step;
    if (chunk < n_chunks) {
      const int cell = checked(ahead);
      valid[s] = __ballot_sync(kFull, cell >= 0);
      fetch(cell, valid[s], s);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
    ahead = listed(chunk + step);
  }
  __syncthreads();   // the query fragments are in place

  int st = 0;
#pragma unroll 1
  for (int chunk = first; chunk < n_chunks; chunk += step) {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 2) : "memory");
    __syncwarp();   // every lane's copies of this stage are in; the stage fetched next has been read by all
    const unsigned ok = valid[0];   // bits i and i + 16: cell i
#pragma unroll
    for (int i = 0; i + 1 < kStages - 1; ++i) valid[i] = valid[i + 1];
    {
      const int nchunk = chunk + (kStages - 1) * step;
      if (nchunk < n_chunks) {
        const int cell = checked(ahead);
        valid[kStages - 2] = __ballot_sync(kFull, cell >= 0);
        fetch(cell, valid[kStages - 2], st == 0 ? kStages - 1 : st - 1);
      }
      asm volatile("cp.async.commit_group;\n" ::: "memory");
      ahead = listed(nchunk + step);
    }
    const uint32_t sk = ring + (uint32_t)st * kStageBytes, sv = sk + kChunk * kRow;
    st = st == kStages - 1 ? 0 : st + 1;
    if (ok == 0u) continue;   // none of the chunk's cells exists

    // ---- the chunk's scales, laid out once for all lanes.  The transposing
    // ldmatrix gives this thread those of cells 2 l4 + {0, 1, 8, 9} in block gid.
    __half2 dv[2];
    {
      uint32_t d[2];
      ldmatrix2_trans(sk + (lane & 15) * kRow + 128, d);
      // an infinite scale of K becomes NaN (a block of such values holds infinities of both signs and NaN):
      // times a block's sum it would be an infinity of either sign, and -inf a cell of probability zero
      const float2 d0 = __half22float2(nan_of_inf(half2_of(d[0]))), d1 = __half22float2(nan_of_inf(half2_of(d[1])));
      sm.kd[warp][gid][2 * l4] = make_float4(d0.x, d0.x, d1.x, d1.x);
      sm.kd[warp][gid][2 * l4 + 1] = make_float4(d0.y, d0.y, d1.y, d1.y);
      ldmatrix2_trans(sv + (lane & 15) * kRow + 128, d);
      dv[0] = half2_of(d[0]), dv[1] = half2_of(d[1]);
    }
    // the chunk's largest and smallest scale of V, and the exponent of its weights
    const uint32_t dx = bits(__hmax2(__habs2(dv[0]), __habs2(dv[1])));
    uint32_t dn = bits(__hmin2(__habs2(dv[0]), __habs2(dv[1])));
    if (ok != kFull) {   // the cells that exist
      const uint32_t a0 = bits(__habs2(dv[0])), a1 = bits(__habs2(dv[1])), o = ok >> (2 * l4);
      const uint32_t e0 = (o & 1u) ? a0 & 0xffffu : 0xffffu, e1 = (o & 2u) ? a0 >> 16 : 0xffffu;
      const uint32_t e2 = (o & 256u) ? a1 & 0xffffu : 0xffffu, e3 = (o & 512u) ? a1 >> 16 : 0xffffu;
      const uint32_t e = min(min(e0, e1), min(e2, e3));
      dn = e | (e << 16);
    }
    const uint32_t dtop = __reduce_max_sync(kFull, max(dx >> 16, dx & 0xffffu));
    uint32_t dbot = __reduce_min_sync(kFull, min(dn >> 16, dn & 0xffffu));
    if (dbot == 0u) {   // a block that is zero in all of the chunk's cells (dims of padding) takes nothing from the others
      const bool zeros = ((__ballot_sync(kFull, dx == 0u) >> (lane & 28)) & 15u) == 15u;
      dbot = __reduce_min_sync(kFull, zeros ? 0x7bffu : min(dn >> 16, dn & 0xffffu));
    }
    const bool plain = dbot >= 0x0400u && dtop < 0x7c00u && dtop <= dbot + kSpread;
    int vexp = plain ? 13 - (int)(dtop >> 10) : 0;   // brings the chunk's largest scale to [2^-2, 2^-1)
    const int nexp = min(wexp, vexp);                // the warp's
    bool near = plain && vexp <= nexp + kNearExp && dtop <= dbot + kNearSpread;
    if (near) vexp = nexp;
    const __half2 up = pow2h(vexp);
    sm.vd[warp][gid][l4] = make_uint2(bits(__hmul2(dv[0], up)), bits(__hmul2(dv[1], up)));
    __syncwarp();

    // ---- scores: s[j] of cell gid + 8 j with heads 2 l4, 2 l4 + 1
    float2 s[2] = {};
#pragma unroll
    for (int bp = 0; bp < 4; ++bp) {   // two blocks: lane l's address is row l % 16 of block 2 bp + l / 16
      uint32_t w[4];
      ldmatrix4(sk + (lane & 15) * kRow + (2 * bp + (lane >> 4)) * 16, w);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int b = 2 * bp + i;
        const uint4 q = sm.q[b][lane];
        const float4 d = sm.kd[warp][b][gid];
        const uint32_t w0 = w[2 * i], w1 = w[2 * i + 1], u0 = w0 >> 8, u1 = w1 >> 8;
        float c[4];
        mma0(c, low_codes(w0), low_codes(w1), high_codes(w0), high_codes(w1), q.x, q.y);
        mma(c, low_codes(u0), low_codes(u1), high_codes(u0), high_codes(u1), q.z, q.w);
        fma2(s[0].x, s[0].y, d.x, d.y, c[0], c[1]);
        fma2(s[1].x, s[1].y, d.z, d.w, c[2], c[3]);
      }
    }
    // ---- softmax of the two heads over the 16 cells (8 lanes hold them)
    float cm[2] = {fmaxf(s[0].x * scale[0], s[1].x * scale[0]), fmaxf(s[0].y * scale[1], s[1].y * scale[1])};
    if (ok != kFull) {   // missing cells: p = 0
      const bool h0 = (ok >> gid) & 1u, h1 = (ok >> (gid + 8)) & 1u;
      cm[0] = fmaxf(h0 ? s[0].x * scale[0] : -INFINITY, h1 ? s[1].x * scale[0] : -INFINITY);
      cm[1] = fmaxf(h0 ? s[0].y * scale[1] : -INFINITY, h1 ? s[1].y * scale[1] : -INFINITY);
    }
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1)
#pragma unroll
      for (int h = 0; h < 2; ++h) cm[h] = fmaxf(cm[h], __shfl_xor_sync(kFull, cm[h], o));
    // m: the next whole numbers, so that the factors between chunks are powers of two (no finite score: far below all)
    const float m[2] = {fmaxf(ceilf(cm[0]), kNoMax), fmaxf(ceilf(cm[1]), kNoMax)};
    if (__any_sync(kFull, m[0] > run_m[0] || m[1] > run_m[1]) || nexp != wexp) {
      float f[2];
      const float fe = wexp == kNoExp ? 1.f : exp2f((float)(nexp - wexp));   // accumulators of an unset exponent are zero
      wexp = nexp;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float nm = m[h] > run_m[h] ? m[h] + kSlack : run_m[h];
        f[h] = exp2f(run_m[h] - nm);
        run_l[h] *= f[h];
        run_m[h] = nm;
        f[h] *= fe;
      }
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc[b][i][0] *= f[0], acc[b][i][1] *= f[1];
          acc[b][i][2] *= f[0], acc[b][i][3] *= f[1];
        }
    }
    near = near && !__any_sync(kFull, m[0] < run_m[0] - kNear || m[1] < run_m[1] - kNear);
    const float m0 = near ? run_m[0] : m[0], m1 = near ? run_m[1] : m[1];
    float p[2][2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      p[j][0] = ex2(fmaf(s[j].x, scale[0], kUp - m0));
      p[j][1] = ex2(fmaf(s[j].y, scale[1], kUp - m1));
      if (ok != kFull && !((ok >> (gid + 8 * j)) & 1u)) p[j][0] = p[j][1] = 0.f;
    }
    float fac[2] = {1.f, 1.f};   // of the chunk
    if (!near) fac[0] = ex2(m0 - run_m[0]), fac[1] = ex2(m1 - run_m[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) run_l[h] = fmaf(p[0][h] + p[1][h], fac[h], run_l[h]);

    if (!plain) {
      // ---- the same cell by cell in fp32: this thread's dims 32 b + 2 gid + {0, 1} and the two 16 further
      // (kept 16 times too large, as below)
      const float up1 = exp2f((float)wexp);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const unsigned char* row = sm.stage[warp][st == 0 ? kStages - 1 : st - 1] + (kChunk + 8 * j + i) * kRow;
          const float w0 = __shfl_sync(kFull, p[j][0], 4 * i + l4) * (fac[0] * up1);
          const float w1 = __shfl_sync(kFull, p[j][1], 4 * i + l4) * (fac[1] * up1);
          const uint4 dr = *reinterpret_cast<const uint4*>(row + 128);
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) {
            const __half2 dh = nan_of_inf(half2_of(b < 2 ? dr.x : b < 4 ? dr.y : b < 6 ? dr.z : dr.w));
            const float d = b & 1 ? __high2float(dh) : __low2float(dh), d0 = w0 * d, d1 = w1 * d;
            const uint32_t c = *reinterpret_cast<const unsigned short*>(row + 16 * b + 2 * gid);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float lo = (float)((int)((c >> (8 * k)) & 15u) - 8), hi = 16.f * (float)((int)((c >> (8 * k + 4)) & 15u) - 8);
              acc[b][k][0] = fmaf(d0, lo, acc[b][k][0]), acc[b][k][1] = fmaf(d1, lo, acc[b][k][1]);
              acc[b][k][2] = fmaf(d0, hi, acc[b][k][2]), acc[b][k][3] = fmaf(d1, hi, acc[b][k][3]);
            }
          }
        }
      continue;
    }

    // the probabilities in two parts, from (cell, heads) to (head, cells)
    __half2 ph[2], pl[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const __half2 hi = __floats2half2_rn(p[j][0], p[j][1]);
      const float2 h = __half22float2(hi);
      ph[j] = half2_of(transposed(bits(hi)));
      pl[j] = half2_of(transposed(bits(__floats2half2_rn(p[j][0] - h.x, p[j][1] - h.y))));
    }

    // ---- o^T[dim][head] += V^T . w, per block of 32 dims: tile i, row gid is
    // dim 32 b + 2 gid + i, row gid + 8 the dim 16 further (16 times too large)
    auto add = [&](auto in_place) {
#pragma unroll
      for (int bp = 0; bp < 4; ++bp) {   // two blocks: lane l's address is row l % 16 of block 2 bp + l / 16
        uint32_t v[4];
        ldmatrix4_trans(sv + (lane & 15) * kRow + (2 * bp + (lane >> 4)) * 16, v);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int b = 2 * bp + i;
          const uint2 d = sm.vd[warp][b][l4];
          const __half2 d0 = half2_of(d.x), d1 = half2_of(d.y);
          const __half2 h0 = __hmul2(ph[0], d0), h1 = __hmul2(ph[1], d1);
          const uint32_t wh0 = bits(h0), wh1 = bits(h1);
          const uint32_t wl0 = bits(__hfma2(pl[0], d0, __hfma2(ph[0], d0, __hneg2(h0))));
          const uint32_t wl1 = bits(__hfma2(pl[1], d1, __hfma2(ph[1], d1, __hneg2(h1))));
          uint32_t x[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t x0 = k ? v[2 * i] >> 8 : v[2 * i], x1 = k ? v[2 * i + 1] >> 8 : v[2 * i + 1];
            x[k][0] = low_codes(x0);
            x[k][1] = high_codes(x0);
            x[k][2] = low_codes(x1);
            x[k][3] = high_codes(x1);
          }
          if constexpr (decltype(in_place)::value) {
#pragma unroll
            for (int k = 0; k < 2; ++k) mma(acc[b][k], x[k][0], x[k][1], x[k][2], x[k][3], wh0, wh1);
#pragma unroll
            for (int k = 0; k < 2; ++k) mma(acc[b][k], x[k][0], x[k][1], x[k][2], x[k][3], wl0, wl1);
          } else {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float c[4];
              mma0(c, x[k][0], x[k][1], x[k][2], x[k][3], wh0, wh1);
              mma(c, x[k][0], x[k][1], x[k][2], x[k][3], wl0, wl1);
              fma2(acc[b][k][0], acc[b][k][1], fac[0], fac[1], c[0], c[1]);
              fma2(acc[b][k][2], acc[b][k][3], fac[0], fac[1], c[2], c[3]);
            }
          }
        }
      }
    };
    if (near) {
      add(std::true_type{});
    } else {
      const float back = exp2f((float)(wexp - vexp));
      fac[0] *= back, fac[1] *= back;
      add(std::false_type{});
    }
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");

  // ---- merge the CTA's warps (in warp order)
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
    float* o = reinterpret_cast<float*>(sm.stage[warp]);   // [8][kPitch]
    const float back = wexp == kNoExp ? 0.f : exp2f((float)-wexp);
    float f[2];   // of heads 2 l4, 2 l4 + 1
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float m = kNoMax;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][2 * l4 + e]);
      f[e] = exp2f(sm.m[warp][2 * l4 + e] - m) * back;
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float* p = o + (2 * l4 + e) * kPitch + 32 * b + 2 * gid;
        *reinterpret_cast<float2*>(p) = make_float2(acc[b][0][e] * f[e], acc[b][1][e] * f[e]);
        *reinterpret_cast<float2*>(p + 16) =
            make_float2(acc[b][0][2 + e] * (f[e] * 0.0625f), acc[b][1][2 + e] * (f[e] * 0.0625f));
      }
  }
  // the CTA's (max, sum) of each head: four lanes of warp 0 a head
  if (warp == 0) {
    float m = kNoMax, l = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][gid]);
#pragma unroll
    for (int w = 0; w < kWarps; w += 4)
      if (w + l4 < kWarps) l += sm.l[w + l4][gid] * exp2f(sm.m[w + l4][gid] - m);
    l += __shfl_xor_sync(kFull, l, 1);
    l += __shfl_xor_sync(kFull, l, 2);
    if (l4 == 0) {
      sm.cta[gid] = m;
      sm.cta[kGqa + gid] = l;
    }
  }
  __syncthreads();
  // four dims of a head, summed over the warps
  auto sum4 = [&](int i) -> float4 {
    const int h = i >> 6, d = (i & 63) * 4;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(sm.stage[w]) + h * kPitch + d);
      o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
    }
    return o;
  };
  float* out = a.out + ((int64_t)t * Hq + g * kGqa) * kHeadDim;
  if (NC == 1) {
    const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0u;   // the call takes any float address
    for (int i = tid; i < kGqa * kHeadDim / 4; i += kThreads) {
      const float4 o = sum4(i);
      const float l = sm.cta[kGqa + (i >> 6)], w = l != 0.f ? 1.0f / l : 0.f;
      const float4 y = make_float4(o.x * w, o.y * w, o.z * w, o.w * w);
      if (wide) {
        reinterpret_cast<float4*>(out)[i] = y;
      } else {
        out[4 * i] = y.x, out[4 * i + 1] = y.y, out[4 * i + 2] = y.z, out[4 * i + 3] = y.w;
      }
    }
    cluster_wait();
    return;
  }
  cluster_wait();   // every CTA of the cluster runs
  for (int i = tid; i < 2 * kGqa * (int)NC; i += kThreads)
    st_dsmem_f32(dsmem_addr(&sm.pm[rank][i % (2 * kGqa)], (uint32_t)(i / (2 * kGqa))), sm.cta[i % (2 * kGqa)]);
  // partial o: dims [r * 256 / NC, ...) go to CTA r
  const int dpc = kHeadDim / (int)NC;
  for (int i = tid; i < kGqa * kHeadDim / 4; i += kThreads) {
    const float4 o = sum4(i);
    const int h = i >> 6, d = (i & 63) * 4;
    st_dsmem_f32x4(dsmem_addr(&sm.po[((int)rank * kGqa + h) * dpc + d % dpc], (uint32_t)(d / dpc)), o);
  }
  cluster_sync();   // all pushes have landed; nobody touches a peer after this
  if (tid < kMaxCluster * kGqa) {   // the partials' weights, a head's in 16 neighbouring lanes
    const int h = tid >> 4, r = tid & 15;
    const float m = r < (int)NC ? sm.pm[r][h] : kNoMax, l = r < (int)NC ? sm.pm[r][kGqa + h] : 0.f;
    float top = m;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    const float w = exp2f(m - top);
    float sum = w * l;
#pragma unroll
    for (int o = 8; o >= 1; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
    sm.w[r][h] = sum != 0.f ? w / sum : 0.f;
  }
  __syncthreads();
  for (int i = tid; i < kGqa * dpc; i += kThreads) {
    const int h = i / dpc, e = i % dpc;
    float o = 0.f;
    for (int r = 0; r < (int)NC; ++r) o = fmaf(sm.w[r][h], sm.po[(r * kGqa + h) * dpc + e], o);
    out[h * kHeadDim + (int)rank * dpc + e] = o;
  }
}

constexpr int kMaxDevices = 64;

// Clusters of 16, 8, 4, 2, 1 CTAs of k_attn_q4<kWarps> that fit the current
// device at once, then its SMs, measured once per device under a lock.
template <int kWarps>
cudaError_t max_clusters(const int** out) {
  static int active[kMaxDevices][6];
  static std::atomic<bool> configured[kMaxDevices];
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  if (!configured[dev].load(std::memory_order_acquire)) {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev].load(std::memory_order_relaxed)) {
      constexpr int kSmem = (int)sizeof(Smem<kWarps>);
      e = cudaFuncSetAttribute(k_attn_q4<kWarps>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
      if (e != cudaSuccess) return e;
      e = cudaFuncSetAttribute(k_attn_q4<kWarps>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      for (int i = 0; i < 5; ++i) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(16u >> i, 1, 1);
        cfg.blockDim = dim3(kWarps * 32, 1, 1);
        cfg.dynamicSmemBytes = (size_t)kSmem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 16u >> i;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int n = 0;
        if (cudaOccupancyMaxActiveClusters(&n, k_attn_q4<kWarps>, &cfg) != cudaSuccess) {
          (void)cudaGetLastError();
          n = 0;
        }
        active[dev][i] = n;
      }
      e = cudaDeviceGetAttribute(&active[dev][5], cudaDevAttrMultiProcessorCount, dev);
      if (e != cudaSuccess) return e;
      configured[dev].store(true, std::memory_order_release);
    }
  }
  *out = active[dev];
  return cudaSuccess;
}

template <int kWarps>
cudaError_t launch(const AttnArgs& a, int nc, unsigned* err, cudaStream_t stream) {
  return launch_pdl(k_attn_q4<kWarps>, dim3((unsigned)nc, (unsigned)a.n_kv_heads, (unsigned)a.n_tokens),
                    dim3(kWarps * 32), sizeof(Smem<kWarps>), stream, (unsigned)nc, a, err);
}

// Cluster size for kWarps warps a CTA, and the time the call then takes by this
// reckoning, in units of 0.05 us.  Fitted to every size and both warp counts at 1
// to 512 tokens (250k cells, 129 chunks): 4.5 us for launch, prologue and merge,
// and for each chunk that a warp takes 0.9 us with 4 warps on the SM, 1.3 with 8
// and 2.3 with 16 (where the SM's throughput decides).  16 tokens: 17 us with as
// many warps as fit, 12 us with half of them and twice the chunks.
template <int kWarps>
cudaError_t plan(int64_t clusters, int chunks, int* nc, int64_t* cost) {
  const int* active = nullptr;
  const cudaError_t e = max_clusters<kWarps>(&active);
  if (e != cudaSuccess) return e;
  *nc = 1;
  *cost = -1;
  const int64_t sms = active[5], slots = active[4] > sms ? active[4] / sms : 1;   // CTAs that share an SM
  for (int i = 0; i < 5; ++i) {
    const int c = 16 >> i;
    if (active[i] <= 0 || c > (chunks > 1 ? chunks : 1)) continue;   // every CTA has a chunk
    const int64_t per_sm = ceil_div(clusters * c, sms), steps = ceil_div((int64_t)chunks, (int64_t)c * kWarps);
    auto chunk = [](int64_t ctas) -> int64_t {   // with so many CTAs on the SM
      const int64_t t = 5 * ctas * kWarps / 2 + 6;
      return t > 18 ? t : 18;
    };
    // past what fits: single CTAs follow one another on an SM, clusters come in waves
    int64_t w;
    if (clusters <= active[i]) w = 90 + steps * chunk(per_sm < slots ? per_sm : slots);
    else if (c > 1) w = ceil_div(clusters, (int64_t)active[i]) * (90 + steps * chunk(slots));
    else w = 90 * ceil_div(per_sm, slots) + steps * (per_sm / slots * chunk(slots) + (per_sm % slots ? chunk(per_sm % slots) : 0));
    if (*cost < 0 || w <= *cost) {   // the smaller of two equals
      *cost = w;
      *nc = c;
    }
  }
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_attn_q4(const AttnArgs& a, unsigned* err, cudaStream_t stream) {
  const int chunks = (int)ceil_div(a.cells_pitch, kChunk);
  const int64_t clusters = (int64_t)a.n_tokens * a.n_kv_heads;
  int nc4 = 1, nc9 = 1;
  int64_t cost4 = 0, cost9 = 0;
  cudaError_t e = plan<4>(clusters, chunks, &nc4, &cost4);
  if (e == cudaSuccess) e = plan<9>(clusters, chunks, &nc9, &cost9);
  if (e != cudaSuccess) return e;
  if (cost9 < cost4) return launch<9>(a, nc9, err, stream);
  return launch<4>(a, nc4, err, stream);
}

}  // namespace qsa
