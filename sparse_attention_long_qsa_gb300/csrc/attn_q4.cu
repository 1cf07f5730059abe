// Sparse attention over the selected cells of a q4_0 cache: one thread-block
// cluster per (token, KV head), as for the other cache types, but the codes
// never become an fp16 tile in shared memory.
//
//   out[h] = sum_c softmax_c(scale * q_h . K_c) V_c,   K_c[i] = d_K[c][i/32] (n_K[c][i] - 8)
//
// A row is 128 bytes of codes and 16 bytes of scales, a quarter of its fp16
// form.  Writing the expanded rows to shared memory for a tcgen05 operand and
// reading them back costs 1 KB + 1 KB of shared-memory traffic per cell and
// head (about 2,000 cycles per 128 cells on an SM), several times the gather
// itself, and the tensor core would use 8 of the 16 columns it needs at least.
// mma.sync takes its operands from registers: ldmatrix hands each thread
// exactly the nibbles of its fragment, and masking them in place makes fp16
// operands (0..15 in the low mantissa bits are the subnormals n * 2^-24, which
// the tensor cores multiply exactly).
//
// Both products are exact in their codes; no K or V value is ever rounded:
//   Q.K  per 32-value block with integer codes, the block's sum then scaled by
//        d_K in fp32; the code's offset of 8 enters as the accumulator's start
//        value -8 * sum_i q_i.  Codes in bits 4..7 of a half weigh 16 times
//        more: their queries are divided by 16.
//   P.V  d_V is folded into the probabilities: w = p * d_V, split into two
//        fp16 parts (22 bits), two products into one fp32 accumulator.  A
//        common power of two keeps w off the fp16 range's ends.
//
// Work split.  A warp takes 16 cells at a time: it copies their rows with
// cp.async into its own ring of stages (kStages - 1 chunks in flight), forms
// the scores of 8 heads x 16 cells, updates its running maximum (lazily: the
// accumulator is rescaled only when a score exceeds the maximum in use by
// 2^kLazy), and adds P.V.  Warps of a CTA and CTAs of a cluster share nothing
// until the end, when their (max, sum, o) are merged in a fixed order through
// shared and distributed shared memory.
#include <atomic>
#include <mutex>

#include "qsa_internal.cuh"
#include "tc_util.cuh"

namespace qsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kChunk = 16;                       // cells of one warp step
constexpr int kRow = 144;                        // 128 B codes + 16 B scales: ldmatrix rows 144 B apart do not conflict
constexpr int kStageBytes = 2 * kChunk * kRow;   // K rows, then V rows
constexpr int kStages = 4;
constexpr int kMaxCluster = 16;
constexpr float kLazy = 8.f;                     // log2 of how far a probability may exceed 1
constexpr int kNoExp = 32;                       // no scale of V seen yet
constexpr int kBlocks = kHeadDim / 32;           // q4_0 blocks of a row

template <int kWarps>
struct Smem {
  alignas(16) unsigned char stage[kWarps][kStages][kStageBytes];   // after the loop: each warp's o, fp32 [8][256]
  float m[kWarps][kGqa], l[kWarps][kGqa];
  int k[kWarps];                                 // exponent of the warp's weights
  float po[kMaxCluster * kGqa * (kHeadDim / kMaxCluster)];   // the cluster's partials of this CTA's dims
  float pm[kMaxCluster][2 * kGqa];               // their (max, sum)
  float w[kMaxCluster][kGqa];
};
static_assert(kStages * kStageBytes >= kGqa * kHeadDim * 4, "a warp's o fits in its stages");

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
__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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
// 2^k as a half, k in [-14, 15]
__device__ __forceinline__ __half2 pow2h(int k) {
  const uint32_t e = (uint32_t)(k + 15) << 10;
  return half2_of(e | (e << 16));
}

template <int kWarps>
__global__ void __launch_bounds__(kWarps * 32)
k_attn_q4(const AttnArgs a, unsigned* err) {
  extern __shared__ unsigned char smem_raw[];
  Smem<kWarps>& sm = *reinterpret_cast<Smem<kWarps>*>(smem_raw);
  constexpr int kThreads = kWarps * 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gid = lane >> 2, l4 = lane & 3;
  const int g = blockIdx.y, t = blockIdx.z;
  const uint32_t rank = cluster_rank(), NC = cluster_size();
  const int G = a.n_kv_heads, Hq = G * kGqa;
  // ---- the query fragments of head gid (an input: read before the wait).
  // Block b, step s: k index 2 l4 + {0, 1} is dim 32 b + 4 l4 + s + {0, 2},
  // k index 8 + 2 l4 + {0, 1} the dim 16 further (divided by 16).  A power of
  // two per head brings its largest query to [2^14, 2^15) first, so that small
  // queries keep their bits through that division.
  uint32_t qa[kBlocks][2][2];
  float qbias[kBlocks];
  float scale;   // of a score, to the log2 domain: without the queries' and the codes' powers of two
  {
    const __half* q = a.q + ((int64_t)t * Hq + g * kGqa + gid) * kHeadDim;
    __half2 qmax = __float2half2_rn(0.f);
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      const uint2 lo = *reinterpret_cast<const uint2*>(q + 32 * b + 4 * l4);
      const uint2 hi = *reinterpret_cast<const uint2*>(q + 32 * b + 16 + 4 * l4);
      qa[b][0][0] = __byte_perm(lo.x, lo.y, 0x5410);
      qa[b][1][0] = __byte_perm(lo.x, lo.y, 0x7632);
      qa[b][0][1] = __byte_perm(hi.x, hi.y, 0x5410);
      qa[b][1][1] = __byte_perm(hi.x, hi.y, 0x7632);
      qmax = __hmax2(qmax, __hmax2(__habs2(half2_of(lo.x)), __habs2(half2_of(lo.y))));
      qmax = __hmax2(qmax, __hmax2(__habs2(half2_of(hi.x)), __habs2(half2_of(hi.y))));
    }
    qmax = __hmax2(qmax, half2_of(__shfl_xor_sync(kFull, bits(qmax), 1)));
    qmax = __hmax2(qmax, half2_of(__shfl_xor_sync(kFull, bits(qmax), 2)));
    const int e = 29 - (int)((bits(__hmax2(qmax, __lowhigh2highlow(qmax))) & 0x7fffu) >> 10);   // -2 .. 29
    const int e0 = min(e, 15);
    const __half2 up0 = pow2h(e0), up1 = pow2h(e - e0), sixteenth = __float2half2_rn(0.0625f);
    scale = a.attn_scale * 1.4426950408889634f * exp2f((float)(24 - e));
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const __half2 x = __hmul2(__hmul2(half2_of(qa[b][i][j]), up0), up1);
          const float2 f = __half22float2(x);
          s += f.x + f.y;
          qa[b][i][j] = bits(j ? __hmul2(x, sixteenth) : x);
        }
      s += __shfl_xor_sync(kFull, s, 1);
      s += __shfl_xor_sync(kFull, s, 2);
      qbias[b] = s * (-8.0f / 16777216.0f);
    }
  }
  cluster_arrive();   // waited for before anything is pushed to a peer
  grid_dep_wait();
  grid_dep_launch();
  const int32_t* crow = a.cells + (int64_t)t * a.cells_pitch;
  int cnt = a.count[t];
  cnt = cnt < 0 ? 0 : (cnt > a.cells_pitch ? a.cells_pitch : cnt);
  const int n_chunks = (cnt + kChunk - 1) / kChunk;
  // chunks go round the cluster's CTAs first, so a short list uses all of them
  const int first = warp * (int)NC + (int)rank, step = kWarps * (int)NC;

  const unsigned char* kc = static_cast<const unsigned char*>(a.k_cache);
  const unsigned char* vc = static_cast<const unsigned char*>(a.v_cache);
  const int64_t codes = a.n_cells * (int64_t)G * (kHeadDim / 2);   // where the scales start
  const uint32_t ring = smem_u32(sm.stage[warp]);

  // the ids of a chunk: lanes i and i + 16 hold cell i (-1: none)
  auto cell_of = [&](int chunk) -> int {
    const int i = chunk * kChunk + (lane & 15);
    if (chunk >= n_chunks || i >= cnt) return -1;
    const int c = crow[i];
    if (c < 0 || c >= a.n_cells) {
      atomicOr(err, kErrCell);
      return -1;
    }
    return c;
  };
  // copies a chunk's rows into a stage; missing cells become zeros
  auto fetch = [&](int cell, int st) {
    const uint32_t dst = ring + (uint32_t)st * kStageBytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 4 * i + (lane >> 3);
      const int c = __shfl_sync(kFull, cell, row);
      const int64_t off = ((int64_t)(c < 0 ? 0 : c) * G + g) * (kHeadDim / 2) + (lane & 7) * 16;
      const uint32_t at = dst + row * kRow + (lane & 7) * 16;
      cp_async16(at, kc + off, c >= 0);
      cp_async16(at + kChunk * kRow, vc + off, c >= 0);
    }
    const int64_t off = codes + ((int64_t)(cell < 0 ? 0 : cell) * G + g) * (2 * kBlocks);
    cp_async16(dst + lane * kRow + 128, (lane < 16 ? kc : vc) + off, cell >= 0);
  };

  float acc[kBlocks][2][4];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[b][i][j] = 0.f;
  float run_m = -INFINITY, run_l = 0.f;   // head gid; run_l: this thread's cells only
  int wexp = kNoExp;                      // weights carry 2^wexp
  unsigned long long valid = 0;           // of the chunks in flight, oldest first: which of the 16 cells exist

  int ahead = cell_of(first);
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    const int chunk = first + s * step;
    if (chunk < n_chunks) {
      valid |= (unsigned long long)(__ballot_sync(kFull, ahead >= 0) & 0xffffu) << (16 * s);
      fetch(ahead, s);
    }
    asm volatile("cp.async.commit_group;\n" ::: "memory");
    ahead = cell_of(chunk + step);
  }

  int st = 0;
#pragma unroll 1
  for (int chunk = first; chunk < n_chunks; chunk += step) {
    asm volatile("cp.async.wait_group %0;\n" ::"n"(kStages - 2) : "memory");
    __syncwarp();   // every lane's copies of this stage are in; the stage fetched next has been read by all
    const unsigned ok = (unsigned)valid & 0xffffu;
    valid >>= 16;
    {
      const int nchunk = chunk + (kStages - 1) * step;
      if (nchunk < n_chunks) {
        valid |= (unsigned long long)(__ballot_sync(kFull, ahead >= 0) & 0xffffu) << (16 * (kStages - 2));
        fetch(ahead, st == 0 ? kStages - 1 : st - 1);
      }
      asm volatile("cp.async.commit_group;\n" ::: "memory");
      ahead = cell_of(nchunk + step);
    }
    const uint32_t sk = ring + (uint32_t)st * kStageBytes, sv = sk + kChunk * kRow;
    st = st == kStages - 1 ? 0 : st + 1;

    // ---- scores: s[j][e] = q_gid . K of cell 8 j + 2 l4 + e
    float s[2][2] = {};
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t dk[2][4];   // scales of the two cells, 8 halves each
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t at = sk + (8 * j + 2 * l4 + e) * kRow + 128;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(dk[e][0]), "=r"(dk[e][1]), "=r"(dk[e][2]), "=r"(dk[e][3])
                     : "r"(at)
                     : "memory");
      }
#pragma unroll
      for (int bq = 0; bq < 2; ++bq) {   // four blocks: lane l's address is row l % 8 of block 4 bq + l / 8
        uint32_t w[4];
        ldmatrix4(sk + (8 * j + (lane & 7)) * kRow + (4 * bq + (lane >> 3)) * 16, w);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int b = 4 * bq + i;
          float c[4] = {qbias[b], qbias[b], 0.f, 0.f};   // rows 8..15 (no head) are not used
          mma(c, qa[b][0][0], 0u, qa[b][0][1], 0u, w[i] & 0x000f000fu, w[i] & 0x00f000f0u);
          const uint32_t u = w[i] >> 8;
          mma(c, qa[b][1][0], 0u, qa[b][1][1], 0u, u & 0x000f000fu, u & 0x00f000f0u);
          const float2 d0 = __half22float2(half2_of(dk[0][b >> 1])), d1 = __half22float2(half2_of(dk[1][b >> 1]));
          s[j][0] = fmaf((b & 1) ? d0.y : d0.x, c[0], s[j][0]);
          s[j][1] = fmaf((b & 1) ? d1.y : d1.x, c[1], s[j][1]);
        }
      }
    }
    // ---- softmax of head gid over the 16 cells (a quad holds them)
    float p[2][2], cm = -INFINITY;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[j][e] = ((ok >> (8 * j + 2 * l4 + e)) & 1u) ? s[j][e] * scale : -INFINITY;
        cm = fmaxf(cm, s[j][e]);
      }
    cm = fmaxf(cm, __shfl_xor_sync(kFull, cm, 1));
    cm = fmaxf(cm, __shfl_xor_sync(kFull, cm, 2));
    // scales of V: their largest magnitude sets the weights' exponent
    uint32_t dv[2][2][4];
    __half2 dmax = __float2half2_rn(0.f);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t at = sv + (8 * j + 2 * l4 + e) * kRow + 128;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];\n"
                     : "=r"(dv[j][e][0]), "=r"(dv[j][e][1]), "=r"(dv[j][e][2]), "=r"(dv[j][e][3])
                     : "r"(at)
                     : "memory");
#pragma unroll
        for (int i = 0; i < 4; ++i) dmax = __hmax2(dmax, __habs2(half2_of(dv[j][e][i])));
      }
    dmax = __hmax2(dmax, half2_of(__shfl_xor_sync(kFull, bits(dmax), 1)));
    dmax = __hmax2(dmax, half2_of(__shfl_xor_sync(kFull, bits(dmax), 2)));
    const uint32_t db = bits(__hmax2(dmax, __lowhigh2highlow(dmax))) & 0x7fffu;
    // d_max * 2^want lies in [2^5, 2^6) (or below, at the exponent's ends)
    const int want = min(15, max(-10, 20 - (int)(db >> 10)));
    const bool grow = cm > run_m + kLazy;
    if (__any_sync(kFull, grow) || (db != 0u && want < wexp - 1)) {
      const int nexp = db != 0u && want < wexp - 1 ? want : wexp;
      const float nm = grow ? cm : run_m;
      const float f = run_m == -INFINITY ? 0.f : exp2f(run_m - nm);
      run_l *= f;
      run_m = nm;
      const float fe = wexp == kNoExp ? 1.f : exp2f((float)(nexp - wexp));   // accumulators of an unset exponent are zero
      wexp = nexp;
      const float f0 = __shfl_sync(kFull, f, 8 * l4) * fe, f1 = __shfl_sync(kFull, f, 8 * l4 + 4) * fe;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          acc[b][i][0] *= f0, acc[b][i][1] *= f1;
          acc[b][i][2] *= f0, acc[b][i][3] *= f1;
        }
    }
    __half2 ph[2], pl[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        p[j][e] = run_m == -INFINITY ? 0.f : exp2f(s[j][e] - run_m);
        run_l += p[j][e];
      }
      ph[j] = __floats2half2_rn(p[j][0], p[j][1]);
      const float2 h = __half22float2(ph[j]);
      pl[j] = __floats2half2_rn(p[j][0] - h.x, p[j][1] - h.y);
    }
    const __half2 up = pow2h(wexp == kNoExp ? 0 : wexp);

    // ---- o^T[dim][head] += V^T . w, per block of 32 dims: tile i, row gid is
    // dim 32 b + 2 gid + i, row gid + 8 the dim 16 further (16 times too large)
#pragma unroll
    for (int bp = 0; bp < 4; ++bp) {   // two blocks: lane l's address is row l % 16 of block 2 bp + l / 16
      uint32_t v[4];
      ldmatrix4_trans(sv + (lane & 15) * kRow + (2 * bp + (lane >> 4)) * 16, v);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int b = 2 * bp + i;
        uint32_t wh[2], wl[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const __half2 d = __hmul2(half2_of(__byte_perm(dv[j][0][b >> 1], dv[j][1][b >> 1], (b & 1) ? 0x7632 : 0x5410)), up);
          const __half2 h = __hmul2(ph[j], d);
          wh[j] = bits(h);
          wl[j] = bits(__hfma2(pl[j], d, __hfma2(ph[j], d, __hneg2(h))));
        }
        const __half2 c1 = half2_of(0x64086408u), c16 = half2_of(0x64806480u);   // 1024 + 8, 1024 + 128
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t x0 = k ? v[2 * i] >> 8 : v[2 * i], x1 = k ? v[2 * i + 1] >> 8 : v[2 * i + 1];
          const uint32_t a0 = bits(__hsub2(half2_of((x0 & 0x000f000fu) | 0x64006400u), c1));
          const uint32_t a1 = bits(__hsub2(half2_of((x0 & 0x00f000f0u) | 0x64006400u), c16));
          const uint32_t a2 = bits(__hsub2(half2_of((x1 & 0x000f000fu) | 0x64006400u), c1));
          const uint32_t a3 = bits(__hsub2(half2_of((x1 & 0x00f000f0u) | 0x64006400u), c16));
          mma(acc[b][k], a0, a1, a2, a3, wh[0], wh[1]);
          mma(acc[b][k], a0, a1, a2, a3, wl[0], wl[1]);
        }
      }
    }
  }
  asm volatile("cp.async.wait_all;\n" ::: "memory");

  // ---- merge the CTA's warps (in warp order)
  run_l += __shfl_xor_sync(kFull, run_l, 1);
  run_l += __shfl_xor_sync(kFull, run_l, 2);
  if (l4 == 0) {
    sm.m[warp][gid] = run_m;
    sm.l[warp][gid] = run_l;
  }
  __syncthreads();   // also: every warp is done with its stages
  float cta_m[2];    // of heads 2 l4, 2 l4 + 1
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    cta_m[e] = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) cta_m[e] = fmaxf(cta_m[e], sm.m[w][2 * l4 + e]);
  }
  {
    float* o = reinterpret_cast<float*>(sm.stage[warp]);   // [8][256]
    const float back = wexp == kNoExp ? 0.f : exp2f((float)-wexp);
    float f[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float mw = sm.m[warp][2 * l4 + e];
      f[e] = mw == -INFINITY ? 0.f : exp2f(mw - cta_m[e]) * back;
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          o[(2 * l4 + e) * kHeadDim + 32 * b + 2 * gid + i] = acc[b][i][e] * f[e];
          o[(2 * l4 + e) * kHeadDim + 32 * b + 2 * gid + i + 16] = acc[b][i][2 + e] * f[e] * 0.0625f;
        }
  }
  __syncthreads();
  cluster_wait();   // every CTA of the cluster runs
  // thread h < 8: the CTA's (max, sum) of head h to every CTA of the cluster
  if (tid < kGqa) {
    float m = -INFINITY, l = 0.f;
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sm.m[w][tid]);
    for (int w = 0; w < kWarps; ++w) l += sm.m[w][tid] == -INFINITY ? 0.f : sm.l[w][tid] * exp2f(sm.m[w][tid] - m);
    for (uint32_t r = 0; r < NC; ++r) {
      st_dsmem_f32(dsmem_addr(&sm.pm[rank][tid], r), m);
      st_dsmem_f32(dsmem_addr(&sm.pm[rank][kGqa + tid], r), l);
    }
  }
  // partial o: dims [r * 256 / NC, ...) go to CTA r
  const int dpc = kHeadDim / (int)NC;
  for (int i = tid; i < kGqa * kHeadDim; i += kThreads) {
    float o = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) o += reinterpret_cast<const float*>(sm.stage[w])[i];
    const int h = i >> 8, d = i & (kHeadDim - 1);
    st_dsmem_f32(dsmem_addr(&sm.po[((int)rank * kGqa + h) * dpc + d % dpc], (uint32_t)(d / dpc)), o);
  }
  cluster_sync();   // all pushes have landed; nobody touches a peer after this
  if (tid < kGqa) {
    float m = -INFINITY, l = 0.f;
    for (int r = 0; r < (int)NC; ++r) m = fmaxf(m, sm.pm[r][tid]);
    for (int r = 0; r < (int)NC; ++r) {
      const float w = sm.pm[r][tid] == -INFINITY ? 0.f : exp2f(sm.pm[r][tid] - m);
      sm.w[r][tid] = w;
      l += w * sm.pm[r][kGqa + tid];
    }
    for (int r = 0; r < (int)NC; ++r) sm.w[r][tid] = l != 0.f ? sm.w[r][tid] / l : 0.f;
  }
  __syncthreads();
  for (int i = tid; i < kGqa * dpc; i += kThreads) {
    const int h = i / dpc, e = i % dpc;
    float o = 0.f;
    for (int r = 0; r < (int)NC; ++r) o = fmaf(sm.w[r][h], sm.po[(r * kGqa + h) * dpc + e], o);
    a.out[((int64_t)t * Hq + g * kGqa + h) * kHeadDim + (int)rank * dpc + e] = o;
  }
}

constexpr int kMaxDevices = 64;

// Clusters of 16, 8, 4, 2, 1 CTAs of k_attn_q4<kWarps> that fit the current
// device at once, measured once per device under a lock.
template <int kWarps>
cudaError_t max_clusters(const int** out) {
  static int active[kMaxDevices][5];
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

}  // namespace

cudaError_t launch_attn_q4(const AttnArgs& a, unsigned* err, cudaStream_t stream) {
  constexpr int kWarps = 4;
  const int* active = nullptr;
  cudaError_t e = max_clusters<kWarps>(&active);
  if (e != cudaSuccess) return e;
  const int chunks = (int)ceil_div(a.cells_pitch, kChunk);
  const int64_t clusters = (int64_t)a.n_tokens * a.n_kv_heads;
  // the largest cluster whose warps all have a chunk and that runs in one
  // wave; past one wave at every size, single CTAs (no cluster to wait for)
  int nc = 1;
  for (int i = 0; i < 5; ++i) {
    const int c = 16 >> i;
    if (active[i] > 0 && clusters <= active[i] && (c == 1 || (c - 1) * kWarps < chunks)) {
      nc = c;
      break;
    }
  }
  return launch<kWarps>(a, nc, err, stream);
}

}  // namespace qsa
