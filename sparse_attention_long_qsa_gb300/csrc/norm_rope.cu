// Head norms of a step's queries, keys and indexer queries with their position
// rotation in the same pass: the rows that the append and the attention take
// "already positioned".
//
// Per head row x of n dims (n = 256, or 128 for the indexer):
//   y = x / sqrt(mean(x^2) + rms_eps) * w
// and then, over the first 2m dims, the half-split pairs (y_i, y_{i+m}), i < m,
// turn by pos[axis(i)] * theta^(-i/m).  The other dims pass through.  Sums,
// norms and rotations are fp32; q and k are rounded once, to the fp16 that the
// cache and the attention hold; the indexer query stays fp32, as the block
// scores take it.
//
// Angles reach 1e6 rad, where an fp32 product would be off by 6e-2 rad, so
// they are reduced exactly in integers (sincos_turn, pool_row.cuh).
//
// One CTA per token: its threads first compute the token's cosines and sines
// (shared by all heads) into shared memory while the first rows load, then a
// warp takes one head row at a time: one 16-byte load per lane for 16-bit
// inputs, a shuffle sum, the partner dims by shuffles, one 16-byte store.
#include <cuda_bf16.h>

#include "pool_row.cuh"

namespace qsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kNrThreads = 256;
constexpr int kNrWarps = kNrThreads / 32;

// The first 8 (kN = 8) or 4 elements of type E at p, 16-byte (8-byte) aligned.
template <int kE, int kN>
__device__ __forceinline__ void load_row(const void* p, float (&x)[8]) {
  if constexpr (kE == QSA_ELEM_F32) {
#pragma unroll
    for (int i = 0; i < kN / 4; ++i) {
      const float4 v = reinterpret_cast<const float4*>(p)[i];
      x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
    }
  } else {
    uint32_t w[4] = {};
    if constexpr (kN == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < kN / 2; ++i) {
      float2 f;
      if constexpr (kE == QSA_ELEM_F16) {
        __half2 h;
        memcpy(&h, &w[i], 4);
        f = __half22float2(h);
      } else {
        f = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
      }
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

template <int kE>
__global__ void __launch_bounds__(kNrThreads)
k_norm_rope(const NormRopeArgs a, const qsa_rope rope) {
  __shared__ float s_cos[kHeadDim / 2], s_sin[kHeadDim / 2], s_icos[kIdxDim / 2], s_isin[kIdxDim / 2];
  grid_dep_wait();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t = blockIdx.x;
  constexpr int64_t kSize = kE == QSA_ELEM_F32 ? 4 : 2;
  const int m = rope.n_rot >> 1;   // pairs
  const int nq = a.q_in ? a.Hq : 0, nk = a.k_in ? a.G : 0, ni = a.qi_in ? kIdxHeads : 0;
  const int rows = nq + nk + ni;
  // row r of the token: its queries, then its keys, then its indexer queries
  auto load = [&](int r, float (&x)[8]) {
    const char* p;
    if (r < nq) p = static_cast<const char*>(a.q_in) + (t * a.q_stride + (int64_t)r * kHeadDim) * kSize;
    else if (r < nq + nk) p = static_cast<const char*>(a.k_in) + (t * a.k_stride + (int64_t)(r - nq) * kHeadDim) * kSize;
    else p = static_cast<const char*>(a.qi_in) + (t * a.qi_stride + (int64_t)(r - nq - nk) * kIdxDim) * kSize;
    if (r < nq + nk) load_row<kE, 8>(p + lane * 8 * kSize, x);
    else load_row<kE, 4>(p + lane * 4 * kSize, x);
  };
  float x[8];
  if (warp < rows) load(warp, x);

  if (tid < m && nq + nk > 0) {
    const int64_t p = a.pos[(int64_t)rope.axis[tid] * a.n_tokens + t];
    sincos_turn((unsigned long long)p * rope.turns[tid], &s_sin[tid], &s_cos[tid]);
  }
  if (ni > 0 && tid >= kNrThreads - kIdxDim / 2) {
    const int i = tid - (kNrThreads - kIdxDim / 2);
    const int64_t p = a.idx_pos[t];
    sincos_turn((unsigned long long)p * rope.idx_turns[i], &s_isin[i], &s_icos[i]);
  }
  __syncthreads();

  // this lane's pairs of a 256-dim row: dims 8 lane .. +7 pair with the same
  // dims m further (first half) or m before (second half)
  const int hl = m >> 3;                                      // lanes of each half
  const bool rot = lane < 2 * hl, second = lane >= hl;
  const int partner = !rot ? lane : (second ? lane - hl : lane + hl);
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int pr = 8 * (second ? lane - hl : lane) + i;
    c[i] = rot ? s_cos[pr] : 1.f;
    s[i] = rot ? (second ? s_sin[pr] : -s_sin[pr]) : 0.f;
  }
  for (int r = warp; r < rows; r += kNrWarps) {
    if (r != warp) load(r, x);
    const bool wide = r < nq + nk;
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = (i < 4 || wide) ? fmaf(x[i], x[i], ss) : ss;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) ss += __shfl_xor_sync(kFull, ss, o);
    const float inv = 1.0f / sqrtf(ss * (wide ? 1.0f / kHeadDim : 1.0f / kIdxDim) + a.eps);
    if (wide) {
      const float4* w = reinterpret_cast<const float4*>(r < nq ? a.q_w : a.k_w) + 2 * lane;
      const float4 w0 = w[0], w1 = w[1];
      const float wv[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
      __half2 o[4];
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * wv[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float other = __shfl_sync(kFull, x[i], partner);
        y[i] = rot ? fmaf(x[i], c[i], other * s[i]) : x[i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __floats2half2_rn(y[2 * i], y[2 * i + 1]);
      __half* dst = r < nq ? a.q + (t * a.Hq + r) * kHeadDim : a.k + (t * a.G + (r - nq)) * kHeadDim;
      uint4 v;
      memcpy(&v, o, 16);
      reinterpret_cast<uint4*>(dst)[lane] = v;
    } else {
      const float4 w = reinterpret_cast<const float4*>(a.qi_w)[lane];
      const float wv[4] = {w.x, w.y, w.z, w.w};
      const int pr = 4 * (lane & 15);
      float y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = x[i] * inv * wv[i];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float other = __shfl_xor_sync(kFull, x[i], 16);
        y[i] = fmaf(x[i], s_icos[pr + i], lane < 16 ? -other * s_isin[pr + i] : other * s_isin[pr + i]);
      }
      reinterpret_cast<float4*>(a.qi + (t * kIdxHeads + (r - nq - nk)) * kIdxDim)[lane] = make_float4(y[0], y[1], y[2], y[3]);
    }
  }
  // the successor reads these rows before its dependency wait: it starts only
  // after this grid's last CTA, so the rows have to be out by then
  __threadfence();
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, const qsa_rope& rope, int elem, cudaStream_t stream) {
  if (a.n_tokens <= 0) return cudaSuccess;
  const dim3 grid((unsigned)a.n_tokens), block(kNrThreads);
  prof_before(kKNormRope, stream);
  cudaError_t e = elem == QSA_ELEM_F16    ? launch_pdl(k_norm_rope<QSA_ELEM_F16>, grid, block, 0, stream, 1, a, rope)
                  : elem == QSA_ELEM_BF16 ? launch_pdl(k_norm_rope<QSA_ELEM_BF16>, grid, block, 0, stream, 1, a, rope)
                                          : launch_pdl(k_norm_rope<QSA_ELEM_F32>, grid, block, 0, stream, 1, a, rope);
  prof_after(kKNormRope, stream);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// turns[i] = theta^(-i/m) / (2 pi) of a turn, scaled to 2^64 and rounded: the
// frequency in double, its fraction of a turn in long double.
unsigned long long turn_of(double theta, double exponent) {
  const long double two_pi = 6.28318530717958647692528676655900577L;
  const double f = std::pow(theta, exponent);
  const long double x = ((long double)f / two_pi) * 18446744073709551616.0L;
  return x >= 18446744073709551615.0L ? ~0ull : (unsigned long long)(x + 0.5L);
}

}  // namespace qsa
