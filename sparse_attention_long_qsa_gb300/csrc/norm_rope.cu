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
// scores take it.  The rotation is linear, so the row's factor 1 / sqrt(...)
// is applied after it and the sum of squares is not waited for.
//
// Angles reach 1e6 rad, where an fp32 product would be off by 6e-2 rad, so
// they are reduced in integers: a frequency is a 64-bit fixed-point fraction of
// a turn, the position times it wraps to the angle's fraction of a turn, whose
// top 32 bits (2^-32 turns, 1.5e-9 rad) are kept.  An angle within an eighth of
// a turn of a quarter then goes through the Taylor series of sine and cosine.
// (The general 64-bit form with sincospi cost as much as the rows: 20 of 55 us
// at 8,192 tokens.)
//
// A warp takes a stretch of the call's row batches (four head rows of a token,
// or its indexer rows) and needs no other warp: every warp of the GPU gets the
// same number, whatever the token count.  Lane l < m/4 holds dims 4l .. 4l+3
// and their partners m + 4l .., the other lanes 8 of the dims that do not turn,
// so every pair lives in one lane and no value crosses lanes but the sum; the
// lane's own pairs are also all the cosines and sines it needs, computed when
// the stretch reaches a token.  The kernel is bound by memory, so its loads do
// not pause: the next batch is in flight while one is finished.
#include <cmath>

#include "qsa_internal.cuh"

namespace qsa {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kNrThreads = 128;
constexpr int kNrWarps = kNrThreads / 32;
constexpr int kNrPerSm = 4;     // CTAs that share an SM (128 registers a thread)
constexpr int kBatch = 4;       // head rows in a batch
static_assert(kIdxHeads == kBatch, "the indexer's rows are one batch");
constexpr int kIdxPairs = kIdxDim / 2;

// Element pairs of one load: kE's element type, kN elements at p.
template <int kE, int kN>
struct Vec {
  static constexpr int kWords = kE == QSA_ELEM_F32 ? kN : kN / 2;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (kWords == 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (kWords == 2) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    }
  }
  // elements 2 i and 2 i + 1
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (kE == QSA_ELEM_F32) {
      return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    } else if constexpr (kE == QSA_ELEM_BF16) {
      return make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
      __half2 h;
      memcpy(&h, &w[i], 4);
      return __half22float2(h);
    }
  }
};

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n .reg .b64 a, b;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mul.rn.f32x2 a, a, b;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n .reg .b64 a, b, c;\n mov.b64 a, {%2, %3};\n mov.b64 b, {%4, %5};\n mov.b64 c, {%6, %7};\n"
      " fma.rn.f32x2 a, a, b, c;\n mov.b64 {%0, %1}, a;\n}\n"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

// Sine and cosine of p * turns / 2^64 turns.
__device__ __forceinline__ void sincos_at(int p, unsigned long long turns, float* sn, float* cs) {
  const uint32_t lo = (uint32_t)turns, hi = (uint32_t)(turns >> 32);
  // bits 32..63 of the product with p's two's complement (2^32 more than a negative p)
  const uint32_t u = (uint32_t)p * hi + __umulhi((uint32_t)p, lo) - (p < 0 ? lo : 0u);
  const uint32_t q = (u + 0x20000000u) >> 30;                  // nearest quarter of a turn
  const float x = (float)(int)(u - (q << 30)) * (6.283185307179586f / 4294967296.0f);   // |x| <= pi / 4
  const float x2 = x * x;
  // to x^9 and x^10: what follows is below 2e-9
  float s = fmaf(x2, 1.0f / 362880.0f, -1.0f / 5040.0f);
  s = fmaf(s, x2, 1.0f / 120.0f);
  s = fmaf(s, x2, -1.0f / 6.0f);
  s = fmaf(s * x2, x, x);
  float c = fmaf(x2, -1.0f / 3628800.0f, 1.0f / 40320.0f);
  c = fmaf(c, x2, -1.0f / 720.0f);
  c = fmaf(c, x2, 1.0f / 24.0f);
  c = fmaf(c, x2, -0.5f);
  c = fmaf(c, x2, 1.0f);
  const float a = (q & 1u) ? c : s, b = (q & 1u) ? s : c;
  *sn = (q & 2u) ? -a : a;
  *cs = ((q + 1u) & 2u) ? -b : b;
}

// Per lane v[i], i < 4: lane l returns the warp's sum of v[l / 8].
__device__ __forceinline__ float warp_sums4(const float (&v)[4], int lane) {
  const bool hi = (lane & 16) != 0, mid = (lane & 8) != 0;
  float a = (hi ? v[2] : v[0]) + __shfl_xor_sync(kFull, hi ? v[0] : v[2], 16);
  float b = (hi ? v[3] : v[1]) + __shfl_xor_sync(kFull, hi ? v[1] : v[3], 16);
  float x = (mid ? b : a) + __shfl_xor_sync(kFull, mid ? a : b, 8);
#pragma unroll
  for (int o = 4; o >= 1; o >>= 1) x += __shfl_xor_sync(kFull, x, o);
  return x;
}

template <int kE>
__global__ void __launch_bounds__(kNrThreads, kNrPerSm)
k_norm_rope(const NormRopeArgs a, const __grid_constant__ qsa_rope rope) {
  constexpr int kSize = kE == QSA_ELEM_F32 ? 4 : 2;
  grid_dep_wait();
  const int lane = threadIdx.x & 31;
  const int m = rope.n_rot >> 1;
  const bool rot = lane < (m >> 2);
  // this lane's two groups of 4 dims
  const int d0 = rot ? 4 * lane : 2 * m + 8 * (lane - (m >> 2)), dd = rot ? m : 4;

  // Every lane has its own entries of the table: read through a generic
  // address, as constant loads of 32 different entries take turns.
  const qsa_rope* table = &rope;
  asm volatile("" : "+l"(table));
  const bool turned = rot && (a.q_in != nullptr || a.k_in != nullptr);
  unsigned long long turns[4] = {};
  unsigned axes = 0u;   // of the four pairs, a byte each
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (turned) {
      turns[j] = table->turns[d0 + j];
      axes |= (unsigned)table->axis[d0 + j] << (8 * j);
    }

  // a token's batches: its query rows, its key rows, its indexer rows
  const int bq = a.q_in ? (a.Hq + kBatch - 1) / kBatch : 0, bk = a.k_in ? (a.G + kBatch - 1) / kBatch : 0;
  const int batches = bq + bk + (a.qi_in ? 1 : 0);
  const int64_t units = (int64_t)a.n_tokens * batches, warps = (int64_t)gridDim.x * kNrWarps;
  const int64_t me = (int64_t)blockIdx.x * kNrWarps + (threadIdx.x >> 5);
  const int64_t begin = units * me / warps, left_units = units * (me + 1) / warps - begin;
  int64_t t = begin / batches;
  int b = (int)(begin - t * batches);

  struct Rows {
    Vec<kE, 4> x[kBatch][2];   // of indexer rows, the first half of each
  };
  auto load = [&](int64_t tk, int bt, Rows& o) {
    if (bt < bq + bk) {
      const bool is_q = bt < bq;
      const int r0 = kBatch * (is_q ? bt : bt - bq), left = (is_q ? a.Hq : a.G) - r0;
      const char* p = (is_q ? static_cast<const char*>(a.q_in) + tk * a.q_stride * kSize
                            : static_cast<const char*>(a.k_in) + tk * a.k_stride * kSize) +
                      (r0 * kHeadDim + d0) * kSize;
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i < left) {
          o.x[i][0].load(p + i * (kHeadDim * kSize));
          o.x[i][1].load(p + i * (kHeadDim * kSize) + dd * kSize);
        }
    } else {
      const char* p = static_cast<const char*>(a.qi_in) + (tk * a.qi_stride + 2 * lane) * kSize;
#pragma unroll
      for (int i = 0; i < kIdxHeads; ++i) {
        Vec<kE, 2> v;
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          v.load(p + (i * kIdxDim + g * kIdxPairs) * kSize);
#pragma unroll
          for (int k = 0; k < Vec<kE, 2>::kWords; ++k) o.x[i][g].w[k] = v.w[k];
        }
      }
    }
  };
  float2 c[2], s[2];   // of this lane's pairs at token t
  auto angles = [&]() {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      c[j] = make_float2(1.f, 1.f), s[j] = make_float2(0.f, 0.f);
      if (turned) {
        const int p0 = a.pos[(int64_t)((axes >> (16 * j)) & 255u) * a.n_tokens + t];
        const int p1 = a.pos[(int64_t)((axes >> (16 * j + 8)) & 255u) * a.n_tokens + t];
        sincos_at(p0, turns[2 * j], &s[j].x, &c[j].x);
        sincos_at(p1, turns[2 * j + 1], &s[j].y, &c[j].y);
      }
    }
  };
  // x[i] of `rows` rows: sum of squares, 1 / root in every lane
  auto roots = [&](const float (&sq)[kBatch], float inv_n, float (&inv)[kBatch]) {
    const float r = rsqrtf(warp_sums4(sq, lane) * inv_n + a.eps);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) inv[i] = __shfl_sync(kFull, r, 8 * i);
  };
  auto finish = [&](const Rows& o) {
    float sq[kBatch], inv[kBatch];
    if (b < bq + bk) {
      const bool is_q = b < bq;
      const int r0 = kBatch * (is_q ? b : b - bq), left = (is_q ? a.Hq : a.G) - r0;
      // out_0 = x_0 (w_0 cos) - x_1 (w_1 sin), out_1 = x_1 (w_1 cos) + x_0 (w_0 sin)
      const float* wp = (is_q ? a.q_w : a.k_w) + d0;
      float2 c0[2], c1[2], s0[2], s1[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 w0 = *reinterpret_cast<const float2*>(wp + 2 * j);
        const float2 w1 = *reinterpret_cast<const float2*>(wp + dd + 2 * j);
        c0[j] = mul2(w0, c[j]), c1[j] = mul2(w1, c[j]), s0[j] = mul2(w0, s[j]);
        s1[j] = mul2(w1, make_float2(-s[j].x, -s[j].y));
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        float2 q = make_float2(0.f, 0.f);
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int j = 0; j < 2; ++j) q = fma2(o.x[i][g].pair(j), o.x[i][g].pair(j), q);
        sq[i] = q.x + q.y;
      }
      roots(sq, 1.0f / kHeadDim, inv);
      __half* out = (is_q ? a.q + (t * a.Hq + r0) * kHeadDim : a.k + (t * a.G + r0) * kHeadDim) + d0;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (i >= left) break;
        const float2 inv2 = make_float2(inv[i], inv[i]);
        __half2 h[2][2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 x0 = o.x[i][0].pair(j), x1 = o.x[i][1].pair(j);
          const float2 lo = mul2(fma2(x0, c0[j], mul2(x1, s1[j])), inv2);
          const float2 hi = mul2(fma2(x1, c1[j], mul2(x0, s0[j])), inv2);
          h[0][j] = __floats2half2_rn(lo.x, lo.y);
          h[1][j] = __floats2half2_rn(hi.x, hi.y);
        }
        uint2 v;
        memcpy(&v, h[0], 8);
        *reinterpret_cast<uint2*>(out + i * kHeadDim) = v;
        memcpy(&v, h[1], 8);
        *reinterpret_cast<uint2*>(out + i * kHeadDim + dd) = v;
      }
      return;
    }
    // ---- indexer rows: dims 2 l, 2 l + 1 and their partners 64 further
    float2 ci, si;
    const int p = a.idx_pos[t];
    sincos_at(p, table->idx_turns[2 * lane], &si.x, &ci.x);
    sincos_at(p, table->idx_turns[2 * lane + 1], &si.y, &ci.y);
    const float2 w0 = *reinterpret_cast<const float2*>(a.qi_w + 2 * lane);
    const float2 w1 = *reinterpret_cast<const float2*>(a.qi_w + kIdxPairs + 2 * lane);
    const float2 c0 = mul2(w0, ci), c1 = mul2(w1, ci), s0 = mul2(w0, si), s1 = mul2(w1, make_float2(-si.x, -si.y));
    float2 x[kIdxHeads][2];
#pragma unroll
    for (int i = 0; i < kIdxHeads; ++i) {
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        Vec<kE, 2> v;
#pragma unroll
        for (int k = 0; k < Vec<kE, 2>::kWords; ++k) v.w[k] = o.x[i][g].w[k];
        x[i][g] = v.pair(0);
      }
      const float2 q = fma2(x[i][0], x[i][0], mul2(x[i][1], x[i][1]));
      sq[i] = q.x + q.y;
    }
    roots(sq, 1.0f / kIdxDim, inv);
    float* out = a.qi + t * (kIdxHeads * kIdxDim) + 2 * lane;
#pragma unroll
    for (int i = 0; i < kIdxHeads; ++i) {
      const float2 inv2 = make_float2(inv[i], inv[i]);
      *reinterpret_cast<float2*>(out + i * kIdxDim) = mul2(fma2(x[i][0], c0, mul2(x[i][1], s1)), inv2);
      *reinterpret_cast<float2*>(out + i * kIdxDim + kIdxPairs) = mul2(fma2(x[i][1], c1, mul2(x[i][0], s0)), inv2);
    }
  };

  // ---- the stretch, two batches in registers in turn
  int64_t left = left_units;
  bool fresh = true;   // the angles of token t are not there yet
  Rows x = {}, y = {};
  auto turn = [&](const Rows& cur, Rows& next) {
    const bool last = b + 1 == batches;
    if (left > 1) load(last ? t + 1 : t, last ? 0 : b + 1, next);
    if (fresh) angles();
    finish(cur);
    fresh = last;
    t += last ? 1 : 0;
    b = last ? 0 : b + 1;
    --left;
  };
  if (left > 0) load(t, b, x);
  while (left > 0) {
    turn(x, y);
    if (left > 0) turn(y, x);
  }
  // the successor reads these rows before its dependency wait: it starts only
  // after this grid's last CTA, so the rows have to be out by then
  __threadfence();
}

template <int kE>
cudaError_t launch(const NormRopeArgs& a, const qsa_rope& rope, cudaStream_t stream) {
  const int64_t batches = (a.q_in ? ceil_div(a.Hq, kBatch) : 0) + (a.k_in ? ceil_div(a.G, kBatch) : 0) + (a.qi_in ? 1 : 0);
  const int64_t ctas = ceil_div(a.n_tokens * batches, kNrWarps);
  constexpr int64_t kResident = 152 * kNrPerSm;
  return launch_pdl(k_norm_rope<kE>, dim3((unsigned)(ctas < kResident ? ctas : kResident)), dim3(kNrThreads), 0, stream,
                    1, a, rope);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeArgs& a, const qsa_rope& rope, int elem, cudaStream_t stream) {
  if (a.n_tokens <= 0) return cudaSuccess;
  prof_before(kKNormRope, stream);
  const cudaError_t e = elem == QSA_ELEM_F16    ? launch<QSA_ELEM_F16>(a, rope, stream)
                        : elem == QSA_ELEM_BF16 ? launch<QSA_ELEM_BF16>(a, rope, stream)
                                                : launch<QSA_ELEM_F32>(a, rope, stream);
  prof_after(kKNormRope, stream);
  if (e != cudaSuccess) return e;
  return cudaGetLastError();
}

// theta^exponent / (2 pi) of a turn, less whole turns (a theta below one gives
// frequencies above one radian), scaled to 2^64 and rounded: the frequency in
// double, its fraction of a turn in long double.
unsigned long long turn_of(double theta, double exponent) {
  const long double two_pi = 6.28318530717958647692528676655900577L;
  const double f = std::pow(theta, exponent);
  const long double turns = (long double)f / two_pi;
  const long double x = (turns - std::floor(turns)) * 18446744073709551616.0L;
  return x >= 18446744073709551615.0L ? ~0ull : (unsigned long long)(x + 0.5L);
}

}  // namespace qsa
