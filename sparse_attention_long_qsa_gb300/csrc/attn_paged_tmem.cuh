// What the tensor-memory kernels of qsa_paged_attn share.
#pragma once

#include "attn_paged.cuh"
#include "tc_util.cuh"

namespace qsa {
namespace {

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};\n" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void bar_named(int id, int threads) {
  asm volatile("bar.sync %0, %1;\n" ::"r"(id), "r"(threads) : "memory");
}
// (x, y) = (x, y) * m + a
__device__ __forceinline__ void fma2(float& x, float& y, float m, float a) {
  asm("{\n .reg .b64 v, w, c;\n mov.b64 v, {%0, %1};\n mov.b64 w, {%2, %2};\n mov.b64 c, {%3, %3};\n"
      " fma.rn.f32x2 v, v, w, c;\n mov.b64 {%0, %1}, v;\n}\n"
      : "+f"(x), "+f"(y)
      : "f"(m), "f"(a));
}
__device__ __forceinline__ void add2(float& x, float& y, float a, float b) {
  asm("{\n .reg .b64 v, w;\n mov.b64 v, {%0, %1};\n mov.b64 w, {%2, %3};\n"
      " add.rn.f32x2 v, v, w;\n mov.b64 {%0, %1}, v;\n}\n"
      : "+f"(x), "+f"(y)
      : "f"(a), "f"(b));
}
// Probabilities of a tile are 2^(s - reference + kUp) of each row, in two fp16 parts, the second what the first leaves:
// 22 bits down to 2^-2 and less below, as a part ends at 2^-24.  So the reference follows the tiles.  It goes up where a
// tile's largest score is kSlack above it (they stay below 2^15.2), and down where the largest is kLow below (of the tile:
// what the cells of other tiles weigh does not cost its weights their bits); what has been summed up is scaled along, which
// fp32 holds as long as no reference is kFar below another.  Ordinary rows are scaled once or twice a run: their tiles'
// largest scores lie a few places apart.  Where a few cells of a tile stand out (kAlone above some eighth of the tile's,
// or above the other half's), the others get what is left of fp16's range: the largest weight starts at its top.
// (With a reference that only went up, 2^7 for the largest: 24 places below a sink without value outputs were 8e-4 off, and
// 40 below meaningless.  Rows of ordinary scores take the same time; scores that spread by 6 places and more take 4 to 10 % more.)
constexpr float kUp = 7.f, kSlack = 8.f, kLow = 13.f, kFar = 64.f, kAlone = 13.f;
// From kBig on a score's last place is so much that its product with the scale, the reference and their difference are
// rounded one by one, so that the largest comes to the reference exactly, which then follows every rise.  (In one rounding
// scores of 1e7 and more were NaN.)
constexpr float kBig = 1048576.f;
__device__ __forceinline__ bool is_big(float m) { return fabsf(m) > kBig && fabsf(m) < -kNoMax; }
// The largest of a row's scores in half a tile, from that of four interleaved parts of it (-inf: nothing is visible), and
// whether it stands out.
__device__ __forceinline__ float tile_top(const float (&t)[4], float scale2, bool& alone) {
  const float top = fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3]));
  float low = top;
#pragma unroll
  for (int j = 0; j < 4; ++j) low = t[j] == -INFINITY ? low : fminf(low, t[j]);
  alone = (top - low) * scale2 > kAlone;
  return top;
}
// The row's reference after a tile whose halves' largest are x and y.  `high`: the highest so far.
__device__ __forceinline__ float next_reference(float m, float& high, float x, float y, bool alone, bool big, float scale2) {
  const float top2 = fmaxf(x, y), top = top2 == -INFINITY ? top2 : top2 * scale2;   // (-inf times zero would be NaN)
  float nm = m;
  if (top > m + (big ? 0.f : kSlack) || top != top) {
    alone = alone || fabsf(x - y) * scale2 > kAlone;
    nm = alone && fminf(x, y) > -INFINITY && fabsf(top) <= kBig ? top - kSlack : top;
  } else if (top < m - kLow && top > -INFINITY) {
    nm = fminf(m, fmaxf(top, high - kFar));
  }
  high = fmaxf(high, nm);
  return nm;
}
// Two probabilities' parts.
__device__ __forceinline__ uint32_t first_part(float x, float y, float2& back) {
  const __half2 h = __floats2half2_rn(x, y);
  back = __half22float2(h);
  return bits(h);
}
// bits [0, n) of a word, any n
__device__ __forceinline__ uint32_t below(int n) { return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u; }

// Infinite values of V and NaN make the sum of their dim, whatever else it has: those that a lane's row sees among the run's
// cells [v0, v_end) (reading order), added up, take its place in the row's 128 columns (null: the lane has no row).
// sees(p): whether the row sees position p.  load(c, k, x): dims 16 k .. + 15 of cell c, as halves.  By a whole warp, after
// its results are out: a lane a cell (a chain of three loads for 32 of them), then a lane a row.
template <typename Sees, typename Load>
__device__ __forceinline__ void put_not_finite(const PagedArgs& a, const Run& run, int v0, int v_end, float* row, Sees sees,
                                               Load load) {
  const int lane = threadIdx.x & 31;
  __syncwarp();   // the rows have been written, by other lanes
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    float y[16] = {};
#pragma unroll 1
    for (int v = v0; v < v_end; v += 32) {
      const int at = v + lane;
      const int c = checked_cell(a, cell_at(a, run, at, slot_at(a, run, at, v_end, false, nullptr), false, nullptr), false, nullptr);
      uint32_t x[8] = {}, any = 0u;
      if (c >= 0) load(c, k, x);
#pragma unroll
      for (int j = 0; j < 8; ++j) any |= ((x[j] & 0x7c007c00u) + 0x04000400u) & 0x80008000u;   // an exponent of ones
      unsigned who = __ballot_sync(kFull, any != 0u);
      const int p = at < v_end ? pos_of(run.g, at) : 0;
#pragma unroll 1
      for (; who; who &= who - 1u) {
        const int l = __ffs((int)who) - 1;
        const bool s = sees(__shfl_sync(kFull, p, l));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t w = __shfl_sync(kFull, x[j], l);
          if (s) add_not_finite(y[2 * j], y[2 * j + 1], w);
        }
      }
    }
    if (row != nullptr) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (y[j] != 0.f) row[16 * k + j] = y[j];
    }
  }
}

// The tensor cores cut each sum to 24 bits, and 2,600 additions in place would leave a run's result 4e-5 too small.  So a
// run is cut into stretches of about 280 additions (5e-6), whose sums are added in fp32 in the run's rows of the workspace.
constexpr int kMostAdditions = 288;
__device__ __forceinline__ int stretch_of(int tiles, int additions) {
  const int most = kMostAdditions / additions, n = (tiles + most - 1) / most;
  return (tiles + n - 1) / n;
}
// A stretch's or a run's sums: of the warp's 32 rows (token first / 8 and on, head first % 8; a lane a row) 128 columns of
// tensor memory, and `old` (if there is one: rows of the same order, 256 values apart) times fs, all times w, to
// base[token * stride + head * 256].  A warp's stores of a lane a row would touch 32 lines each, so 16 columns at a time
// pass through shared memory and go out as 64 bytes of eight rows.  kCheck: returns whether the lane's row holds columns
// that are not finite.
constexpr int kOutPitch = 20;
template <bool kCheck>
__device__ __forceinline__ bool write_rows(uint32_t taddr, float (*buf)[kOutPitch], float w, float* base, int64_t stride,
                                           const float* old, float fs, int first, int tokens) {
  const int lane = threadIdx.x & 31, col = 4 * (lane & 3), sub = lane >> 2;
  const bool wide = (reinterpret_cast<uintptr_t>(base) & 15u) == 0u;
  // sums added where they are: without waiting for them, where no row has another reference since
  const bool add = old == base && __all_sync(kFull, fs == 1.f);
  const bool read = old != nullptr && !add;
  // this lane stores four columns of rows 8 i + sub: of tokens first / 8 + i, head sub
  const int have = tokens - (first >> 3);
  float* out = base + (first >> 3) * stride + sub * kHeadDim + col;
  const float* from = old + (int64_t)(first + sub) * kHeadDim + col;
  float rw[4], rf[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) rw[i] = __shfl_sync(kFull, w, 8 * i + sub), rf[i] = __shfl_sync(kFull, fs, 8 * i + sub);
  float z[4] = {};   // zeros, or NaN
#pragma unroll 1
  for (int k = 0; k < 8; k += 2) {
    uint32_t o[2][16];
    tmem_ld16_nowait(taddr + 16 * k, o[0]);
    tmem_ld16_nowait(taddr + 16 * k + 16, o[1]);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float4 y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (read && i < have) y[i] = __ldcg(reinterpret_cast<const float4*>(from + i * (8 * kHeadDim) + 16 * (k + c)));
      }
      if constexpr (kCheck) {
#pragma unroll
        for (int j = 0; j < 16; ++j) z[j & 3] = fmaf(__uint_as_float(o[c][j]), 0.f, z[j & 3]);
      }
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 16; j += 4)
        *reinterpret_cast<uint4*>(&buf[lane][j]) = make_uint4(o[c][j], o[c][j + 1], o[c][j + 2], o[c][j + 3]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float4 x = *reinterpret_cast<const float4*>(&buf[8 * i + sub][col]);
        float* to = out + i * stride + 16 * (k + c);
        if (i >= have) continue;
        if (add) {
          asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};\n" ::"l"(to), "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w)
                       : "memory");
          continue;
        }
        x.x = fmaf(rf[i], y[i].x, x.x) * rw[i], x.y = fmaf(rf[i], y[i].y, x.y) * rw[i];
        x.z = fmaf(rf[i], y[i].z, x.z) * rw[i], x.w = fmaf(rf[i], y[i].w, x.w) * rw[i];
        if (wide) {
          *reinterpret_cast<float4*>(to) = x;
        } else {
          to[0] = x.x, to[1] = x.y, to[2] = x.z, to[3] = x.w;
        }
      }
    }
  }
  return kCheck && (z[0] + z[1]) + (z[2] + z[3]) != 0.f;
}

}  // namespace
}  // namespace qsa
