// rotary.cuh -- rotary position embedding of packed bf16 rows, and the pair
// arithmetic that the paged-cache append shares with it.
//
// With R = 2 * num_freqs <= head_dim, pair i < R/2 of a row at position pos is
// (x[i], x[i + R/2]) in the half layout and (x[2i], x[2i + 1]) in the
// interleaved one, and becomes, for theta = pos * inv_freq[i],
//   a' = m (a cos theta - b sin theta),  b' = m (b cos theta + a sin theta);
// x[R:] is copied.  The map is orthogonal up to m, so its gradient is the same
// map with -theta (`sign` = -1).
//
// The angle, its reduction by quarter turns and its sine and cosine are taken in
// 64 bits, by Taylor sums on [-pi/4, pi/4], and rounded to fp32 once: a position
// of a million loses nothing (in fp32 the product alone would be off by 2^-4
// radians there), and neither do pairs that nearly cancel (an angle rounded to
// fp32 before its sine turns them by up to 2^-23).  The pair is computed in fp32
// and rounded to bf16 once.
//
// Work unit: 16 elements of a row = 8 pairs = two 16-byte loads and stores.  In
// the half layout they are x[8c..] and x[R/2 + 8c..], so the lanes of a row
// touch two contiguous runs.  One thread owns unit c of a token and walks over
// heads: the 8 cosines and sines, which cost more than the pairs of one head,
// are computed once per token and unit and stay in registers.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace attn {

struct RopeParams {
  const double* inv_freq;  // [half]
  int half;                // pairs per row; 0: nothing is rotated
  int interleaved;
  float mscale;
  float sign;              // +1, or -1 for the inverse rotation (the gradient)
};

// rows [tokens][heads][D], last dimension contiguous; strides in elements
struct RowsIn {
  const uint16_t* p;
  int64_t st, sh;
};
struct RowsOut {
  uint16_t* p;
  int64_t st, sh;
};

// the two 8-element runs of unit c
__device__ __forceinline__ void rope_offsets(const RopeParams& r, int c, int* a, int* b) {
  const bool turned = 8 * c < r.half;
  const bool split = turned && !r.interleaved;
  *a = split ? 8 * c : 16 * c;
  *b = split ? r.half + 8 * c : 16 * c + 8;
}

// cosines and sines (times mscale) of unit c at a position; c * 8 < half
__device__ __forceinline__ void rope_angles(const RopeParams& r, int c, int pos, float (&cs)[8],
                                            float (&sn)[8]) {
  const double p = static_cast<double>(pos);
  constexpr double M = 6755399441055744.0;  // 1.5 2^52: h + M rounds h to a whole number,
#pragma unroll                              // whose low bits are those of the sum
  for (int i = 0; i < 8; ++i) {
    const double h = __dmul_rn(__dmul_rn(p, r.inv_freq[8 * c + i]), 0.63661977236758134308);
    const double t = __dadd_rn(h, M);
    const int quarter = __double2loint(t) & 3;
    // the rest, at most half a quarter turn, in radians; cut off below 2^-32 of the results
    const double z = __dmul_rn(__dsub_rn(h, __dsub_rn(t, M)), 1.57079632679489661923);
    const double u = __dmul_rn(z, z);
    double a = __fma_rn(u, -1.0 / 39916800.0, 1.0 / 362880.0);
    a = __fma_rn(a, u, -1.0 / 5040.0);
    a = __fma_rn(a, u, 1.0 / 120.0);
    a = __fma_rn(a, u, -1.0 / 6.0);
    double b = __fma_rn(u, -1.0 / 3628800.0, 1.0 / 40320.0);
    b = __fma_rn(b, u, -1.0 / 720.0);
    b = __fma_rn(b, u, 1.0 / 24.0);
    b = __fma_rn(b, u, -0.5);
    const float s = static_cast<float>(__fma_rn(__dmul_rn(z, u), a, z));
    const float k = static_cast<float>(__fma_rn(u, b, 1.0));
    // turned by the whole quarters: (k, s), (-s, k), (-k, -s), (s, -k)
    const float ck = quarter & 1 ? s : k, sk = quarter & 1 ? k : s;
    cs[i] = r.mscale * ((quarter + 1) & 2 ? -ck : ck);
    sn[i] = r.mscale * (r.sign * (quarter & 2 ? -sk : sk));
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// the 8 pairs of a unit, in place; the roundings are spelled out, so that every
// kernel that rotates gives the same bits
__device__ __forceinline__ void rope_turn(const RopeParams& r, const float (&cs)[8],
                                          const float (&sn)[8], uint4& a, uint4& b) {
  uint32_t* wa = reinterpret_cast<uint32_t*>(&a);
  uint32_t* wb = reinterpret_cast<uint32_t*>(&b);
  auto first = [](float x, float y, float c, float s) { return __fmaf_rn(x, c, -__fmul_rn(y, s)); };
  auto second = [](float x, float y, float c, float s) { return __fmaf_rn(y, c, __fmul_rn(x, s)); };
  if (r.interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x = bf16_lo(wa[i]), y = bf16_hi(wa[i]);
      wa[i] = bf16_pair(first(x, y, cs[i], sn[i]), second(x, y, cs[i], sn[i]));
      x = bf16_lo(wb[i]), y = bf16_hi(wb[i]);
      wb[i] = bf16_pair(first(x, y, cs[4 + i], sn[4 + i]), second(x, y, cs[4 + i], sn[4 + i]));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x0 = bf16_lo(wa[i]), x1 = bf16_hi(wa[i]);
      const float y0 = bf16_lo(wb[i]), y1 = bf16_hi(wb[i]);
      const float c0 = cs[2 * i], c1 = cs[2 * i + 1], s0 = sn[2 * i], s1 = sn[2 * i + 1];
      wa[i] = bf16_pair(first(x0, y0, c0, s0), first(x1, y1, c1, s1));
      wb[i] = bf16_pair(second(x0, y0, c0, s0), second(x1, y1, c1, s1));
    }
  }
}

// the segment of packed row t: the last b with cu[b] <= t (empty segments
// before it are skipped); -1 for a row outside [cu[0], cu[batch])
__device__ __forceinline__ int find_segment(const int32_t* cu, int batch, int t) {
  if (t < cu[0] || t >= cu[batch]) return -1;
  int lo = 0, hi = batch;  // cu[lo] <= t < cu[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= t)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

struct RotaryParams {
  RopeParams rope;
  RowsIn q, k;
  RowsOut qo, ko;
  const int32_t* positions;  // [total], or null
  const int32_t* cu;         // [batch + 1], or null: position = row
  const int32_t* offsets;    // [batch], or null
  int zero_outside;          // rows of no segment: written as zeros, or left
  int batch, total, hq, heads;  // heads = hq + key/value heads
  int heads_per_thread;
};

constexpr int kRotaryThreads = 256;

// grid: (units of all rows / 256, groups of heads_per_thread heads).  Bound by
// HBM: every element is read once and written once.
template <int D>
__global__ void __launch_bounds__(kRotaryThreads, 3) attn_rotary_kernel(const RotaryParams p) {
  constexpr int UNITS = D / 16;
  const int64_t id = static_cast<int64_t>(blockIdx.x) * kRotaryThreads + threadIdx.x;
  const int t = static_cast<int>(id / UNITS), c = static_cast<int>(id % UNITS);
  if (t >= p.total) return;
  int pos = t;
  bool outside = false;
  if (p.positions) {
    pos = p.positions[t];
  } else if (p.cu) {
    const int b = find_segment(p.cu, p.batch, t);
    outside = b < 0;
    if (outside && !p.zero_outside) return;
    if (!outside) pos = t - p.cu[b] + (p.offsets ? p.offsets[b] : 0);
  }
  const bool turned = 8 * c < p.rope.half && !outside;
  float cs[8], sn[8];
  if (turned) rope_angles(p.rope, c, pos, cs, sn);
  int oa, ob;
  rope_offsets(p.rope, c, &oa, &ob);
  const int h0 = blockIdx.y * p.heads_per_thread;
  const int h1 = min(h0 + p.heads_per_thread, p.heads);
  constexpr int U = 4;  // heads in flight per thread
  for (int h = h0; h < h1; h += U) {
    uint4 a[U], b[U];
    uint16_t* dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u < h1) {
        const bool isq = h + u < p.hq;
        const RowsIn& in = isq ? p.q : p.k;
        const RowsOut& out = isq ? p.qo : p.ko;
        const int hh = isq ? h + u : h + u - p.hq;
        const uint16_t* src = in.p + t * in.st + hh * in.sh;
        dst[u] = out.p + t * out.st + hh * out.sh;
        a[u] = *reinterpret_cast<const uint4*>(src + oa);
        b[u] = *reinterpret_cast<const uint4*>(src + ob);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h + u < h1) {
        if (outside) a[u] = b[u] = make_uint4(0, 0, 0, 0);
        if (turned) rope_turn(p.rope, cs, sn, a[u], b[u]);
        *reinterpret_cast<uint4*>(dst[u] + oa) = a[u];
        *reinterpret_cast<uint4*>(dst[u] + ob) = b[u];
      }
    }
  }
}

}  // namespace attn
