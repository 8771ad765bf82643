// paged_append.cuh -- new keys and values written into a paged cache, the keys
// (and, in the same launch, the queries) rotated on the way.
//
// Token i of the n new ones of sequence b has position p = seqlens_k[b] - n + i
// (seqlens_k counts the new tokens); its row goes to slot p % page_size of page
// block_table[b][p / page_size].  A bf16 cache holds the rotated row rounded to
// bf16, the same bits attn_rotary gives.
//
// An e4m3 cache holds code = e4m3(y / s) of that bf16 row y, with one scale s
// for each (page, key/value head):
//   need = the least power of two >= 2^-64 with max |y| <= 448 need, over the
//          finite y that this call writes to the page,
//   s'   = need if this call writes slot 0 of the page, else max(s, need).
// Powers of two: a floating-point code loses nothing in relative precision by
// them (only the codes below 2^-6 s have fewer bits), y / s is exact, and when
// a page's scale grows, its earlier codes move by an exact factor and change
// only where they fall below the smallest normal code.  Values that are not
// finite are held as NaN and left out of the maximum.
//
// Two kernels, chosen by the largest number of new tokens (kAppendFew):
//   few   one group of D / 16 lanes per (sequence, page, head), for K and for V,
//         and per (token, query head): all heads at once, the maximum by
//         shuffles, the few tokens of a page in a loop.  Bound by latency.
//   page  one CTA per (sequence, page, group of heads); a thread owns unit c of
//         one or more rows, keeps their cosines and sines in registers and
//         walks over the heads; the page's maximum by one redux and one shared
//         atomic per warp.  Bound by HBM.
// Rows whose position is negative or past the block table, and pages outside
// the pool, are not written; their queries are rotated all the same.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "rotary.cuh"

namespace attn {

struct CacheView {
  uint8_t* p;
  float* scale;               // [num_pages][nheads_kv]; null for bf16
  int64_t s_page, s_token, s_head;  // in elements
};

struct AppendParams {
  RopeParams rope;            // half = 0: no rotation
  RowsIn k, v, q;             // q.p null: no queries
  RowsOut qo;
  CacheView kc, vc;
  const int32_t* table;       // [batch][table_stride], pages_per_seq used
  int64_t table_stride;
  const int32_t* cu;          // [batch + 1]
  const int32_t* seqlens;     // [batch]
  int batch, total, hq, hkv;
  int page_shift, num_pages, pages_per_seq;
  int page_bound;             // pages the new tokens of a sequence can touch
  int heads_per_cta;          // page kernel: key/value heads per CTA
  int kv_groups;              // page kernel: grid.y of the key/value part
  int q_heads_per_cta;
};

constexpr int kMinScaleExp = -64;
constexpr int kAppendFew = 8;

// the new tokens of sequence b in the page_index-th page they touch
struct PageSpan {
  int page;       // -1: nothing to write
  int first, last;  // positions [first, last)
  int64_t row0;   // packed row of position 0 (row = row0 + position)
};

__device__ __forceinline__ PageSpan page_span(const AppendParams& p, int b, int j) {
  PageSpan s;
  const int c0 = p.cu[b], n = p.cu[b + 1] - c0, len = p.seqlens[b];
  const int start = len - n;
  const int jp = (start >> p.page_shift) + j;  // below 0 for positions below 0
  s.row0 = static_cast<int64_t>(c0) - start;
  // (a page may begin or end past 32 bits)
  const int64_t begin = static_cast<int64_t>(jp) << p.page_shift;
  const int64_t end = begin + (int64_t(1) << p.page_shift);
  s.first = begin >= len ? len : max(start, static_cast<int>(begin));
  s.last = end < len ? static_cast<int>(end) : len;
  s.page = -1;
  if (n > 0 && s.first < s.last && jp >= 0 && jp < p.pages_per_seq) {
    const int page = p.table[b * p.table_stride + jp];
    if (static_cast<unsigned>(page) < static_cast<unsigned>(p.num_pages)) s.page = page;
  }
  return s;
}

// largest |bf16| of 16 elements as bits: a value of 0x7f80 or more is not finite
__device__ __forceinline__ uint32_t abs_max_bits(const uint4& a, const uint4& b) {
  constexpr uint32_t M = 0x7fff7fffu;
  uint32_t m = __vmaxu2(__vmaxu2(a.x & M, a.y & M), __vmaxu2(a.z & M, a.w & M));
  m = __vmaxu2(m, __vmaxu2(__vmaxu2(b.x & M, b.y & M), __vmaxu2(b.z & M, b.w & M)));
  return max(m & 0xffffu, m >> 16);
}
// the same over the finite elements only
__device__ __forceinline__ uint32_t finite_max_bits(const uint4& a, const uint4& b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t lo = w[i] & 0x7fffu, hi = (w[i] >> 16) & 0x7fffu;
    if (lo < 0x7f80u) m = max(m, lo);
    if (hi < 0x7f80u) m = max(m, hi);
  }
  return m;
}

// exponent of the least power of two s >= 2^kMinScaleExp with amax <= 448 s;
// 448 = 1.75 * 2^8, amax is the bits of a finite bf16
__device__ __forceinline__ int scale_exponent(uint32_t amax_bits) {
  const int e = static_cast<int>(amax_bits >> 7) - 127 - 8 + ((amax_bits & 0x7fu) > 0x60u ? 1 : 0);
  return max(e, kMinScaleExp);  // amax 0 and subnormals fall under the floor too
}
__device__ __forceinline__ float exp2_int(int e) {  // -126 <= e <= 127
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// two fp32 -> two e4m3 codes, round to nearest even; not finite -> NaN
__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  uint32_t w = r;
  // an infinity would saturate; finite quotients here are at most 448 (and a
  // rounding, under a scale that is not a power of two)
  if (fabsf(lo) > 1e30f) w |= 0x007fu;
  if (fabsf(hi) > 1e30f) w |= 0x7f00u;
  return w;
}

// 8 bf16 -> 8 codes of x / scale.  Under a power of two that is a product.  Under another
// quantiser's scale the product with the reciprocal is corrected by the remainder, which
// rounds as a division does: the product alone misses ties between codes (23/16 x 1.75 is
// one).  (The correction under every scale costs 3 of 77 us of the prompts below.)
struct ScaleOf {
  float s, inv;
};
__device__ __forceinline__ ScaleOf scale_of(float s) { return {s, __frcp_rn(s)}; }

__device__ __forceinline__ float quotient(float x, const ScaleOf& s) {
  const float q = __fmul_rn(x, s.inv);
  const float r = __fmaf_rn(__fmaf_rn(-q, s.s, x), s.inv, q);  // not finite: NaN
  return __uint_as_float(__float_as_uint(r) | (__float_as_uint(x) & 0x80000000u));  // -0
}

__device__ __forceinline__ uint2 quantise8(const uint4& a, const ScaleOf& s) {
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
  uint32_t c[4];
  if ((__float_as_uint(s.s) & 0x7fffffu) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = e4m3_pair(bf16_lo(w[i]) * s.inv, bf16_hi(w[i]) * s.inv);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = e4m3_pair(quotient(bf16_lo(w[i]), s), quotient(bf16_hi(w[i]), s));
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// 4 codes times a factor <= 1, rounded to codes again
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"(static_cast<uint16_t>(w & 0xffffu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"(static_cast<uint16_t>(w >> 16)));
  float x[4];
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
      : "=f"(x[0]), "=f"(x[1]) : "r"(h0));
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
      : "=f"(x[2]), "=f"(x[3]) : "r"(h1));
  return e4m3_pair(x[0] * f, x[1] * f) | (e4m3_pair(x[2] * f, x[3] * f) << 16);
}

__device__ __forceinline__ uint4 rescale16(const uint4& z, float f) {
  return make_uint4(rescale4(z.x, f), rescale4(z.y, f), rescale4(z.z, f), rescale4(z.w, f));
}

// the scale after this call: *grow is old / new where earlier codes have to move
__device__ __forceinline__ float next_scale(float old, int need_exp, bool fresh, float* grow) {
  const float need = exp2_int(need_exp);
  *grow = 1.f;
  if (fresh) return need;
  if (need > old) {
    *grow = old / need;
    return need;
  }
  return old;
}

__device__ __forceinline__ void load_unit(const RowsIn& r, int64_t row, int h, int oa, int ob,
                                          uint4& a, uint4& b) {
  const uint16_t* src = r.p + row * r.st + h * r.sh;
  a = *reinterpret_cast<const uint4*>(src + oa);
  b = *reinterpret_cast<const uint4*>(src + ob);
}

__device__ __forceinline__ void store_bf16(const CacheView& c, int64_t page, int slot, int h,
                                           int oa, int ob, const uint4& a, const uint4& b) {
  uint16_t* dst = reinterpret_cast<uint16_t*>(c.p) + page * c.s_page + slot * c.s_token +
                  h * c.s_head;
  *reinterpret_cast<uint4*>(dst + oa) = a;
  *reinterpret_cast<uint4*>(dst + ob) = b;
}

__device__ __forceinline__ void store_e4m3(const CacheView& c, int64_t page, int slot, int h,
                                           int oa, int ob, const uint4& a, const uint4& b,
                                           const ScaleOf& s) {
  uint8_t* dst = c.p + page * c.s_page + slot * c.s_token + h * c.s_head;
  *reinterpret_cast<uint2*>(dst + oa) = quantise8(a, s);
  *reinterpret_cast<uint2*>(dst + ob) = quantise8(b, s);
}

// ---------------------------------------------------------------------------
// few new tokens per sequence
// ---------------------------------------------------------------------------
template <int D, bool E4M3>
__global__ void __launch_bounds__(128) attn_append_few_kernel(const AppendParams p) {
  constexpr int L = D / 16;  // lanes of a group
  const int64_t g = (static_cast<int64_t>(blockIdx.x) * 128 + threadIdx.x) / L;
  const int c = threadIdx.x % L;
  const int lane = threadIdx.x & 31;
  const uint32_t mask = ((1u << L) - 1u) << (lane - c);
  const bool turned = 8 * c < p.rope.half;
  float cs[8], sn[8];
  const int64_t kv_work = static_cast<int64_t>(p.batch) * p.page_bound * 2 * p.hkv;
  if (g >= kv_work) {  // a query head of a token
    if (!p.q.p) return;
    const int64_t i = g - kv_work;
    const int64_t t = i / p.hq;
    const int h = static_cast<int>(i - t * p.hq);
    if (t >= p.total) return;
    const int b = find_segment(p.cu, p.batch, static_cast<int>(t));
    if (b < 0) return;
    int oa, ob;
    rope_offsets(p.rope, c, &oa, &ob);
    uint4 x, y;
    load_unit(p.q, t, h, oa, ob, x, y);
    const int pos = p.seqlens[b] - p.cu[b + 1] + static_cast<int>(t);
    if (turned) {
      rope_angles(p.rope, c, pos, cs, sn);
      rope_turn(p.rope, cs, sn, x, y);
    }
    uint16_t* dst = p.qo.p + t * p.qo.st + h * p.qo.sh;
    *reinterpret_cast<uint4*>(dst + oa) = x;
    *reinterpret_cast<uint4*>(dst + ob) = y;
    return;
  }
  int h = static_cast<int>(g % (2 * p.hkv));
  const int64_t bj = g / (2 * p.hkv);
  const int b = static_cast<int>(bj / p.page_bound), j = static_cast<int>(bj % p.page_bound);
  const PageSpan s = page_span(p, b, j);
  if (s.page < 0) return;
  const bool is_v = h >= p.hkv;
  if (is_v) h -= p.hkv;
  const RowsIn& in = is_v ? p.v : p.k;
  const CacheView& out = is_v ? p.vc : p.kc;
  const bool turn = turned && !is_v;
  int oa = 16 * c, ob = 16 * c + 8;
  if (!is_v) rope_offsets(p.rope, c, &oa, &ob);
  const int slot_mask = (1 << p.page_shift) - 1;

  auto row = [&](int pos, uint4& x, uint4& y) {
    load_unit(in, s.row0 + pos, h, oa, ob, x, y);
    if (turn) {
      rope_angles(p.rope, c, pos, cs, sn);
      rope_turn(p.rope, cs, sn, x, y);
    }
  };
  if constexpr (!E4M3) {
    for (int pos = s.first; pos < s.last; ++pos) {
      uint4 x, y;
      row(pos, x, y);
      store_bf16(out, s.page, pos & slot_mask, h, oa, ob, x, y);
    }
  } else {
    const int slot0 = s.first & slot_mask;
    float* scale = out.scale + static_cast<int64_t>(s.page) * p.hkv + h;
    const float old = *scale;
    uint32_t m = 0;
    uint4 x, y;
    for (int pos = s.first; pos < s.last; ++pos) {
      row(pos, x, y);
      m = max(m, finite_max_bits(x, y));
    }
#pragma unroll
    for (int o = 1; o < L; o <<= 1) m = max(m, __shfl_xor_sync(mask, m, o));
    float grow;
    const float now = next_scale(old, scale_exponent(m), slot0 == 0, &grow);
    const ScaleOf by = scale_of(now);
    const bool one = s.last - s.first == 1;  // x, y still hold it
    for (int pos = s.first; pos < s.last; ++pos) {
      if (!one) row(pos, x, y);
      store_e4m3(out, s.page, pos & slot_mask, h, oa, ob, x, y, by);
    }
    if (grow != 1.f) {
      uint8_t* base = out.p + s.page * out.s_page + h * out.s_head + 16 * c;
      constexpr int U = 16;  // rows in flight: one group moves the whole page
      for (int r = 0; r < slot0; r += U) {
        uint4 z[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (r + u < slot0) z[u] = *reinterpret_cast<uint4*>(base + (r + u) * out.s_token);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (r + u < slot0)
            *reinterpret_cast<uint4*>(base + (r + u) * out.s_token) = rescale16(z[u], grow);
      }
    }
    __syncwarp(mask);  // every lane has read the old scale
    if (c == 0) *scale = now;
  }
}

// ---------------------------------------------------------------------------
// many new tokens per sequence
// ---------------------------------------------------------------------------
// block: page_size * (D / 16) / IPT threads; grid: (batch * page_bound,
// kv_groups + query head groups)
// (two CTAs an SM instead of one at 79 registers: 104 -> 78 us for 16384 tokens)
template <int D, bool E4M3, int IPT>
__global__ void __launch_bounds__(512, IPT == 1 ? 2 : 1)
    attn_append_page_kernel(const AppendParams p) {
  constexpr int L = D / 16;
  __shared__ uint32_t amax[3][2];  // [head modulo 3][K, V]
  const int b = static_cast<int>(blockIdx.x / p.page_bound);
  const int j = static_cast<int>(blockIdx.x % p.page_bound);
  const PageSpan s = page_span(p, b, j);
  const bool queries = static_cast<int>(blockIdx.y) >= p.kv_groups;
  if (s.first >= s.last || (s.page < 0 && !queries)) return;  // uniform over the CTA
  const int c = threadIdx.x % L;
  const int rows_per_step = blockDim.x / L;
  const int slot_mask = (1 << p.page_shift) - 1;
  const bool turned = 8 * c < p.rope.half;
  int oa, ob;
  rope_offsets(p.rope, c, &oa, &ob);

  int pos[IPT];
  bool live[IPT];
  float cs[IPT][8], sn[IPT][8];
#pragma unroll
  for (int i = 0; i < IPT; ++i) {
    // slot of the page this item owns, in the page's order
    const int slot = i * rows_per_step + threadIdx.x / L;
    pos[i] = (s.first & ~slot_mask) + slot;
    live[i] = pos[i] >= s.first && pos[i] < s.last;
    if (live[i] && turned) rope_angles(p.rope, c, pos[i], cs[i], sn[i]);
  }

  if (queries) {
    const int h0 = (blockIdx.y - p.kv_groups) * p.q_heads_per_cta;
    const int h1 = min(h0 + p.q_heads_per_cta, p.hq);
#pragma unroll
    for (int i = 0; i < IPT; ++i) {
      if (!live[i]) continue;
      const int64_t t = s.row0 + pos[i];
      constexpr int U = 4;
      for (int h = h0; h < h1; h += U) {
        uint4 x[U], y[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (h + u < h1) load_unit(p.q, t, h + u, oa, ob, x[u], y[u]);
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (h + u < h1) {
            if (turned) rope_turn(p.rope, cs[i], sn[i], x[u], y[u]);
            uint16_t* dst = p.qo.p + t * p.qo.st + (h + u) * p.qo.sh;
            *reinterpret_cast<uint4*>(dst + oa) = x[u];
            *reinterpret_cast<uint4*>(dst + ob) = y[u];
          }
      }
    }
    return;
  }

  const int h0 = blockIdx.y * p.heads_per_cta;
  const int h1 = min(h0 + p.heads_per_cta, p.hkv);
  if constexpr (!E4M3) {
    for (int h = h0; h < h1; ++h) {
#pragma unroll
      for (int i = 0; i < IPT; ++i) {
        if (!live[i]) continue;
        uint4 x, y, z, w;
        load_unit(p.k, s.row0 + pos[i], h, oa, ob, x, y);
        load_unit(p.v, s.row0 + pos[i], h, 16 * c, 16 * c + 8, z, w);
        if (turned) rope_turn(p.rope, cs[i], sn[i], x, y);
        store_bf16(p.kc, s.page, pos[i] & slot_mask, h, oa, ob, x, y);
        store_bf16(p.vc, s.page, pos[i] & slot_mask, h, 16 * c, 16 * c + 8, z, w);
      }
    }
  } else {
    const int slot0 = s.first & slot_mask;
    if (threadIdx.x < 6) amax[threadIdx.x >> 1][threadIdx.x & 1] = 0;
    __syncthreads();
    for (int h = h0; h < h1; ++h) {
      const int at = (h - h0) % 3;
      uint4 x[IPT], y[IPT], z[IPT], w[IPT];
      uint32_t mk = 0, mv = 0;
      const int64_t si = static_cast<int64_t>(s.page) * p.hkv + h;
      const float old_k = p.kc.scale[si], old_v = p.vc.scale[si];
#pragma unroll
      for (int i = 0; i < IPT; ++i) {
        if (!live[i]) continue;
        load_unit(p.k, s.row0 + pos[i], h, oa, ob, x[i], y[i]);
        load_unit(p.v, s.row0 + pos[i], h, 16 * c, 16 * c + 8, z[i], w[i]);
      }
#pragma unroll
      for (int i = 0; i < IPT; ++i) {
        if (!live[i]) continue;
        if (turned) rope_turn(p.rope, cs[i], sn[i], x[i], y[i]);
        uint32_t a = abs_max_bits(x[i], y[i]), v = abs_max_bits(z[i], w[i]);
        if (a >= 0x7f80u) a = finite_max_bits(x[i], y[i]);
        if (v >= 0x7f80u) v = finite_max_bits(z[i], w[i]);
        mk = max(mk, a), mv = max(mv, v);
      }
      mk = __reduce_max_sync(0xffffffffu, mk);
      mv = __reduce_max_sync(0xffffffffu, mv);
      if ((threadIdx.x & 31) == 0) {
        atomicMax(&amax[at][0], mk);
        atomicMax(&amax[at][1], mv);
      }
      __syncthreads();  // the maxima of this head are complete, its old scales read
      float grow_k, grow_v;
      const float now_k = next_scale(old_k, scale_exponent(amax[at][0]), slot0 == 0, &grow_k);
      const float now_v = next_scale(old_v, scale_exponent(amax[at][1]), slot0 == 0, &grow_v);
      const ScaleOf by_k = scale_of(now_k), by_v = scale_of(now_v);
#pragma unroll
      for (int i = 0; i < IPT; ++i) {
        if (!live[i]) continue;
        const int slot = pos[i] & slot_mask;
        store_e4m3(p.kc, s.page, slot, h, oa, ob, x[i], y[i], by_k);
        store_e4m3(p.vc, s.page, slot, h, 16 * c, 16 * c + 8, z[i], w[i], by_v);
      }
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) {
        const float grow = kv ? grow_v : grow_k;
        const CacheView& out = kv ? p.vc : p.kc;
        if (grow == 1.f) continue;
        for (int r = threadIdx.x / L; r < slot0; r += rows_per_step) {
          uint4* q4 = reinterpret_cast<uint4*>(out.p + s.page * out.s_page + r * out.s_token +
                                               h * out.s_head + 16 * c);
          *q4 = rescale16(*q4, grow);
        }
      }
      if (threadIdx.x == 0) {
        p.kc.scale[si] = now_k;
        p.vc.scale[si] = now_v;
      }
      // the previous head's slots are free (all read them before this head's
      // barrier) and are written again two heads on, after the next barrier
      if (threadIdx.x < 2) amax[(at + 2) % 3][threadIdx.x] = 0;
    }
  }
}

}  // namespace attn
