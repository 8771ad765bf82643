// paged_tc.cuh -- attention over a paged cache for 9 to 128 query rows of a group
// per CTA, on the tensor cores' tcgen05 path: drafts being verified, short chunks,
// wide groups.  The mma.sync kernel of paged_attn.cuh is bound by its matrix
// instructions and conversions there (16 rows 1.6, 64 rows 4 times the time HBM
// needs for an e4m3 cache of head_dim 128).
//
//   S = Q K^T  (128 rows x 64 keys),  O += P V  (128 rows x head_dim)
//
// Tensor memory holds Q and P as first operands, S and O: P overwrites S.  Keys and
// values are the second operands in shared memory, in panels of 64 keys x 128 bytes
// with the 128-byte swizzle, K as a K-major, V as an MN-major operand.  bf16: both as
// they are.  e4m3: K's codes as they are (kind::f8f6f4), against Q as the sum of two
// e4m3 rows, which holds a bf16 exactly; V converted to f16 (exact), since a weight
// needs f16's range and bits.  (With K converted too the conversions, at 3 to 4 cycles
// a pair and scheduler, set the pace: 44 ns a key of 512 CTAs of 32 rows.)
//
// The 128 rows are RT = 32, 64 or 128 query rows times KG = 4, 2 or 1 groups of
// the tile's keys: a thread of the softmax warps owns one lane, that is one row
// and 16, 32 or 64 of the 64 keys, with an m, l and O of its own; it writes zeros
// as the weights of the other keys.  So the softmax needs no exchange between
// threads, all four warps work for few rows too, and the groups' parts are
// merged once at the end.  The MMAs multiply the zeros: they have the time, as
// HBM needs 680 cycles for a tile (e4m3, head_dim 128) and the MMAs 256.
//
// Warps 0-3: softmax.  Warps 4-7: the loads by cp.async (bf16: straight into one of
// three buffers; e4m3: codes, which their thread converts into one of two buffers).  Warp 8: the MMAs.  S of tile t + 1 is
// issued when P V of tile t is done; a tile's chain S -> softmax -> P V takes
// about 700 cycles, and two CTAs share an SM (one at head_dim 256).
//
// The weights, m and l are as in paged_attn.cuh.  Every wait is bounded.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "paged_common.cuh"
#include "ptx.cuh"

namespace attn {

// device error word codes (kernel id << 8 | wait id)
enum : uint32_t {
  ERR_PAGED_LOAD = 0x1200,
  ERR_PAGED_MMA = 0x1300,
  ERR_PAGED_SOFTMAX = 0x1400,
};

struct PagedTcParams {
  PagedParams a;
  uint32_t* err;
  uint64_t timeout_ns;
};

template <int D, bool FP8, int KG>
struct PagedTcCfg {
  static constexpr int BK = 64;
  static constexpr int RT = 128 / KG;        // query rows per CTA
  static constexpr int NC = BK / KG;         // keys per softmax thread and tile
  static constexpr int THREADS = 288;
  static constexpr int PANEL = BK * 128;     // 64 keys x 64 columns of 2 bytes
  static constexpr int TILE = PANEL * (D / 64);  // V of a tile, or K in bf16
  // bf16: three buffers of K and V.  e4m3: two of V in f16, RAW tiles of V's codes on
  // their way, and K's codes in a ring that holds those and the two in use
  static constexpr int NBUF = FP8 ? 2 : 3;
  static constexpr int RAW = FP8 ? (D == 64 ? 4 : 2) : 0;
  static constexpr int RAW_TILE = FP8 ? BK * D + 32 : 0;  // codes of V, scales
  static constexpr int NK = FP8 ? RAW + 2 : NBUF;
  static constexpr int K_TILE = FP8 ? PANEL * (D > 128 ? 2 : 1) : TILE;  // 128 codes a row
  static constexpr int V_OFF = NK * K_TILE;
  static constexpr int RAW_OFF = V_OFF + NBUF * TILE;
  static constexpr int TILES_END = RAW_OFF + RAW * RAW_TILE;
  static constexpr int Q_COL = 64, O_COL = 64 + D / 2;  // S at column 0
  static constexpr int TMEM_COLS = D == 256 ? 512 : 256;
  static constexpr int CTAS = D == 256 || KG == 1 ? 1 : 2;  // (64 keys a thread need registers)
  // bits of a tile's values that are not finite, [NBUF][2 signs][64 keys][D / 32], and
  // of what each of the 128 lanes has seen
  static constexpr int WORDS = D / 32;
  static constexpr int STAGE_ROW = 68;       // floats: a chunk of 64 columns of O at the end
  static constexpr int STAGE = 128 * STAGE_ROW * 4;
  static constexpr int BAR_OFF = TILES_END > STAGE ? TILES_END : STAGE;
  static constexpr int SCALE_OFF = BAR_OFF + 128;              // [NBUF][4] float2
  static constexpr int FLAG_OFF = SCALE_OFF + NBUF * 32;       // [NBUF] ints, abort, tmem
  static constexpr int ML_OFF = FLAG_OFF + 32;                 // [128] m, l
  static constexpr int BAD_OFF = ML_OFF + 128 * 8;             // [NBUF][2][64][WORDS]
  static constexpr int SEEN_OFF = BAD_OFF + NBUF * 2 * 64 * WORDS * 4;  // [2][128][WORDS]
  static constexpr int USED = SEEN_OFF + 2 * 128 * WORDS * 4 + 1024;  // 1024-byte alignment
  // no third CTA on an SM: it would wait for tensor memory
  static constexpr int SMEM = USED > 80 * 1024 ? USED : 80 * 1024;
  static constexpr float OFFSET = FP8 ? 6.f : 0.f;
  static constexpr float RAISE = 8.f + OFFSET;
  static constexpr uint32_t FORMAT = FP8 ? ~((1u << 7) | (1u << 10)) : ~0u;  // f16: zeros
  // e4m3: S by kind::f8f6f4, whose formats are all 0 for e4m3
  static constexpr uint32_t IDESC_S = idesc_bf16(128, BK, false, false) & FORMAT;
  static constexpr uint32_t IDESC_O = idesc_bf16(128, D, false, true) & FORMAT;
};

// byte offset of chunk c (8 columns) of panel row `key` in a swizzled panel
__device__ __forceinline__ uint32_t tc_chunk(int key, int c) {
  return key * 128 + ((c ^ (key & 7)) << 4);
}
__device__ __forceinline__ void st_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                            uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// tcgen05.mma kind::f8f6f4, A (e4m3, four to a column) from tensor memory, B from shared
// memory, fp32 accumulation; executed like mma_ts
__device__ __forceinline__ void mma_ts_f8(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 2-byte values of a 16-byte chunk that are not finite: bits of columns (as +inf, -inf, both for
// NaN); they are replaced by zeros
template <bool FP8>
__device__ __forceinline__ void tc_clean(uint32_t (&w)[4], uint32_t* plus, uint32_t* minus) {
  constexpr uint32_t E = FP8 ? 0x7c00u : 0x7f80u, F = FP8 ? 0x03ffu : 0x007fu;
  *plus = *minus = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t v = (w[i >> 1] >> (16 * (i & 1))) & 0xffffu;
    if ((v & E) == E) {
      const bool nan = (v & F) != 0;
      if (nan || !(v & 0x8000u)) *plus |= 1u << i;
      if (nan || (v & 0x8000u)) *minus |= 1u << i;
      w[i >> 1] &= ~(0xffffu << (16 * (i & 1)));
    }
  }
}

template <int D, bool FP8, int KG>
__global__ void __launch_bounds__(288, PagedTcCfg<D, FP8, KG>::CTAS)
    attn_paged_tc_kernel(const PagedTcParams tp) {
  using C = PagedTcCfg<D, FP8, KG>;
  constexpr int BK = C::BK, RT = C::RT, NC = C::NC, WORDS = C::WORDS, NBUF = C::NBUF;
  const PagedParams& p = tp.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  PagedPlace w{};
  if (!w.find<D, RT, C::THREADS>(p)) return;
  const int rows = w.rows, kb = w.kb, ke = w.ke;
  const int tiles = (ke - kb + BK - 1) / BK;

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);  // [NBUF] it is written
  uint64_t* empty = full + NBUF;                                    // [NBUF] its P V is done
  uint64_t* s_full = full + 2 * NBUF;
  uint64_t* p_full = full + 2 * NBUF + 1;
  float2* scales = reinterpret_cast<float2*>(smem + C::SCALE_OFF);
  int* tile_bad = reinterpret_cast<int*>(smem + C::FLAG_OFF);       // [NBUF]
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::FLAG_OFF + 16);
  uint32_t* tmem_at = reinterpret_cast<uint32_t*>(smem + C::FLAG_OFF + 20);
  float2* ml = reinterpret_cast<float2*>(smem + C::ML_OFF);
  uint32_t* bad = reinterpret_cast<uint32_t*>(smem + C::BAD_OFF);
  uint32_t* seen = reinterpret_cast<uint32_t*>(smem + C::SEEN_OFF);

  if (warp == 8) {
    tmem_alloc(tmem_at, C::TMEM_COLS);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(&full[i], 128);
      mbar_init(&empty[i], 1);
      tile_bad[i] = 0;
    }
    mbar_init(s_full, 1);
    mbar_init(p_full, 128);
    *abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  auto mixed = [&](int t) {  // some key of the tile is seen by some rows only
    return kb + t * BK < w.in_lo || min(kb + t * BK + BK, ke) > w.in_hi;
  };

  if (warp < 4) {
    // ---------------------------------------------------------------- softmax
    const int kg = KG == 4 ? warp : KG == 2 ? warp >> 1 : 0;
    const int r = KG == 4 ? lane : KG == 2 ? (warp & 1) * 32 + lane : tid;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    // this row of Q into tensor memory, scaled as in paged_queries
    float f_row = p.scale_log2;
    int lo, hi;
    {
      const bool live = r < rows;
      const uint4* src =
          reinterpret_cast<const uint4*>(p.q + w.row_index(p, live ? r : 0) * D);
      if constexpr (FP8) {
        // scaled so that the largest element is in [2^7, 2^8), and as a sum of two codes:
        // 4 significant bits, then the rest; exact for elements down to 2^-10 of that
        uint32_t m = 0;
#pragma unroll 8
        for (int i = 0; i < D / 8; ++i) {
          const uint4 x = src[i];
          constexpr uint32_t M = 0x7fff7fffu;
          const uint32_t v = __vmaxu2(__vmaxu2(x.x & M, x.y & M), __vmaxu2(x.z & M, x.w & M));
          m = max(m, max(v & 0xffffu, v >> 16));
        }
        const int e = m >= 0x7f80u ? 7 : max(static_cast<int>(m >> 7) - 127, -100);
        const float up = exp2_int(7 - e);
        f_row *= exp2_int(e - 7);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {  // 32 elements: 8 columns of each part
          uint32_t hi8[8], lo8[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 x = src[c * 4 + i];
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float v[4] = {bf16_lo(y[2 * k]) * up, bf16_hi(y[2 * k]) * up,
                                  bf16_lo(y[2 * k + 1]) * up, bf16_hi(y[2 * k + 1]) * up};
              const uint32_t h = e4m3_pair(v[0], v[1]) | (e4m3_pair(v[2], v[3]) << 16);
              const uint32_t h01 = pg_f16_lo(h), h23 = pg_f16_hi(h);
              const uint32_t g =
                  e4m3_pair(v[0] - pg_weight<true>(h01), v[1] - pg_weight<true>(h01 >> 16)) |
                  (e4m3_pair(v[2] - pg_weight<true>(h23), v[3] - pg_weight<true>(h23 >> 16)) << 16);
              hi8[2 * i + k] = live ? h : 0u;
              lo8[2 * i + k] = live ? g : 0u;
            }
          }
          tmem_st8(lanes + C::Q_COL + c * 8, hi8);
          tmem_st8(lanes + C::Q_COL + D / 4 + c * 8, lo8);
        }
      } else {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {  // 16 columns of tensor memory: 32 elements
          uint32_t q[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 x = src[c * 4 + i];
            q[4 * i] = live ? x.x : 0u;
            q[4 * i + 1] = live ? x.y : 0u;
            q[4 * i + 2] = live ? x.z : 0u;
            q[4 * i + 3] = live ? x.w : 0u;
          }
          tmem_st16(lanes + C::Q_COL + c * 16, q);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      const int i = (w.r0 + min(r, rows - 1)) / p.group;
      lo = w.row_lo(p, i);
      hi = min(w.row_hi(p, i), ke - 1);
    }
    named_bar_sync(1, 160);  // Q is there for the MMA warp
    const bool capped = p.cap_log2 > 0.f;
    float m = -INFINITY, l = 0.f;
    bool poisoned = false;
    bool ok = true;
    for (int t = 0; t < tiles; ++t) {
      const int b = t % NBUF;
      if (!mbar_wait(&full[b], (t / NBUF) & 1, abort, tp.err, ERR_PAGED_SOFTMAX | 1,
                     tp.timeout_ns) ||
          !mbar_wait(s_full, t & 1, abort, tp.err, ERR_PAGED_SOFTMAX | 2, tp.timeout_ns))
        ok = false;
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      uint32_t sr[NC];
      if constexpr (NC == 16)
        tmem_ld16(lanes + kg * NC, sr);
      else if constexpr (NC == 32)
        tmem_ld32(lanes + kg * NC, sr);
      else
        tmem_ld64(lanes, sr);
      const int key0 = kb + t * BK + kg * NC;
      const bool edge = mixed(t) || kb + t * BK + BK > ke;
      float top = -INFINITY;
#pragma unroll
      for (int g = 0; g < NC / 16; ++g) {
        PagedScales sc;
        if constexpr (FP8) sc = PagedScales(scales[b * 4 + kg * (NC / 16) + g]);
        float f = fmaxf(f_row * sc.ks, 1.2e-38f);
        if (capped) {
#pragma unroll
          for (int i = 0; i < 16; ++i)
            sr[16 * g + i] = __float_as_uint(
                pg_cap(__uint_as_float(sr[16 * g + i]) * f * p.cap_mul, p.cap_log2));
          f = 1.f;
        }
        if (edge) {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int key = key0 + 16 * g + i;
            if (key < lo || key > hi) sr[16 * g + i] = 0xff800000u;  // -inf
          }
        }
        float v = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; i += 2)
          v = fmax3(v, __uint_as_float(sr[16 * g + i]), __uint_as_float(sr[16 * g + i + 1]));
        top = fmaxf(top, __fmaf_rn(v, f, sc.lv));
      }
      const bool raise = top > m + C::RAISE;
      if (__any_sync(0xffffffffu, raise)) {
        float a = 1.f;
        if (raise) {
          const float to = top - C::OFFSET;
          a = m == -INFINITY ? 0.f : pg_ex2(m - to);
          l *= a;
          m = to;
        }
        if (t > 0) {  // P V of the tile before is done, or S would not be there
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            uint32_t o[32];
            tmem_ld32(lanes + C::O_COL + c, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
            tmem_st32(lanes + C::O_COL + c, o);
          }
        }
      }
      const float base = m == -INFINITY ? 0.f : m;
      uint32_t pw[NC / 2];
#pragma unroll
      for (int g = 0; g < NC / 16; ++g) {
        PagedScales sc;
        if constexpr (FP8) sc = PagedScales(scales[b * 4 + kg * (NC / 16) + g]);
        const float f = capped ? 1.f : fmaxf(f_row * sc.ks, 1.2e-38f);
        const float c = sc.lv - base;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = pg_ex2(__fmaf_rn(__uint_as_float(sr[16 * g + 2 * i]), f, c));
          const float y = pg_ex2(__fmaf_rn(__uint_as_float(sr[16 * g + 2 * i + 1]), f, c));
          sum += x + y;
          pw[8 * g + i] = FP8 ? pg_f16_pair(x, y) : bf16_pair(x, y);
        }
        l = __fmaf_rn(sum, sc.iv, l);
      }
      // weights of this thread's keys, zeros for the other groups'
#pragma unroll
      for (int g = 0; g < KG; ++g) {
        if constexpr (NC == 16) {
          uint32_t x[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) x[i] = g == kg ? pw[i] : 0u;
          tmem_st8(lanes + g * 8, x);
        } else if constexpr (NC == 32) {
          uint32_t x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = g == kg ? pw[i] : 0u;
          tmem_st16(lanes + g * 16, x);
        } else {
          tmem_st32(lanes, pw);
        }
      }
      tmem_st_wait();
      tc_fence_before();
      if (mixed(t) && tile_bad[b]) {
        // values that are not finite, taken out of the tile: noted for the rows that see them
        if (!poisoned) {
          for (int i = 0; i < WORDS; ++i) seen[tid * WORDS + i] = seen[(128 + tid) * WORDS + i] = 0;
          poisoned = true;
        }
        for (int k = kg * NC; k < kg * NC + NC; ++k) {
          const int key = kb + t * BK + k;
          if (key < lo || key > hi) continue;
          for (int i = 0; i < WORDS; ++i) {
            seen[tid * WORDS + i] |= bad[((b * 2 + 0) * 64 + k) * WORDS + i];
            seen[(128 + tid) * WORDS + i] |= bad[((b * 2 + 1) * 64 + k) * WORDS + i];
          }
        }
      }
      mbar_arrive(p_full);
    }
    const int last = tiles - 1;
    if (ok) ok = mbar_wait(&empty[last % NBUF], (last / NBUF) & 1, abort, tp.err,
                           ERR_PAGED_SOFTMAX | 3, tp.timeout_ns);
    // O of the groups of a row, merged: in chunks of 64 columns through shared memory
    // (the buffers are free)
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    ml[tid] = make_float2(m, l);
    if (!poisoned) {
      for (int i = 0; i < WORDS; ++i) seen[tid * WORDS + i] = seen[(128 + tid) * WORDS + i] = 0;
    }
    named_bar_sync(2, 128);
    if (!*abort) {  // the same for the four warps: set before the barrier, or by none of them
      float top = -INFINITY, sum = 0.f;
#pragma unroll
      for (int g = 0; g < KG; ++g) top = fmaxf(top, ml[g * RT + r].x);
      const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int g = 0; g < KG; ++g) {
        const float2 x = ml[g * RT + r];
        sum += pg_ex2(x.x - base) * x.y;
      }
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      const float mine = pg_ex2(m - base) * inv;
      const float l2 = sum == 0.f ? -INFINITY : base + pg_lg2(sum);
      if (kg == 0 && r < rows) {
        if (p.num_splits > 1)
          p.part_lse[static_cast<int64_t>(w.split) * p.total_q * p.hq + w.row_index(p, r)] = l2;
        else if (p.lse)
          w.store_lse(p, r, l2);
      }
      float* stage = reinterpret_cast<float*>(smem);  // [128][STAGE_ROW]
      constexpr int SROW = C::STAGE_ROW;
#pragma unroll 1
      for (int c = 0; c < D; c += 64) {
#pragma unroll
        for (int hlf = 0; hlf < 2; ++hlf) {
          uint32_t o[32];
          tmem_ld32(lanes + C::O_COL + c + hlf * 32, o);
          float4* dst = reinterpret_cast<float4*>(stage + tid * SROW + hlf * 32);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            dst[i] = make_float4(
                __uint_as_float(o[4 * i]) * mine, __uint_as_float(o[4 * i + 1]) * mine,
                __uint_as_float(o[4 * i + 2]) * mine, __uint_as_float(o[4 * i + 3]) * mine);
        }
        named_bar_sync(2, 128);
        for (int x = tid; x < rows * 16; x += 128) {
          const int row = x >> 4, q4 = (x & 15) * 4;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          uint32_t plus = 0, minus = 0;
#pragma unroll
          for (int g = 0; g < KG; ++g) {
            const float4 y = *reinterpret_cast<const float4*>(stage + (g * RT + row) * SROW + q4);
            v.x += y.x, v.y += y.y, v.z += y.z, v.w += y.w;
            const int word = (g * RT + row) * WORDS + (c + q4) / 32;
            plus |= seen[word] >> ((c + q4) & 31);
            minus |= seen[128 * WORDS + word] >> ((c + q4) & 31);
          }
          if ((plus | minus) & 15u) {
            auto mark = [&](int i, float y) {
              if ((plus >> i) & (minus >> i) & 1u) return __uint_as_float(0x7fffffffu);
              if ((plus >> i) & 1u) return y + INFINITY;
              if ((minus >> i) & 1u) return y - INFINITY;
              return y;
            };
            v = make_float4(mark(0, v.x), mark(1, v.y), mark(2, v.z), mark(3, v.w));
          }
          const int64_t g = w.row_index(p, row);
          if (p.num_splits > 1)
            *reinterpret_cast<float4*>(
                p.part_o + (static_cast<int64_t>(w.split) * p.total_q * p.hq + g) * D + c + q4) = v;
          else
            *reinterpret_cast<uint2*>(p.out + g * D + c + q4) =
                make_uint2(bf16_pair(v.x, v.y), bf16_pair(v.z, v.w));
        }
        named_bar_sync(2, 128);
      }
    }
    tc_fence_before();
  } else if (warp < 8) {
    // ------------------------------------------------------------------ loads
    const int lt = tid - 128;
    constexpr int ESZ = FP8 ? 1 : 2;
    constexpr int CPR = D * ESZ / 16;          // 16-byte pieces of a cached row
    constexpr int STEP = 128 / CPR;            // rows between a thread's pieces
    constexpr int N = BK / STEP;               // pieces of K (and of V) per thread and tile
    const int piece = lt % CPR, row0 = lt / CPR;
    const uint8_t* kbase = p.kc.p + p.kc.s_head * ESZ * w.h + piece * 16;
    const uint8_t* vbase = p.vc.p + p.vc.s_head * ESZ * w.h + piece * 16;
    const int32_t* table = p.table + w.b * p.table_stride;
    const int slot_mask = (1 << p.page_shift) - 1, last_entry = (ke - 1) >> p.page_shift;
    const uint32_t spread = ke - w.klo;
    int page[N];
    auto find_pages = [&](int t) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        page[i] = __ldg(table + min((kb + t * BK + row0 + i * STEP) >> p.page_shift, last_entry));
    };
    // a piece's place in the pools; false: zeros
    auto source = [&](int t, int i, uint64_t* ko, uint64_t* vo) {
      const int key = kb + t * BK + row0 + i * STEP;
      const uint32_t pg = page[i];
      const bool live = static_cast<uint32_t>(key - w.klo) < spread &&
                        pg < static_cast<uint32_t>(p.num_pages);
      const uint32_t slot = key & slot_mask;
      *ko = static_cast<uint64_t>(live ? pg : 0u) * p.k_page + static_cast<uint64_t>(slot) * p.k_token;
      *vo = static_cast<uint64_t>(live ? pg : 0u) * p.v_page + static_cast<uint64_t>(slot) * p.v_token;
      return live;
    };
    // a tile with keys that only some rows see: values that are not finite are noted
    // and replaced by zeros, because a zero weight would not hide them
    auto clear_bad = [&](int b) {
      for (int i = lt; i < 2 * 64 * WORDS; i += 128) bad[b * 2 * 64 * WORDS + i] = 0;
      if (lt == 0) tile_bad[b] = 0;
      named_bar_sync(3, 128);
    };
    auto clean = [&](int b, int key, int d0, uint32_t (&x)[4]) {  // 8 columns from d0
      uint32_t plus, minus;
      tc_clean<FP8>(x, &plus, &minus);
      if (plus | minus) {
        atomicOr(&bad[((b * 2 + 0) * 64 + key) * WORDS + d0 / 32], plus << (d0 & 31));
        atomicOr(&bad[((b * 2 + 1) * 64 + key) * WORDS + d0 / 32], minus << (d0 & 31));
        tile_bad[b] = 1;
      }
      return (plus | minus) != 0;
    };
    auto wait_empty = [&](int t) {
      bool ok = t < NBUF || mbar_wait(&empty[t % NBUF], ((t / NBUF) + 1) & 1, abort, tp.err,
                                   ERR_PAGED_LOAD | 1, tp.timeout_ns);
      return __all_sync(0xffffffffu, ok) != 0;
    };
    if constexpr (FP8) {
      // A thread converts the codes that it loaded itself, so it waits for its own
      // copies only; they lie [piece][thread], every access in different banks.
      const uint32_t mine = sbase + C::RAW_OFF + lt * 16;
      auto issue = [&](int t) {
        const uint32_t st = mine + (t % C::RAW) * C::RAW_TILE;
        const uint32_t kd = sbase + (t % C::NK) * C::K_TILE + (piece >> 3) * C::PANEL;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          uint64_t ko, vo;
          const bool live = source(t, i, &ko, &vo);
          pg_cp16(kd + tc_chunk(row0 + i * STEP, piece & 7), kbase + ko, live);
          pg_cp16(st + i * 2048, vbase + vo, live);
        }
        if (lt < 8) {  // scales of the tile's four 16-key blocks
          const int key = kb + t * BK + (lt >> 1) * 16;
          const uint32_t pg = __ldg(table + min(key >> p.page_shift, last_entry));
          const bool live = key < ke && pg < static_cast<uint32_t>(p.num_pages);
          pg_cp4(sbase + C::RAW_OFF + (t % C::RAW) * C::RAW_TILE + BK * D + lt * 4,
                 ((lt & 1) ? p.vc.scale : p.kc.scale) +
                     static_cast<int64_t>(live ? pg : 0u) * p.hkv + w.h,
                 live);
        }
      };
      find_pages(0);
#pragma unroll 1
      for (int t = 0; t < C::RAW; ++t) {
        if (t < tiles) issue(t);
        pg_commit();
        find_pages(t + 1);  // (past the last tile: the last entry again)
      }
      for (int t = 0; t < tiles; ++t) {
        const int b = t % NBUF;
        pg_wait<C::RAW - 1>();
        if (!wait_empty(t)) break;
        const bool mix = mixed(t);
        if (mix) clear_bad(b);
        const uint8_t* codes = smem + C::RAW_OFF + (t % C::RAW) * C::RAW_TILE;
        const uint32_t vd = sbase + C::V_OFF + b * C::TILE + (piece >> 2) * C::PANEL;
        // the two chunks of a piece; the lanes of an odd panel take them in the other
        // order, so that the 8 lanes of a store lie in different banks
        const int swap = (piece >> 2) & 1, c0 = 2 * (piece & 3) + swap;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int key = row0 + i * STEP;
          const uint4 x = *reinterpret_cast<const uint4*>(codes + i * 2048 + lt * 16);
          const uint32_t w0 = swap ? x.z : x.x, w1 = swap ? x.w : x.y;
          const uint32_t w2 = swap ? x.x : x.z, w3 = swap ? x.y : x.w;
          uint32_t first[4] = {pg_f16_lo(w0), pg_f16_hi(w0), pg_f16_lo(w1), pg_f16_hi(w1)};
          uint32_t second[4] = {pg_f16_lo(w2), pg_f16_hi(w2), pg_f16_lo(w3), pg_f16_hi(w3)};
          if (mix) {
            clean(b, key, piece * 16 + 8 * swap, first);
            clean(b, key, piece * 16 + 8 - 8 * swap, second);
          }
          st_shared16(vd + tc_chunk(key, c0), first[0], first[1], first[2], first[3]);
          st_shared16(vd + tc_chunk(key, c0 ^ 1), second[0], second[1], second[2], second[3]);
        }
        if (lt < 8)
          reinterpret_cast<float*>(scales + b * 4)[lt] =
              reinterpret_cast<const float*>(codes + BK * D)[lt];
        fence_async_smem();
        mbar_arrive(&full[b]);
        if (t + C::RAW < tiles) issue(t + C::RAW);
        pg_commit();
        find_pages(t + C::RAW + 1);
      }
      pg_wait<0>();
    } else {
      // two tiles are on their way while one is handed over and used
      auto issue = [&](int t) {
        const int b = t % NBUF;
        const uint32_t kd = sbase + b * C::TILE + (piece >> 3) * C::PANEL;
#pragma unroll
        for (int i = 0; i < N; ++i) {
          uint64_t ko, vo;
          const bool live = source(t, i, &ko, &vo);
          const uint32_t o = tc_chunk(row0 + i * STEP, piece & 7);
          pg_cp16(kd + o, kbase + ko, live);
          pg_cp16(kd + C::V_OFF + o, vbase + vo, live);
        }
      };
      find_pages(0);
#pragma unroll 1
      for (int t = 0; t < NBUF - 1; ++t) {
        if (t < tiles) issue(t);
        pg_commit();
        find_pages(t + 1);
      }
      for (int t = 0; t < tiles; ++t) {
        const int b = t % NBUF;
        pg_wait<NBUF - 2>();
        if (mixed(t)) {
          clear_bad(b);
          const uint32_t vd = sbase + C::V_OFF + b * C::TILE + (piece >> 3) * C::PANEL;
          for (int i = 0; i < N; ++i) {
            const int key = row0 + i * STEP;
            uint4* at = reinterpret_cast<uint4*>(smem + (vd - sbase) + tc_chunk(key, piece & 7));
            const uint4 x = *at;
            uint32_t y[4] = {x.x, x.y, x.z, x.w};
            if (clean(b, key, piece * 8, y)) *at = make_uint4(y[0], y[1], y[2], y[3]);
          }
        }
        fence_async_smem();
        mbar_arrive(&full[b]);
        if (t + NBUF - 1 < tiles) {
          if (!wait_empty(t + NBUF - 1)) break;
          issue(t + NBUF - 1);
        }
        pg_commit();
        find_pages(t + NBUF);
      }
      pg_wait<0>();
    }
  } else {
    // ------------------------------------------------------------------- MMAs
    named_bar_sync(1, 160);
    tc_fence_after();
    const uint64_t kdesc = sdesc_sw128(sbase, 16, 1024);
    const uint64_t vdesc = sdesc_sw128(sbase + C::V_OFF, C::PANEL, 1024);
    for (int t = 0; t < tiles; ++t) {
      const int b = t % NBUF;
      const uint64_t kt = kdesc + static_cast<uint64_t>(t % C::NK) * (C::K_TILE >> 4);
      const uint64_t vt = vdesc + static_cast<uint64_t>(b) * (C::TILE >> 4);
      // the tile is there; S is free: P V of the tile before has read P
      if (!mbar_wait_warp(&full[b], (t / NBUF) & 1, abort, tp.err, ERR_PAGED_MMA | 1,
                          tp.timeout_ns))
        break;
      if (t > 0 && !mbar_wait_warp(&empty[(t - 1) % NBUF], ((t - 1) / NBUF) & 1, abort, tp.err,
                                   ERR_PAGED_MMA | 2, tp.timeout_ns))
        break;
      tc_fence_after();
      if constexpr (FP8) {
#pragma unroll
        for (int k = 0; k < 2 * (D / 32); ++k) {  // both parts of Q, 32 columns of the head each
          const int c = k % (D / 32);
          mma_ts_f8(tmem, tmem + C::Q_COL + k * 8, kt + (c >> 2) * (C::PANEL >> 4) + (c & 3) * 2,
                    C::IDESC_S, k != 0);
        }
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ts(tmem, tmem + C::Q_COL + k * 8, kt + (k >> 2) * (C::PANEL >> 4) + (k & 3) * 2,
                 C::IDESC_S, k != 0);
      }
      mma_commit(s_full);
      if (!mbar_wait_warp(p_full, t & 1, abort, tp.err, ERR_PAGED_MMA | 3, tp.timeout_ns)) break;
      tc_fence_after();
#pragma unroll
      for (int k = 0; k < BK / 16; ++k)
        mma_ts(tmem + C::O_COL, tmem + k * 8, vt + k * (16 * 128 >> 4), C::IDESC_O,
               (t | k) != 0);
      mma_commit(&empty[b]);
    }
    // a CTA that gave up: what was issued has to end before its memory goes
    if (*abort) {
      mma_commit(s_full);
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 100000) {  // 100 us, far above any tile's MMAs
      }
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace attn
