// paged_tc.cuh -- attention over a paged cache for 9 (e4m3: 17) to 128 query rows of a
// group per CTA, on the tensor cores' tcgen05 path: drafts being verified, short
// chunks, wide groups.  The mma.sync kernel of paged_attn.cuh is bound by its matrix
// instructions and conversions there (32 rows 1.6 and 64 rows 4 times the time HBM
// needs for an e4m3 cache of head_dim 128).
//
//   S = Q K^T  (128 rows x 64 or 128 keys),  O += P V  (128 rows x head_dim)
//
// Tensor memory holds Q and P as first operands, S and O: P overwrites S.  Keys and
// values are the second operands in shared memory, in swizzled panels (K of 64 or 128
// bytes a key, K-major; V of 64 columns, MN-major).  bf16: both as they are.  e4m3: K's
// codes as they are (kind::f8f6f4), against Q as the sum of two e4m3 rows, which holds
// a bf16 exactly (to 2^-17 of the row's largest element); V converted to f16 (exact), since a weight needs f16's range and
// bits.  (With K converted too the conversions, at 3 to 4 cycles a pair and scheduler,
// set the pace.)
//
// The 128 rows are RT = 32, 64 or 128 query rows times KG = 4, 2 or 1 groups of
// the tile's keys: a thread of the softmax warps owns one lane, that is one row
// and BK / KG of the tile's BK keys, with an m, l and O of its own; it writes zeros
// as the weights of the other keys.  So the softmax needs no exchange between
// threads, all four warps work for few rows too, and the groups' parts are
// merged once at the end.  The MMAs multiply the zeros; they have the time.
//
// Warps 0-3: softmax.  Warps 4-7: V, converted to f16 (e4m3); keys outside the part
// cleared, and values that are not finite taken out of tiles where only some rows see
// the key.  Warp 8: the MMAs; S of tile t + 1 goes to the second slot while the softmax
// works on tile t.  Warp 9: the loads by TMA, one box per page and panel, three or four
// stages ahead.  (Four warps issuing cp.async took 1000 to 2000 cycles a tile.)
//
// What bounds it: a tile's chain.  Softmax of a tile about 1200 cycles for 32 keys a
// thread (its scheduler runs one softmax and one conversion warp), then 250 for the
// signal to the MMA warp, 150 + 540 for P V, 250 + 450 for S of the tile after the next,
// which needs the slot: about 1500 cycles a tile, whatever its size.  (head_dim 256: the
// 16 MMAs of 64 keys for S take about 50 cycles each, a full-rate one would take 16; with
// P V they fill 1400 of the 1500.)  P V from a warp of its own, or the zero weights
// written before the softmax, changed nothing.  One CTA alone, 32
// rows, 128K keys, e4m3: 5.7, 6.7 and 12.5 ns a key of head_dim 64, 128, 256; bf16 4.3,
// 5.9, 13.5; 148 of them with 4096 keys each, launch and drain included, 8.6, 11.2, 20.4
// and 8.9, 13.3, 24.2 (bf16 of head_dim 256: 6.3 TB/s).  More CTAs an SM (smaller tiles, one slot
// of S) gave 41 ns a key of 512 CTAs of e4m3 and head_dim 128, one CTA with these 38.
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
  static constexpr int ESZ = FP8 ? 1 : 2;
  static constexpr int BK = D == 256 ? 64 : 128;  // keys per tile
  static constexpr int RT = 128 / KG;        // query rows per CTA
  static constexpr int NC = BK / KG;         // keys per softmax thread and tile: 16 .. 128
  static constexpr int THREADS = 320;
  // K: panels of KROW bytes a key.  V in bf16 likewise; in e4m3 as codes [key][D], and
  // converted to f16 in two buffers of 64-column panels.
  static constexpr int KROW = D * ESZ < 128 ? 64 : 128;
  static constexpr int KPANEL = BK * KROW;
  static constexpr int VPANEL = BK * 128;
  static constexpr int HALF = BK * D * ESZ;  // K or V of a stage
  static constexpr int STAGE = 2 * HALF;
  static constexpr int STAGES = FP8 ? 4 : 3;
  static constexpr int NBUF = FP8 ? 2 : STAGES;  // tiles of V ready for the MMAs
  static constexpr int VBUF = FP8 ? BK * D * 2 : 0;
  static constexpr int VBUF_OFF = STAGES * STAGE;
  static constexpr int TILES_END = VBUF_OFF + (FP8 ? NBUF * VBUF : 0);
  // tensor memory: two slots of S, Q, O; 352, 448 or 512 columns
  static constexpr int Q_COL = 2 * BK, O_COL = 2 * BK + D / 2;
  static constexpr int TMEM_COLS = 512;
  // bits of a tile's values that are not finite, [NBUF][2 signs][keys][D / 32], and
  // of what each of the 128 lanes has seen
  static constexpr int WORDS = D / 32;
  static constexpr int OUT_ROW = 68;         // floats: a chunk of 64 columns of O at the end
  static constexpr int OUT = 128 * OUT_ROW * 4;
  static constexpr int BAR_OFF = TILES_END > OUT ? TILES_END : OUT;
  static constexpr int FLAG_OFF = BAR_OFF + 192;  // [NBUF][4] bytes of the V warps, abort, tmem
  static constexpr int ML_OFF = FLAG_OFF + 32;                 // [128] m, l
  static constexpr int BAD_OFF = ML_OFF + 128 * 8;             // [NBUF][2][BK][WORDS]
  static constexpr int SEEN_OFF = BAD_OFF + NBUF * 2 * BK * WORDS * 4;  // [2][128][WORDS]
  static constexpr int USED = SEEN_OFF + 2 * 128 * WORDS * 4 + 1024;  // 1024-byte alignment
  // one CTA an SM: a second one would wait for tensor memory
  static constexpr int SMEM = USED > 116 * 1024 ? USED : 116 * 1024;
  // the 128 threads of warps 4-7 take pieces of 16 bytes; a warp's are of whole keys, so
  // that what is noted of a key (BAD_OFF) belongs to one warp
  static constexpr int CPR = D * ESZ / 16;
  static_assert(32 % CPR == 0 && BK % (128 / CPR) == 0);
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

// columns, token, head, page of a pool
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint64_t* bar,
                                            int c0, int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// K-major operand of 64-byte rows with the 64-byte swizzle: 8-row atoms of 512 bytes
__device__ __forceinline__ uint64_t sdesc_sw64(uint32_t saddr, uint32_t sbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr >> 4) & 0x3FFFu);
  d |= static_cast<uint64_t>(1u) << 16;
  d |= static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32;
  d |= static_cast<uint64_t>(1u) << 46;  // descriptor version for SM100
  d |= static_cast<uint64_t>(4u) << 61;  // 64-byte swizzle
  return d;
}

// one arrival for a warp whose lanes have fenced what they wrote: 128 single arrivals
// on a barrier took about 800 cycles
__device__ __forceinline__ void tc_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
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
__global__ void __launch_bounds__(320, 1)
    attn_paged_tc_kernel(const __grid_constant__ CUtensorMap k_map,
                         const __grid_constant__ CUtensorMap v_map, const PagedTcParams tp) {
  using C = PagedTcCfg<D, FP8, KG>;
  constexpr int BK = C::BK, RT = C::RT, NC = C::NC, WORDS = C::WORDS, NBUF = C::NBUF,
                STAGES = C::STAGES;
  const PagedParams& p = tp.a;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + ((1024u - (raw & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  PagedPlace w{};
  // parts begin at whole pages, so that a tile is whole boxes of the tensor maps
  if (!w.find<D, RT, C::THREADS, 128>(p)) return;
  const int rows = w.rows, kb = w.kb, ke = w.ke;
  const int tiles = (ke - kb + BK - 1) / BK;

  uint64_t* landed = reinterpret_cast<uint64_t*>(smem + C::BAR_OFF);  // [STAGES] TMA is done
  uint64_t* left = landed + STAGES;  // [STAGES] the stage is free (bf16: P V is done)
  uint64_t* ready = left + STAGES;   // [NBUF] V is ready for the MMAs (bf16: K and V)
  uint64_t* used = ready + NBUF;     // [NBUF] e4m3: P V is done
  uint64_t* s_full = used + NBUF;    // [2] a slot holds S,
  uint64_t* p_full = s_full + 2;     // [2] or P
  int* tile_bad = reinterpret_cast<int*>(smem + C::FLAG_OFF);  // [NBUF], a byte of each V warp
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
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&landed[i], 1);
      mbar_init(&left[i], FP8 ? 5 : 1);  // e4m3: S is done, four warps have converted V
    }
    for (int i = 0; i < NBUF; ++i) {
      mbar_init(&ready[i], 4);
      mbar_init(&used[i], 1);
      tile_bad[i] = 0;
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
    }
    *abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_at;
  int issued = 0;  // warp 9: tiles whose loads were issued
  auto mixed = [&](int t) {  // some key of the tile is seen by some rows only
    return kb + t * BK < w.in_lo || min(kb + t * BK + BK, ke) > w.in_hi;
  };
  // P V of tile t is done
  auto wait_pv = [&](int t, uint32_t code) {
    return FP8 ? mbar_wait(&used[t % NBUF], (t / NBUF) & 1, abort, tp.err, code, tp.timeout_ns)
               : mbar_wait(&left[t % STAGES], (t / STAGES) & 1, abort, tp.err, code,
                           tp.timeout_ns);
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
        // 4 significant bits, then the rest; exact for elements down to 2^-2, which are those
        // down to 2^-9 of the largest, and smaller ones are off by at most half the least
        // code, 2^-17 of the largest
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
    // scales of this warp's blocks of 16 keys: lane 2 i (K), 2 i + 1 (V) has block i's,
    // of the next tile, and its page of the tile after that
    constexpr int BLOCKS = NC / 16;
    const int32_t* table = p.table + w.b * p.table_stride;
    const float* my_scale = ((lane & 1) ? p.vc.scale : p.kc.scale) + w.h;
    auto block_key = [&](int t) { return kb + t * BK + kg * NC + min(lane >> 1, BLOCKS - 1) * 16; };
    auto block_page = [&](int t) {
      return __ldg(table + (min(block_key(t), ke - 1) >> p.page_shift));
    };
    auto block_scale = [&](int t, uint32_t pg) {
      return block_key(t) < ke && pg < static_cast<uint32_t>(p.num_pages)
                 ? __ldg(my_scale + static_cast<int64_t>(pg) * p.hkv)
                 : 0.f;
    };
    float next_scale = 0.f;
    int next_page = 0;
    if constexpr (FP8) {
      next_scale = block_scale(0, block_page(0));
      next_page = block_page(1);
    }
    for (int t = 0; t < tiles; ++t) {
      const int b = t % NBUF;
      // even lanes: K's factor; odd lanes: log2 and inverse of V's scale.  (Pages outside
      // the pool have zeros: their keys count as x = 0 and V = 0.)
      const float scale = next_scale == 0.f ? 1.f : next_scale;
      const float log_or_k = (lane & 1) ? pg_lg2(scale) : scale, inverse = pg_rcp(scale);
      if constexpr (FP8) {
        next_scale = block_scale(t + 1, next_page);
        next_page = block_page(t + 2);
      }
      auto factor = [&](int g) {  // never 0: a masked score stays -inf
        return FP8 ? fmaxf(f_row * __shfl_sync(0xffffffffu, log_or_k, 2 * g), 1.2e-38f) : f_row;
      };
      auto log_scale = [&](int g) {
        return FP8 ? __shfl_sync(0xffffffffu, log_or_k, 2 * g + 1) : 0.f;
      };
      auto inverse_scale_of = [&](int g) {
        return FP8 ? __shfl_sync(0xffffffffu, inverse, 2 * g + 1) : 1.f;
      };
      if (!mbar_wait(&s_full[t & 1], (t >> 1) & 1, abort, tp.err, ERR_PAGED_SOFTMAX | 1,
                     tp.timeout_ns))
        ok = false;
      if (!__all_sync(0xffffffffu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t slot = lanes + (t & 1) * BK;
      uint32_t sr[NC];
      if constexpr (NC == 16)
        tmem_ld16(slot + kg * NC, sr);
      else if constexpr (NC == 32)
        tmem_ld32(slot + kg * NC, sr);
      else if constexpr (NC == 64)
        tmem_ld64(slot + kg * NC, sr);
      else
        tmem_ld128(slot, sr);
      const int key0 = kb + t * BK + kg * NC;
      const bool edge = mixed(t) || kb + t * BK + BK > ke;
      // (the common case runs without a branch between the blocks, so that their
      // instructions overlap: a warp has its scheduler almost to itself)
      if (capped) {
        // where no score of the warp is large, all by the polynomial, in pairs (not in
        // tiles with keys that are not seen: among those are some that were not loaded,
        // and what their memory happens to hold must not decide)
        float big = 0.f;
#pragma unroll
        for (int g = 0; g < NC / 16; ++g) {
          const float f = factor(g);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float x = __uint_as_float(sr[16 * g + i]) * f;
            big = fmaxf(big, fabsf(x));
            sr[16 * g + i] = __float_as_uint(x);
          }
        }
        const float ky = p.cap_mul * kCapY;
        if (!edge && __all_sync(0xffffffffu, big * ky <= tanhpoly::kY0)) {
          const uint64_t k2 = f2_pack(ky, ky);
#pragma unroll
          for (int i = 0; i < NC; i += 2) {
            const uint64_t x2 =
                f2_pack(__uint_as_float(sr[i]), __uint_as_float(sr[i + 1]));
            const uint64_t y2 = f2_mul(x2, k2), u2 = f2_mul(y2, y2);
            auto both = [](float a) { return f2_pack(a, a); };
            uint64_t r = f2_fma(both(tanhpoly::kA4), u2, both(tanhpoly::kA3));
            r = f2_fma(r, u2, both(tanhpoly::kA2));
            r = f2_fma(r, u2, both(tanhpoly::kA1));
            r = f2_fma(r, u2, both(tanhpoly::kA0));
            float a, b;
            f2_unpack(f2_mul(x2, r), a, b);
            sr[i] = __float_as_uint(a);
            sr[i + 1] = __float_as_uint(b);
          }
        } else {
#pragma unroll
          for (int i = 0; i < NC; ++i)
            sr[i] = __float_as_uint(pg_cap(__uint_as_float(sr[i]), p.cap_mul, p.cap_log2));
        }
      }
      if (edge) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          const int key = key0 + i;
          if (key < lo || key > hi) sr[i] = __float_as_uint(-INFINITY);
        }
      }
      float top = -INFINITY;
#pragma unroll
      for (int g = 0; g < NC / 16; ++g) {
        float v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i] = fmaxf(fmax3(__uint_as_float(sr[16 * g + i]), __uint_as_float(sr[16 * g + 4 + i]),
                             __uint_as_float(sr[16 * g + 8 + i])),
                       __uint_as_float(sr[16 * g + 12 + i]));
        top = fmaxf(top, __fmaf_rn(fmaxf(fmax3(v[0], v[1], v[2]), v[3]),
                                   capped ? 1.f : factor(g), log_scale(g)));
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
        // O may be changed when P V of the tile before is done
        if (t > 0 && !wait_pv(t - 1, ERR_PAGED_SOFTMAX | 2)) ok = false;
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (t > 0) {
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
        const float f = capped ? 1.f : factor(g), c = log_scale(g) - base;
        const uint64_t f2 = f2_pack(f, f), c2 = f2_pack(c, c);
        uint64_t sum = f2_pack(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          float x, y;
          f2_unpack(f2_fma(f2_pack(__uint_as_float(sr[16 * g + 2 * i]),
                                   __uint_as_float(sr[16 * g + 2 * i + 1])),
                           f2, c2),
                    x, y);
          x = pg_ex2(x);
          y = pg_ex2(y);
          sum = f2_add(sum, f2_pack(x, y));
          pw[8 * g + i] = FP8 ? pg_f16_pair(x, y) : bf16_pair(x, y);
        }
        float x, y;
        f2_unpack(sum, x, y);
        l = __fmaf_rn(x + y, inverse_scale_of(g), l);
      }
      // weights of this thread's keys, zeros for the other groups'
#pragma unroll
      for (int g = 0; g < KG; ++g) {
        if constexpr (NC == 16) {
          uint32_t x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
          if (g == kg)
            tmem_st8(slot + g * 8, pw);
          else
            tmem_st8(slot + g * 8, x);
        } else if constexpr (NC == 32) {
          uint32_t x[16] = {0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0};
          if (g == kg)
            tmem_st16(slot + g * 16, pw);
          else
            tmem_st16(slot + g * 16, x);
        } else {
#pragma unroll
          for (int h = 0; h < NC / 64; ++h) {
            uint32_t x[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = g == kg ? pw[32 * h + i] : 0u;
            tmem_st32(slot + g * (NC / 2) + h * 32, x);
          }
        }
      }
      tmem_st_wait();
      tc_fence_before();
      if (mixed(t)) {  // the values have been looked at
        ok = mbar_wait(&ready[b], (t / NBUF) & 1, abort, tp.err, ERR_PAGED_SOFTMAX | 3,
                       tp.timeout_ns);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
      }
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
            seen[tid * WORDS + i] |= bad[((b * 2 + 0) * BK + k) * WORDS + i];
            seen[(128 + tid) * WORDS + i] |= bad[((b * 2 + 1) * BK + k) * WORDS + i];
          }
        }
      }
      tc_arrive(&p_full[t & 1], lane);
    }
    const int last = tiles - 1;
    if (ok) ok = wait_pv(last, ERR_PAGED_SOFTMAX | 4);
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
      float* stage = reinterpret_cast<float*>(smem);  // [128][OUT_ROW]
      constexpr int SROW = C::OUT_ROW;
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
    // ---------------------------------------------------- V for the MMAs (bf16: checked)
    const int lt = tid - 128;
    constexpr int CPR = C::CPR;                // 16-byte pieces of a key's row
    constexpr int STEP = 128 / CPR;            // keys between a thread's pieces
    constexpr int N = BK / STEP;               // pieces of a thread and tile
    const int piece = lt % CPR, row0 = lt / CPR;
    // a tile with keys that only some rows see: values that are not finite are noted
    // and replaced by zeros, because a zero weight would not hide them.  Each warp clears
    // the words of its own keys (CPR | 32) and has a flag byte of its own: a barrier of
    // the four warps here could wait for one that has given up.
    uint8_t* flags = reinterpret_cast<uint8_t*>(tile_bad) + (warp - 4);  // of buffer b at 4 b
    auto clear_bad = [&](int b) {
      constexpr int KEYS = 32 / CPR;  // of a warp and step
      for (int i = lane; i < 2 * N * KEYS * WORDS; i += 32) {
        const int word = i % WORDS, k = i / WORDS % (N * KEYS), sign = i / (WORDS * N * KEYS);
        const int key = k / KEYS * STEP + (warp - 4) * KEYS + k % KEYS;
        bad[((b * 2 + sign) * BK + key) * WORDS + word] = 0;
      }
      if (lane == 0) flags[4 * b] = 0;
      __syncwarp();
    };
    auto clean = [&](int b, int key, int d0, uint32_t (&x)[4]) {  // 8 columns from d0
      uint32_t plus, minus;
      tc_clean<FP8>(x, &plus, &minus);
      if (plus | minus) {
        atomicOr(&bad[((b * 2 + 0) * BK + key) * WORDS + d0 / 32], plus << (d0 & 31));
        atomicOr(&bad[((b * 2 + 1) * BK + key) * WORDS + d0 / 32], minus << (d0 & 31));
        flags[4 * b] = 1;
      }
    };
    for (int t = 0; t < tiles; ++t) {
      const int b = t % NBUF, st = t % STAGES, key0 = kb + t * BK;
      bool ok = mbar_wait(&landed[st], (t / STAGES) & 1, abort, tp.err, ERR_PAGED_LOAD | 1,
                          tp.timeout_ns);
      if (FP8 && ok && t >= NBUF) ok = wait_pv(t - NBUF, ERR_PAGED_LOAD | 2);
      if (!__all_sync(0xffffffffu, ok)) break;
      const bool mix = mixed(t);
      const bool edge = key0 < w.klo || key0 + BK > ke;  // rows that are not this part's: zeros
      if (mix) clear_bad(b);
      uint8_t* codes = smem + st * C::STAGE + C::HALF;
      if constexpr (FP8) {
        const uint32_t vd = sbase + C::VBUF_OFF + b * C::VBUF + (piece >> 2) * C::VPANEL;
        // the two chunks of a piece; the lanes of an odd panel take them in the other
        // order, so that the 8 lanes of a store lie in different banks
        const int swap = (piece >> 2) & 1, c0 = 2 * (piece & 3) + swap;
        uint4 v[N];
#pragma unroll
        for (int i = 0; i < N; ++i)
          v[i] = *reinterpret_cast<const uint4*>(codes + (row0 + i * STEP) * D + piece * 16);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const int key = row0 + i * STEP;
          uint4 x = v[i];
          if (edge && (key0 + key < w.klo || key0 + key >= ke)) x = make_uint4(0, 0, 0, 0);
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
        fence_async_smem();
        tc_arrive(&ready[b], lane);
        if (lane == 0) mbar_arrive(&left[st]);
      } else {
        if (mix || edge) {
          for (int i = 0; i < N; ++i) {
            const int key = row0 + i * STEP;
            uint4* at = reinterpret_cast<uint4*>(codes + (piece >> 3) * C::VPANEL +
                                                 tc_chunk(key, piece & 7));
            const uint4 x = *at;
            uint32_t y[4] = {x.x, x.y, x.z, x.w};
            if (key0 + key < w.klo || key0 + key >= ke)
              y[0] = y[1] = y[2] = y[3] = 0;
            else if (mix)
              clean(b, key, piece * 8, y);
            *at = make_uint4(y[0], y[1], y[2], y[3]);
          }
          fence_async_smem();
        }
        tc_arrive(&ready[b], lane);
      }
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------------ loads
    const int tokens = min(1 << p.page_shift, BK), boxes = BK / tokens;  // of a tile: 1 .. 8
    const int32_t* table = p.table + w.b * p.table_stride;
    auto box_key = [&](int t) { return kb + t * BK + min(lane, boxes - 1) * tokens; };
    auto box_page = [&](int t) { return __ldg(table + (min(box_key(t), ke - 1) >> p.page_shift)); };
    int next_page = box_page(0);
    int t = 0;
    for (; t < tiles; ++t) {
      const int st = t % STAGES, page = next_page, key = box_key(t);
      next_page = box_page(t + 1);
      if (t >= STAGES && !mbar_wait_warp(&left[st], ((t / STAGES) + 1) & 1, abort, tp.err,
                                         ERR_PAGED_LOAD | 3, tp.timeout_ns))
        break;
      const bool live = lane < boxes && key < ke;
      const int n = __popc(__ballot_sync(0xffffffffu, live));
      if (lane == 0) mbar_expect_tx(&landed[st], n * tokens * D * C::ESZ * 2);
      __syncwarp();
      if (live) {
        const int slot = key & ((1 << p.page_shift) - 1);
        const uint32_t kd = sbase + st * C::STAGE + lane * tokens * C::KROW;
#pragma unroll
        for (int c = 0; c < C::HALF / C::KPANEL; ++c)
          tma_load_4d(kd + c * C::KPANEL, &k_map, &landed[st], c * (C::KROW / C::ESZ), slot, w.h,
                      page);
        if constexpr (FP8) {
          tma_load_4d(sbase + st * C::STAGE + C::HALF + lane * tokens * D, &v_map, &landed[st], 0,
                      slot, w.h, page);
        } else {
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(kd + C::HALF + c * C::VPANEL, &v_map, &landed[st], c * 64, slot, w.h, page);
        }
      }
      __syncwarp();
    }
    issued = t;
  } else {
    // ------------------------------------------------------------------- MMAs
    named_bar_sync(1, 160);
    tc_fence_after();
    const uint64_t kdesc = C::KROW == 64 ? sdesc_sw64(sbase, 512) : sdesc_sw128(sbase, 16, 1024);
    const uint64_t vdesc =
        sdesc_sw128(sbase + (FP8 ? C::VBUF_OFF : C::HALF), C::VPANEL, 1024);
    auto issue_s = [&](int t) {
      const int st = t % STAGES;
      const uint64_t kt = kdesc + static_cast<uint64_t>(st) * (C::STAGE >> 4);
      const uint32_t d = tmem + (t & 1) * BK;
      if (!mbar_wait_warp(FP8 ? &landed[st] : &ready[st], (t / STAGES) & 1, abort, tp.err,
                          ERR_PAGED_MMA | 1, tp.timeout_ns))
        return false;
      tc_fence_after();
      if constexpr (FP8) {
        constexpr int KS = D / 32;  // steps of 32 columns, for both parts of Q
#pragma unroll
        for (int k = 0; k < 2 * KS; ++k) {
          const int c = k % KS;
          mma_ts_f8(d, tmem + C::Q_COL + k * 8, kt + (c >> 2) * (C::KPANEL >> 4) + (c & 3) * 2,
                    C::IDESC_S, k != 0);
        }
      } else {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_ts(d, tmem + C::Q_COL + k * 8, kt + (k >> 2) * (C::KPANEL >> 4) + (k & 3) * 2,
                 C::IDESC_S, k != 0);
      }
      mma_commit(&s_full[t & 1]);
      if (FP8) mma_commit(&left[st]);
      return true;
    };
    bool ok = issue_s(0);
    for (int t = 0; ok && t < tiles; ++t) {
      const int b = t % NBUF;
      // S of the next tile while the softmax works on this one; its slot is free when
      // P V of the tile before has read P
      if (t + 1 < tiles) {
        ok = t == 0 || __all_sync(0xffffffffu, wait_pv(t - 1, ERR_PAGED_MMA | 2));
        if (!ok || !issue_s(t + 1)) break;
      }
      if (!mbar_wait_warp(&p_full[t & 1], (t >> 1) & 1, abort, tp.err, ERR_PAGED_MMA | 3,
                          tp.timeout_ns) ||
          (FP8 && !mbar_wait_warp(&ready[b], (t / NBUF) & 1, abort, tp.err, ERR_PAGED_MMA | 4,
                                  tp.timeout_ns)))
        break;
      tc_fence_after();
      const uint64_t vt = vdesc + static_cast<uint64_t>(b) * ((FP8 ? C::VBUF : C::STAGE) >> 4);
#pragma unroll
      for (int k = 0; k < BK / 16; ++k)
        mma_ts(tmem + C::O_COL, tmem + (t & 1) * BK + k * 8, vt + k * (16 * 128 >> 4), C::IDESC_O,
               (t | k) != 0);
      mma_commit(FP8 ? &used[b] : &left[b]);
    }
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  if (*abort) {
    // A CTA that gave up, in whichever warp: the copies and MMAs that were issued have to
    // end before its memory goes.  (Known here for all warps: the loads and the MMAs of
    // a warp that went through may still be under way when another one's wait ran out.)
    if (warp == 9)
      for (int u = max(0, issued - STAGES); u < issued; ++u)
        mbar_wait_drain(&landed[u % STAGES], (u / STAGES) & 1, tp.timeout_ns);
    if (warp == 8) {
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 100000) {  // 100 us, far above any tile's MMAs
      }
    }
  }
  if (warp == 8) tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace attn
