// paged_attn.cuh -- attention of up to 8 query rows of a group per sequence (a
// decoding step, or a few rows of a small group), 16 in e4m3, over a paged key/value
// cache in bf16 or e4m3 (one scale per page and key/value head).
//
//   x_j = log2(e) scale (q . Kcode_j) kscale_j        (then softcap and mask)
//   l = sum_j 2^(x_j - m),   O = sum_j 2^(x_j - m) vscale_j Vcode_j / l
//
// Bound by HBM for up to 8 rows: each code is read once and does 8 multiply-adds, far
// under the tensor cores' ridge.  So the design feeds the loads: cp.async fills tiles of
// 64 or 128 keys, and two or three CTAs share an SM.
//
// The products run transposed, on mma.m16n8k16: S^T = K Q^T with 16 keys as the
// matrix rows and the 8 query rows as its columns, O^T = V^T P^T with 16 columns
// of the head as rows.  The cache is then always the 16-row operand, and a
// decoding step of 4 or 8 heads wastes little.  (tcgen05 works on 128-row tiles
// with both operands in their final type in shared memory: nothing to gain while
// HBM sets the pace.)  Each of the four warps takes a quarter of a tile's keys
// and keeps its own m, l and O, merged once at the end through shared memory.
//
// e4m3: codes become f16 (exact) in registers, 2 at a time.  K: the 4 bytes a
// thread gets from ldmatrix are 4 neighbouring head columns, used as columns
// 2q, 2q+1 and 2q+8, 2q+9 of the MMA; Q is laid out in the same order.  V:
// ldmatrix.trans moves pairs of bytes, so a thread gets two head columns of two
// keys; one byte permute separates them and they become rows r and r + 8.
// (Measured: 3 to 4 cycles a conversion and scheduler, about 260 cycles per 16
// keys of 128 columns of K and V, when HBM delivers them in 680.)
// P carries the V scale: w_j = 2^(x_j - m) vscale_j, where m follows the
// largest x_j + log2 vscale_j, so f16 holds the weights that matter whatever the
// spread of the scales.  m is kept 6 below the maximum (w up to 2^15) so that
// f16's subnormals begin 2^20 below it.  m is raised only when exceeded by 2^8;
// any m gives the same quotient, and the sum l is taken in fp32 before rounding.
// bf16: operands as they are, P rounded to bf16.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "paged_common.cuh"

namespace attn {

template <int D, bool FP8, int NT>
struct PagedCfg {
  static constexpr int ESZ = FP8 ? 1 : 2;
  static constexpr int ROWB = D * ESZ;       // bytes of a cached row
  static constexpr int CPR = ROWB / 16;      // 16-byte pieces of it
  static constexpr int THREADS = 128;
  static constexpr int WK = 4;               // warps, along a tile's keys
  // Tiles and stages measured on 16 sequences of 64K (e4m3, head_dim 128): 128
  // keys x 2 stages 351 us, 128 x 3 382, 64 x 4 381: a third CTA on an SM (64 KB
  // each) beats deeper stages.  Rows of 256 bytes: 64 x 2 334 us against 64 x 3
  // 341 and 64 x 4 494 (128 ragged sequences in bf16).  Rows of 64 bytes: 3
  // stages 91 us, 2 stages 93.
  static constexpr int BK = ROWB <= 128 ? 128 : 64;  // keys per tile
  static constexpr int KW = BK / WK / 16;    // 16-key blocks per warp and tile;
  // so many at once: 2 for 8 rows (327 us against 341 with one; 64-byte rows are
  // faster with one), all of up to 4 for more
  static constexpr int KT_MOST = NT > 1 ? 4 : ROWB == 64 ? 1 : 2;
  static constexpr int KT = KW < KT_MOST ? KW : KT_MOST;
  static constexpr int RT = 8 * NT;          // query rows per CTA
  static constexpr int TILE = BK * ROWB;
  static constexpr int STAGES = ROWB == 64 ? 3 : 2;
  static constexpr int STAGE = 2 * TILE + 2 * (BK / 16) * 4;  // K, V, their scales
  static constexpr int QROW = D + 8;         // padded, in elements
  static constexpr int OROW = D + 4;
  static constexpr int Q_OFF = STAGES * STAGE;
  static constexpr int FAC_OFF = Q_OFF + RT * QROW * 2;
  static constexpr int LO_OFF = FAC_OFF + RT * 4;
  static constexpr int HI_OFF = LO_OFF + RT * 4;
  static constexpr int PAGES_OFF = HI_OFF + RT * 4;
  static constexpr int SMEM_LOOP = PAGES_OFF + 2 * STAGES * (BK / 16) * 4;
  static constexpr int ML_OFF = 4 * 8 * NT * OROW * 4;  // at the end: O of the warps, m and l
  static constexpr int SMEM_END = ML_OFF + 2 * 4 * 8 * NT * 4;
  static constexpr int SMEM = SMEM_LOOP > SMEM_END ? SMEM_LOOP : SMEM_END;
  // CTAs that share an SM (registers are bounded for them): with 3 instead of 2 the
  // decoding cases above run at the copy rate, with more rows 2 are faster
  static constexpr int FIT = (227 * 1024) / (SMEM + 1024);
  static constexpr int CTAS = FIT < (NT == 1 ? 3 : 2) ? FIT : (NT == 1 ? 3 : 2);
  static constexpr bool QREG = D * NT <= 256;  // Q fragments live in registers
  static constexpr float OFFSET = FP8 ? 6.f : 0.f;
  static constexpr float RAISE = 8.f + OFFSET;  // above m by this, m is raised
};

template <int D, bool FP8, int NT>
__global__ void __launch_bounds__(128, PagedCfg<D, FP8, NT>::CTAS)
    attn_paged_kernel(const PagedParams p) {
  using C = PagedCfg<D, FP8, NT>;
  constexpr int BK = C::BK, KT = C::KT, WK = C::WK, RT = C::RT, CPR = C::CPR;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int quad = lane & 3, oct = lane >> 2;
  const int mat = lane >> 3, in8 = lane & 7;

  PagedPlace w{};
  if (!w.find<D, RT, 128>(p)) return;
  const int rows = w.rows, kb = w.kb, ke = w.ke;
  const int tiles = (ke - kb + BK - 1) / BK;
  const PagedLoader<C> loads(p, w, smem, C::PAGES_OFF);
#pragma unroll
  for (int t = 0; t < C::STAGES - 1; ++t) {
    if (t < tiles) loads.issue(p, t);
    pg_commit();
  }

  uint16_t* qs = reinterpret_cast<uint16_t*>(smem + C::Q_OFF);
  float* fac = reinterpret_cast<float*>(smem + C::FAC_OFF);
  int* row_lo = reinterpret_cast<int*>(smem + C::LO_OFF);
  int* row_hi = reinterpret_cast<int*>(smem + C::HI_OFF);
  paged_queries<D, FP8, RT, C::QROW, 128>(p, w, qs, fac);
  if (tid < RT) {
    const int i = (w.r0 + min(tid, rows - 1)) / p.group;
    row_lo[tid] = w.row_lo(p, i);
    row_hi[tid] = w.row_hi(p, i);
  }
  __syncthreads();
  const uint16_t* q_row = qs + oct * C::QROW;
  uint32_t qf[C::QREG ? NT : 1][C::QREG ? D / 16 : 1][2];
  if constexpr (C::QREG) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
        pg_query_frag<FP8>(q_row + nt * 8 * C::QROW, s, quad, qf[nt][s][0], qf[nt][s][1]);
  }
  auto q_frag = [&](int nt, int s, uint32_t& b0, uint32_t& b1) {
    if constexpr (C::QREG)
      b0 = qf[nt][s][0], b1 = qf[nt][s][1];
    else
      pg_query_frag<FP8>(q_row + nt * 8 * C::QROW, s, quad, b0, b1);
  };
  const bool capped = p.cap_log2 > 0.f;
  // per column (query row) 2 quad, 2 quad + 1 of each 8
  float rf[NT][2], m[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      rf[nt][j] = fac[nt * 8 + 2 * quad + j];
      m[nt][j] = -INFINITY;
      l[nt][j] = 0.f;
    }
  float o[D / 16][NT][4];
#pragma unroll
  for (int d = 0; d < D / 16; ++d)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[d][nt][x] = 0.f;

  for (int t = 0; t < tiles; ++t) {
    pg_wait<C::STAGES - 2>();
    __syncthreads();  // tile t has landed; every warp is done with tile t - 1
    if (t + C::STAGES - 1 < tiles) {
      loads.issue(p, t + C::STAGES - 1);
      loads.next_pages(p, t);
    }
    pg_commit();
    const uint32_t st = sbase + (t % C::STAGES) * C::STAGE;
    const uint8_t* stage = smem + (t % C::STAGES) * C::STAGE;
    const float2* scales = reinterpret_cast<const float2*>(stage + 2 * C::TILE) ;
#pragma unroll 1
    for (int step = 0; step < C::KW / KT; ++step) {
      const int kr0 = (warp * C::KW + step * KT) * 16;  // the warp's rows of the tile
      const int key0 = kb + t * BK + kr0;
      if (key0 >= ke) break;  // the sequence ends before them

      // ---- products of the warp's keys; two chains of MMAs where there are few
      float s[KT][NT][4];
      constexpr int CH = KT * NT <= 2 ? 2 : 1;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        float acc[CH][NT][4];
#pragma unroll
        for (int ch = 0; ch < CH; ++ch)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[ch][nt][x] = 0.f;
        const int row = kr0 + kt * 16 + (mat & 1) * 8 + in8;
#pragma unroll
        for (int pr = 0; pr < CPR / 2; ++pr) {
          uint32_t a[4];
          pg_ldm(a, st + pg_swizzle<C::ROWB>(row, 2 * pr + (mat >> 1)));
          if constexpr (FP8) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t a0 = pg_f16_lo(a[2 * u]), a1 = pg_f16_lo(a[2 * u + 1]);
              const uint32_t a2 = pg_f16_hi(a[2 * u]), a3 = pg_f16_hi(a[2 * u + 1]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                uint32_t b0, b1;
                q_frag(nt, 2 * pr + u, b0, b1);
                pg_mma<true>(acc[u % CH][nt], a0, a1, a2, a3, b0, b1);
              }
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t b0, b1;
              q_frag(nt, pr, b0, b1);
              pg_mma<false>(acc[pr % CH][nt], a[0], a[1], a[2], a[3], b0, b1);
            }
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            s[kt][nt][x] = CH == 2 ? acc[0][nt][x] + acc[CH - 1][nt][x] : acc[0][nt][x];
      }

      // ---- softcap and masks; the scores are s f, with f of a row and a block of keys
      auto factor = [&](const PagedScales& sc, int nt, int j) {
        // (never 0: a masked score stays -inf)
        return capped ? 1.f : fmaxf(rf[nt][j] * sc.ks, 1.2e-38f);
      };
      float top[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) top[nt][0] = top[nt][1] = -INFINITY;
      PagedScales sc[KT];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const int k0 = key0 + kt * 16;
        if constexpr (FP8) sc[kt] = PagedScales(scales[kr0 / 16 + kt]);
        if (capped) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              s[kt][nt][x] = pg_cap(s[kt][nt][x] * (rf[nt][x & 1] * sc[kt].ks), p.cap_mul,
                                    p.cap_log2);
        }
        if (k0 < w.in_lo || k0 + 16 > w.in_hi || k0 + 16 > ke) {  // some row does not see some key
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int key = k0 + oct + (x >> 1) * 8, r = nt * 8 + 2 * quad + (x & 1);
              if (key < row_lo[r] || key > row_hi[r] || key >= ke) s[kt][nt][x] = -INFINITY;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j)
            top[nt][j] = fmaxf(top[nt][j], __fmaf_rn(fmaxf(s[kt][nt][j], s[kt][nt][j + 2]),
                                                     factor(sc[kt], nt, j), sc[kt].lv));
      }
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) raise |= top[nt][j] > m[nt][j] + C::RAISE;
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float v = top[nt][j];
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            if (v > m[nt][j] + C::RAISE) {
              const float to = v - C::OFFSET;
              const float a = m[nt][j] == -INFINITY ? 0.f : pg_ex2(m[nt][j] - to);
              l[nt][j] *= a;
#pragma unroll
              for (int d = 0; d < D / 16; ++d) {
                o[d][nt][j] *= a;
                o[d][nt][j + 2] *= a;
              }
              m[nt][j] = to;
            }
          }
      }
      // ---- weights 2^(s f + log2 vscale - m), with keys along the registers' pairs; the
      // sums take them without the V scale
      uint32_t pf[KT][NT][2];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float e[4];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float f = factor(sc[kt], nt, j);
            const float c = sc[kt].lv - (m[nt][j] == -INFINITY ? 0.f : m[nt][j]);
            e[j] = pg_ex2(__fmaf_rn(s[kt][nt][j], f, c));
            e[j + 2] = pg_ex2(__fmaf_rn(s[kt][nt][j + 2], f, c));
            l[nt][j] = __fmaf_rn(e[j] + e[j + 2], sc[kt].iv, l[nt][j]);
          }
          if constexpr (FP8) {
            pf[kt][nt][0] = pg_transpose(pg_f16_pair(e[0], e[1]));
            pf[kt][nt][1] = pg_transpose(pg_f16_pair(e[2], e[3]));
          } else {
            pf[kt][nt][0] = pg_transpose(bf16_pair(e[0], e[1]));
            pf[kt][nt][1] = pg_transpose(bf16_pair(e[2], e[3]));
          }
        }
      // ---- O^T += V^T P^T
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const int kr = kr0 + kt * 16, k0 = key0 + kt * 16;
        const int row = kr + (FP8 ? mat & 1 : mat >> 1) * 8 + in8;
        const int side = FP8 ? mat >> 1 : mat & 1;
        if (k0 < w.in_lo || k0 + 16 > w.in_hi) {
          // Keys that only some rows see.  A value that is not finite must not reach
          // the others through their zero weights: such a block is summed one by one.
          bool bad = false;
#pragma unroll
          for (int pr = 0; pr < CPR / 2; ++pr) {
            uint32_t a[4];
            pg_ldm_t(a, st + C::TILE + pg_swizzle<C::ROWB>(row, 2 * pr + side));
#pragma unroll
            for (int x = 0; x < 4; ++x) bad |= pg_not_finite<FP8>(a[x]);
          }
          if (__any_sync(0xffffffffu, bad)) {
#pragma unroll 1
            for (int k = 0; k < 16; ++k) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                  const int r = nt * 8 + 2 * quad + j;
                  const uint32_t pair =
                      __shfl_sync(0xffffffffu, k < 8 ? pf[kt][nt][0] : pf[kt][nt][1],
                                  (2 * quad + j) * 4 + (k & 7) / 2);
                  const float pr = pg_weight<FP8>(k & 1 ? pair >> 16 : pair & 0xffffu);
                  if (k0 + k >= row_lo[r] && k0 + k <= row_hi[r] && k0 + k < ke) {
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                      const int c = d * 16 + (FP8 ? 2 * oct : oct);
                      o[d][nt][j] += pr * pg_tile_value<FP8, C::ROWB>(stage + C::TILE, kr + k, c);
                      o[d][nt][j + 2] += pr * pg_tile_value<FP8, C::ROWB>(stage + C::TILE, kr + k,
                                                                          c + (FP8 ? 1 : 8));
                    }
                  }
                }
            }
            continue;
          }
        }
#pragma unroll
        for (int pr = 0; pr < CPR / 2; ++pr) {
          uint32_t a[4];
          pg_ldm_t(a, st + C::TILE + pg_swizzle<C::ROWB>(row, 2 * pr + side));
          if constexpr (FP8) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t a0, a1, a2, a3;
              pg_value_frag(a[2 * u], a0, a1);
              pg_value_frag(a[2 * u + 1], a2, a3);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                pg_mma<true>(o[2 * pr + u][nt], a0, a1, a2, a3, pf[kt][nt][0], pf[kt][nt][1]);
            }
          } else {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              pg_mma<false>(o[pr][nt], a[0], a[1], a[2], a[3], pf[kt][nt][0], pf[kt][nt][1]);
          }
        }
      }
    }
  }
  pg_wait<0>();
  __syncthreads();  // the tiles' memory is free

  // ---- merge the warps' parts, write O and the LSE
  float* ob = reinterpret_cast<float*>(smem);
  float* ml = reinterpret_cast<float*>(smem + C::ML_OFF);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float v = l[nt][j];
      v += __shfl_xor_sync(0xffffffffu, v, 4);
      v += __shfl_xor_sync(0xffffffffu, v, 8);
      v += __shfl_xor_sync(0xffffffffu, v, 16);
      const int r = warp * 8 * NT + nt * 8 + 2 * quad + j;  // [warp][row of the warp]
      if (oct == 0) {
        ml[2 * r] = m[nt][j];
        ml[2 * r + 1] = v;
      }
      float* dst = ob + r * C::OROW;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        if constexpr (FP8) {
          *reinterpret_cast<float2*>(dst + d * 16 + 2 * oct) =
              make_float2(o[d][nt][j], o[d][nt][j + 2]);
        } else {
          dst[d * 16 + oct] = o[d][nt][j];
          dst[d * 16 + oct + 8] = o[d][nt][j + 2];
        }
      }
    }
  __syncthreads();
  constexpr int V4 = D / 4;
  for (int x = tid; x < rows * V4; x += 128) {
    const int r = x / V4, c = (x % V4) * 4;
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < WK; ++i) top = fmaxf(top, ml[2 * (r + i * 8 * NT)]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
    for (int i = 0; i < WK; ++i) {
      const int q = r + i * 8 * NT;
      const float f = pg_ex2(ml[2 * q] - base);
      const float4 v = *reinterpret_cast<const float4*>(ob + q * C::OROW + c);
      sum += f * ml[2 * q + 1];
      a0 += f * v.x, a1 += f * v.y, a2 += f * v.z, a3 += f * v.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float l2 = sum == 0.f ? -INFINITY : base + pg_lg2(sum);
    const int64_t g = w.row_index(p, r);
    if (p.num_splits > 1) {
      const int64_t at = static_cast<int64_t>(w.split) * p.total_q * p.hq + g;
      *reinterpret_cast<float4*>(p.part_o + at * D + c) =
          make_float4(a0 * inv, a1 * inv, a2 * inv, a3 * inv);
      if (c == 0) p.part_lse[at] = l2;
    } else {
      *reinterpret_cast<uint2*>(p.out + g * D + c) =
          make_uint2(bf16_pair(a0 * inv, a1 * inv), bf16_pair(a2 * inv, a3 * inv));
      if (c == 0 && p.lse) w.store_lse(p, r, l2);
    }
  }
}

}  // namespace attn
