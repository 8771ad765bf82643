// paged_attn.cuh -- attention of a few query rows per sequence over a paged
// key/value cache in bf16 or e4m3 (one scale per page and key/value head).
//
// One CTA serves one key/value head, RT packed query rows of one sequence (row
// r = query row r / G of head r % G of the head's group) and one part of the
// sequence's keys:
//
//   x_j = 2log(e) scale (q . Kcode_j) kscale_j        (then softcap and mask)
//   l = sum_j 2^(x_j - m),   O = sum_j 2^(x_j - m) vscale_j Vcode_j / l
//
// Bound by HBM: each code is read once and does 2 G multiply-adds a row, far
// under the tensor cores' ridge.  So the design feeds the loads: cp.async keeps
// STAGES - 1 tiles of BK keys in flight per CTA and two or three CTAs share an
// SM; rows of pages are found through the block table one 16-byte piece at a
// time, so any page size, pool order and page end inside a tile is one path.
// Keys past the sequence (or masked for every row of the CTA) are filled with
// zeros and never read, so what a page holds there cannot reach the result.
//
// The products run transposed, on mma.m16n8k16: S^T = K Q^T with 16 keys as the
// matrix rows and 8 query rows as its columns, O^T = V^T P^T with 16 columns of
// the head as rows.  The cache is then always the 16-row operand, which is read
// once per 8 NT query rows, and a decoding step of 4 or 8 heads wastes little.
// (tcgen05 would need the cache as an operand in shared memory next to 128-row
// tiles, for no gain while HBM sets the pace; many rows take another path.)
// The four warps are WK parts of a tile's keys times WR parts of the rows; each
// warp keeps its own m, l and O, merged once at the end through shared memory.
//
// e4m3: codes become f16 (exact) in registers, 2 at a time.  K: the 4 bytes a
// thread gets from ldmatrix are 4 neighbouring head columns, used as columns
// 2q, 2q+1 and 2q+8, 2q+9 of the MMA; Q is laid out in the same order.  V:
// ldmatrix.trans moves pairs of bytes, so a thread gets two head columns of two
// keys; one byte permute separates them and they become rows r and r + 8.
// q is scaled by a power of two per row so that its largest element is near
// 2^14 in f16: it keeps all 8 bits of elements down to 2^-31 of that.
// P carries the V scale: w_j = 2^(x_j - m) vscale_j, where m follows the
// largest x_j + log2 vscale_j, so f16 holds the weights that matter whatever the
// spread of the scales.  m is kept 6 below the maximum (w up to 2^14) so that
// f16's subnormals begin 2^20 below it.  m is raised only when exceeded by 2^8;
// any m gives the same quotient, and the sum l is taken in fp32 before rounding.
// bf16: operands as they are, P rounded to bf16.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "paged_append.cuh"

namespace attn {

constexpr int32_t kPagedNoBound = 0x3fffffff;

struct PagedParams {
  const uint16_t* q;
  CacheView kc, vc;
  const int32_t* table;
  int64_t table_stride;
  const int32_t* cu;
  const int32_t* seqlens;
  uint16_t* out;
  float* lse;        // [hq][total_q], or null
  float* part_o;     // [num_splits][total_q * hq][D], when num_splits > 1
  float* part_lse;   // [num_splits][total_q * hq], log2 units
  int total_q, hq, hkv, group;
  int page_shift, num_pages, pages_per_seq;
  float scale_log2;  // scale * log2(e)
  float cap_mul, cap_log2;  // softcap c: 2 / c, c log2(e); 0: none
  int hi_off, lo_off;      // as in FwdParams, kPagedNoBound: none
  int num_splits, chunk, row_tiles;
  uint32_t k_page, k_token, v_page, v_token;  // strides in bytes
};

// keys of sequence b: what its row of the block table can hold, and under 2^29
// so that bounds and offsets add up in 32 bits
__device__ __forceinline__ int paged_length(const PagedParams& p, int b) {
  const int64_t room = static_cast<int64_t>(p.pages_per_seq) << p.page_shift;
  const int64_t most = room < (1 << 29) ? room : (1 << 29);
  return static_cast<int>(min(static_cast<int64_t>(max(p.seqlens[b], 0)), most));
}

template <int D, bool FP8, int NT, int WR>
struct PagedCfg {
  static constexpr int ESZ = FP8 ? 1 : 2;
  static constexpr int ROWB = D * ESZ;       // bytes of a cached row
  static constexpr int CPR = ROWB / 16;      // 16-byte pieces of it
  static constexpr int WK = 4 / WR;
  // Tiles and stages measured on 16 sequences of 64K (e4m3, head_dim 128): 128
  // keys x 2 stages 351 us, 128 x 3 382, 64 x 4 381: a third CTA on an SM (64 KB
  // each) beats deeper stages.  Rows of 256 bytes: 64 x 2 334 us against 64 x 3
  // 341 and 64 x 4 494 (128 ragged sequences in bf16).  Rows of 64 bytes: 3
  // stages 91 us, 2 stages 93.
  static constexpr int BK = ROWB <= 128 ? 128 : 64;  // keys per tile
  static constexpr int KT = BK / WK / 16;    // 16-key blocks per warp and tile
  static constexpr int RT = 8 * NT * WR;     // query rows per CTA
  static constexpr int TILE = BK * ROWB;
  static constexpr int STAGES = ROWB == 64 ? 3 : 2;
  static constexpr int STAGE = 2 * TILE + 2 * (BK / 16) * 4;  // K, V, their scales
  static constexpr int QROW = D + 8;         // padded, in elements
  static constexpr int OROW = D + 4;
  static constexpr int Q_OFF = STAGES * STAGE;
  static constexpr int FAC_OFF = Q_OFF + RT * QROW * 2;
  static constexpr int SMEM_LOOP = FAC_OFF + RT * 4;
  static constexpr int ML_OFF = 4 * 8 * NT * OROW * 4;  // epilogue: O of 4 warps, then m and l
  static constexpr int SMEM_END = ML_OFF + 2 * 4 * 8 * NT * 4;
  static constexpr int SMEM = SMEM_LOOP > SMEM_END ? SMEM_LOOP : SMEM_END;
  static constexpr bool QREG = D * NT <= 256;  // Q fragments live in registers
  static constexpr float OFFSET = FP8 ? 6.f : 0.f;
};

__device__ __forceinline__ float pg_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float pg_lg2(float x) {
  float r;
  asm("lg2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void pg_cp16(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void pg_cp4(uint32_t dst, const void* src, bool live) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
               "r"(live ? 4 : 0)
               : "memory");
}
__device__ __forceinline__ void pg_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void pg_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void pg_ldm(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void pg_ldm_t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t pg_transpose(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool F16>
__device__ __forceinline__ void pg_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                       uint32_t a3, uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// two codes (low or high half of w) -> two f16, exact
__device__ __forceinline__ uint32_t pg_f16_lo(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pg_f16_hi(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.f16x2.e4m3x2 %0, b;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pg_f16_pair(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// c log2(e) tanh(x), x given as 2 log2(e) x: 1 - 2 / (1 + e^2x)
__device__ __forceinline__ float pg_cap(float x2, float cap_log2) {
  return cap_log2 * (1.f - __fdividef(2.f, 1.f + pg_ex2(x2)));
}

template <int D, bool FP8, int NT, int WR>
__global__ void __launch_bounds__(128) attn_paged_kernel(const PagedParams p) {
  using C = PagedCfg<D, FP8, NT, WR>;
  constexpr int BK = C::BK, KT = C::KT, WK = C::WK, RT = C::RT, CPR = C::CPR;
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int wk = warp % WK, wr = warp / WK;
  const int quad = lane & 3, oct = lane >> 2;

  // this CTA's head, rows, sequence and part of the keys (heads fastest: CTAs
  // that run together read neighbouring rows of a token-major pool)
  int64_t id = blockIdx.x;
  const int h = static_cast<int>(id % p.hkv);
  id /= p.hkv;
  const int tile = static_cast<int>(id % p.row_tiles);
  id /= p.row_tiles;
  const int split = static_cast<int>(id % p.num_splits);
  const int b = static_cast<int>(id / p.num_splits);
  const int c0 = p.cu[b], nq = p.cu[b + 1] - c0;
  const int r0 = tile * RT;
  const int64_t all_rows = static_cast<int64_t>(nq) * p.group;
  if (r0 >= all_rows) return;
  const int rows = static_cast<int>(all_rows - r0 < RT ? all_rows - r0 : RT);
  const int nk = paged_length(p, b);
  const int delta = nk - nq;
  // keys [lo, hi] of a query row
  auto row_hi = [&](int i) {
    return p.hi_off >= kPagedNoBound ? nk - 1 : min(nk - 1, i + delta + p.hi_off);
  };
  auto row_lo = [&](int i) {
    return p.lo_off >= kPagedNoBound ? 0 : max(0, i + delta - p.lo_off);
  };
  const int i_first = r0 / p.group, i_last = (r0 + rows - 1) / p.group;
  const int klo = row_lo(i_first), khi = row_hi(i_last) + 1;   // seen by some row
  const int in_lo = row_lo(i_last), in_hi = row_hi(i_first) + 1;  // seen by every row
  const int64_t kb64 = static_cast<int64_t>(klo & ~15) + static_cast<int64_t>(split) * p.chunk;
  int ke = khi;
  if (split + 1 < p.num_splits && kb64 + p.chunk < khi) ke = static_cast<int>(kb64 + p.chunk);
  const int64_t row_base = static_cast<int64_t>(c0) * p.hq + static_cast<int64_t>(h) * p.group;
  // packed (token, head) index of the CTA's row r
  auto row_index = [&](int r) {
    const int g = r0 + r, i = g / p.group;
    return row_base + static_cast<int64_t>(i) * p.hq + (g - i * p.group);
  };
  auto store_lse = [&](int r, float l2) {  // natural log
    const int64_t g = row_index(r);
    const int64_t t = g / p.hq;
    p.lse[(g - t * p.hq) * static_cast<int64_t>(p.total_q) + t] = l2 * 0.6931471805599453f;
  };
  // the merge may be put on the SMs as they empty; it waits for this grid's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (kb64 >= ke) {  // no key of this part is seen
    if (p.num_splits > 1) {
      if (tid < rows)
        p.part_lse[static_cast<int64_t>(split) * p.total_q * p.hq + row_index(tid)] = -INFINITY;
    } else {
      for (int x = tid; x < rows * (D / 8); x += 128)
        *reinterpret_cast<uint4*>(p.out + row_index(x / (D / 8)) * D + (x % (D / 8)) * 8) =
            make_uint4(0, 0, 0, 0);
      if (p.lse && tid < rows) store_lse(tid, -INFINITY);
    }
    return;
  }
  const int kb = static_cast<int>(kb64);
  const int tiles = (ke - kb + BK - 1) / BK;

  // ---- loads: 32-bit products of a page or slot with a stride, added to 64-bit bases
  const uint8_t* kbase = p.kc.p + p.kc.s_head * C::ESZ * h + (tid % CPR) * 16;
  const uint8_t* vbase = p.vc.p + p.vc.s_head * C::ESZ * h + (tid % CPR) * 16;
  const int32_t* table = p.table + b * p.table_stride;
  const int slot_mask = (1 << p.page_shift) - 1;
  const int row_in_tile = tid / CPR;
  auto swizzle = [](int row, int c) -> uint32_t {
    if constexpr (C::ROWB >= 128) {
      return row * C::ROWB + ((c ^ (row & 7)) << 4);
    } else {
      const uint32_t o = row * C::ROWB + (c << 4);
      return o ^ (((o >> 7) & 7) << 4);
    }
  };
  uint32_t dst[BK * CPR / 128];
#pragma unroll
  for (int i = 0; i < BK * CPR / 128; ++i)
    dst[i] = sbase + swizzle(row_in_tile + i * (128 / CPR), tid % CPR);
  const uint32_t spread = ke - klo;
  auto issue = [&](int t) {
    const uint32_t st = (t % C::STAGES) * C::STAGE;
    const int key0 = kb + t * BK;
#pragma unroll
    for (int i = 0; i < BK * CPR / 128; ++i) {
      const int key = key0 + row_in_tile + i * (128 / CPR);
      uint32_t page = 0;
      bool live = static_cast<uint32_t>(key - klo) < spread;
      if (live) {
        page = __ldg(table + (key >> p.page_shift));
        live = page < static_cast<uint32_t>(p.num_pages);
      }
      if (!live) page = 0;
      const uint32_t slot = key & slot_mask;
      pg_cp16(st + dst[i],
              kbase + static_cast<uint64_t>(page) * p.k_page + static_cast<uint64_t>(slot) * p.k_token,
              live);
      pg_cp16(st + C::TILE + dst[i],
              vbase + static_cast<uint64_t>(page) * p.v_page + static_cast<uint64_t>(slot) * p.v_token,
              live);
    }
    if constexpr (FP8) {
      if (tid < 2 * (BK / 16)) {
        const int key = key0 + (tid >> 1) * 16;  // a block of 16 keys lies in one page
        uint32_t page = 0;
        bool live = key < ke;
        if (live) {
          page = __ldg(table + (key >> p.page_shift));
          live = page < static_cast<uint32_t>(p.num_pages);
        }
        if (!live) page = 0;
        const float* src = ((tid & 1) ? p.vc.scale : p.kc.scale) +
                           static_cast<int64_t>(page) * p.hkv + h;
        pg_cp4(sbase + st + 2 * C::TILE + tid * 4, src, live);
      }
    }
  };
#pragma unroll
  for (int t = 0; t < C::STAGES - 1; ++t) {
    if (t < tiles) issue(t);
    pg_commit();
  }

  // ---- queries: rows in shared memory, in the MMA's type
  uint16_t* qs = reinterpret_cast<uint16_t*>(smem + C::Q_OFF);
  float* fac = reinterpret_cast<float*>(smem + C::FAC_OFF);
  constexpr int EPL = D / 32;  // elements per lane
  for (int r = warp; r < RT; r += 4) {
    uint32_t w[EPL / 2];
#pragma unroll
    for (int i = 0; i < EPL / 2; ++i) w[i] = 0;
    if (r < rows) {
      const uint16_t* src = p.q + row_index(r) * D + lane * EPL;
#pragma unroll
      for (int i = 0; i < EPL / 2; ++i) w[i] = *reinterpret_cast<const uint32_t*>(src + 2 * i);
    }
    float f = p.scale_log2;
    if constexpr (FP8) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < EPL / 2; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
      m = __reduce_max_sync(0xffffffffu, m);
      // exponent of the row's largest element; rows that are not finite stay as
      // they are (their scores are not finite either), and tiny ones stop at 2^-100
      const int e = m >= 0x7f80u ? 14 : max(static_cast<int>(m >> 7) - 127, -100);
      const float up = exp2_int(14 - e);
      f *= exp2_int(e - 14);
#pragma unroll
      for (int i = 0; i < EPL / 2; ++i)
        w[i] = pg_f16_pair(bf16_lo(w[i]) * up, bf16_hi(w[i]) * up);
    }
#pragma unroll
    for (int i = 0; i < EPL / 2; ++i)
      *reinterpret_cast<uint32_t*>(qs + r * C::QROW + lane * EPL + 2 * i) = w[i];
    if (lane == 0) fac[r] = f;
  }
  __syncthreads();
  const uint16_t* qw = qs + (wr * 8 * NT + oct) * C::QROW;
  auto q_frag = [&](int nt, int s, uint32_t& b0, uint32_t& b1) {
    const uint16_t* src = qw + nt * 8 * C::QROW + s * 16;
    if constexpr (FP8) {
      const uint2 x = *reinterpret_cast<const uint2*>(src + 4 * quad);
      b0 = x.x, b1 = x.y;
    } else {
      b0 = *reinterpret_cast<const uint32_t*>(src + 2 * quad);
      b1 = *reinterpret_cast<const uint32_t*>(src + 8 + 2 * quad);
    }
  };
  uint32_t qf[C::QREG ? NT : 1][C::QREG ? D / 16 : 1][2];
  if constexpr (C::QREG) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int s = 0; s < D / 16; ++s) q_frag(nt, s, qf[nt][s][0], qf[nt][s][1]);
  }
  // per column (query row) 2 quad, 2 quad + 1 of each 8
  float rf[NT][2], m[NT][2], l[NT][2];
  int lo[NT][2], hi[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = wr * 8 * NT + nt * 8 + 2 * quad + j;
      rf[nt][j] = fac[r];
      m[nt][j] = -INFINITY;
      l[nt][j] = 0.f;
      const int i = (r0 + min(r, rows - 1)) / p.group;
      lo[nt][j] = row_lo(i);
      hi[nt][j] = row_hi(i);
    }
  const bool capped = p.cap_log2 > 0.f;

  float o[D / 16][NT][4];
#pragma unroll
  for (int d = 0; d < D / 16; ++d)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) o[d][nt][x] = 0.f;

  // the lane's row and piece of the 8x8 matrices: K: keys, then pieces; V (bf16):
  // pieces, then keys; V (e4m3) as K
  const int mat = lane >> 3, in8 = lane & 7;
  auto piece = [&](uint32_t base, int row, int c) { return base + swizzle(row, c); };

  for (int t = 0; t < tiles; ++t) {
    pg_wait<C::STAGES - 2>();
    __syncthreads();  // tile t has landed; every warp is done with tile t - 1
    if (t + C::STAGES - 1 < tiles) issue(t + C::STAGES - 1);
    pg_commit();
    const uint32_t st = sbase + (t % C::STAGES) * C::STAGE;
    const float* scales =
        reinterpret_cast<const float*>(smem + (t % C::STAGES) * C::STAGE + 2 * C::TILE);
    const int key0 = kb + t * BK + wk * KT * 16;  // this warp's keys
    if (key0 >= ke) continue;  // the sequence ends before them

    float s[KT][NT][4];
    float vs[KT];
    // two chains of MMAs per score where there are few: half the latency
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
      const int row = wk * KT * 16 + kt * 16 + (mat & 1) * 8 + in8;
#pragma unroll
      for (int pr = 0; pr < CPR / 2; ++pr) {
        uint32_t a[4];
        pg_ldm(a, piece(st, row, 2 * pr + (mat >> 1)));
        if constexpr (FP8) {
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t a0 = pg_f16_lo(a[2 * u]), a1 = pg_f16_lo(a[2 * u + 1]);
            const uint32_t a2 = pg_f16_hi(a[2 * u]), a3 = pg_f16_hi(a[2 * u + 1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              uint32_t b0, b1;
              if constexpr (C::QREG)
                b0 = qf[nt][2 * pr + u][0], b1 = qf[nt][2 * pr + u][1];
              else
                q_frag(nt, 2 * pr + u, b0, b1);
              pg_mma<true>(acc[u % CH][nt], a0, a1, a2, a3, b0, b1);
            }
          }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            uint32_t b0, b1;
            if constexpr (C::QREG)
              b0 = qf[nt][pr][0], b1 = qf[nt][pr][1];
            else
              q_frag(nt, pr, b0, b1);
            pg_mma<false>(acc[pr % CH][nt], a[0], a[1], a[2], a[3], b0, b1);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[kt][nt][x] = CH == 2 ? acc[0][nt][x] + acc[CH - 1][nt][x]
                                                          : acc[0][nt][x];
    }
    // scores in log2 units; the maximum of score + exponent of the V scale
    float mx[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) mx[nt][0] = mx[nt][1] = -INFINITY;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int k0 = key0 + kt * 16;
      float ks = 1.f, lv = 0.f;
      vs[kt] = 1.f;
      if constexpr (FP8) {
        const float2 sc = *reinterpret_cast<const float2*>(scales + 2 * (wk * KT + kt));
        ks = sc.x;
        vs[kt] = sc.y;
        // (a page outside the pool has scales of 0: its keys count as x = 0)
        if (vs[kt] != 0.f)
          lv = static_cast<float>(static_cast<int>(__float_as_uint(vs[kt]) >> 23) - 127);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 4; ++x) s[kt][nt][x] *= rf[nt][x & 1] * ks;
      if (capped) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[kt][nt][x] = pg_cap(s[kt][nt][x] * p.cap_mul, p.cap_log2);
      }
      if (k0 < in_lo || k0 + 16 > in_hi || k0 + 16 > ke) {  // some row does not see some key
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int key = k0 + oct + (x >> 1) * 8;
            if (key < lo[nt][x & 1] || key > hi[nt][x & 1] || key >= ke)
              s[kt][nt][x] = -INFINITY;
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          mx[nt][j] = fmaxf(mx[nt][j], fmaxf(s[kt][nt][j], s[kt][nt][j + 2]) + lv);
    }
    bool raise = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) raise |= mx[nt][j] > m[nt][j] + (8.f + C::OFFSET);
    if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float v = mx[nt][j];
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          if (v > m[nt][j] + (8.f + C::OFFSET)) {
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
    uint32_t pf[KT][NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float m0 = m[nt][0] == -INFINITY ? 0.f : m[nt][0];
      const float m1 = m[nt][1] == -INFINITY ? 0.f : m[nt][1];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const float p0 = pg_ex2(s[kt][nt][0] - m0), p1 = pg_ex2(s[kt][nt][1] - m1);
        const float p2 = pg_ex2(s[kt][nt][2] - m0), p3 = pg_ex2(s[kt][nt][3] - m1);
        l[nt][0] += p0 + p2;
        l[nt][1] += p1 + p3;
        uint32_t x, y;
        if constexpr (FP8) {
          x = pg_f16_pair(p0 * vs[kt], p1 * vs[kt]);
          y = pg_f16_pair(p2 * vs[kt], p3 * vs[kt]);
        } else {
          x = bf16_pair(p0, p1);
          y = bf16_pair(p2, p3);
        }
        pf[kt][nt][0] = pg_transpose(x);
        pf[kt][nt][1] = pg_transpose(y);
      }
    }
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int kr = wk * KT * 16 + kt * 16;
#pragma unroll
      for (int pr = 0; pr < CPR / 2; ++pr) {
        uint32_t a[4];
        if constexpr (FP8) {
          pg_ldm_t(a, piece(st + C::TILE, kr + (mat & 1) * 8 + in8, 2 * pr + (mat >> 1)));
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t x = __byte_perm(a[2 * u], 0, 0x3120);
            const uint32_t y = __byte_perm(a[2 * u + 1], 0, 0x3120);
            const uint32_t a0 = pg_f16_lo(x), a1 = pg_f16_hi(x);
            const uint32_t a2 = pg_f16_lo(y), a3 = pg_f16_hi(y);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              pg_mma<true>(o[2 * pr + u][nt], a0, a1, a2, a3, pf[kt][nt][0], pf[kt][nt][1]);
          }
        } else {
          pg_ldm_t(a, piece(st + C::TILE, kr + (mat >> 1) * 8 + in8, 2 * pr + (mat & 1)));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            pg_mma<false>(o[pr][nt], a[0], a[1], a[2], a[3], pf[kt][nt][0], pf[kt][nt][1]);
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
          *reinterpret_cast<float2*>(dst + d * 16 + 2 * oct) = make_float2(o[d][nt][j],
                                                                           o[d][nt][j + 2]);
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
    const int src = (r / (8 * NT)) * WK * 8 * NT + r % (8 * NT);  // row in the first warp's part
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < WK; ++w) top = fmaxf(top, ml[2 * (src + w * 8 * NT)]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f, a0 = 0.f, a1 = 0.f, a2 = 0.f, a3 = 0.f;
#pragma unroll
    for (int w = 0; w < WK; ++w) {
      const int q = src + w * 8 * NT;
      const float f = pg_ex2(ml[2 * q] - base);
      const float4 v = *reinterpret_cast<const float4*>(ob + q * C::OROW + c);
      sum += f * ml[2 * q + 1];
      a0 += f * v.x, a1 += f * v.y, a2 += f * v.z, a3 += f * v.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const float l2 = sum == 0.f ? -INFINITY : base + pg_lg2(sum);
    const int64_t g = row_index(r);
    if (p.num_splits > 1) {
      const int64_t at = static_cast<int64_t>(split) * p.total_q * p.hq + g;
      *reinterpret_cast<float4*>(p.part_o + at * D + c) =
          make_float4(a0 * inv, a1 * inv, a2 * inv, a3 * inv);
      if (c == 0) p.part_lse[at] = l2;
    } else {
      *reinterpret_cast<uint2*>(p.out + g * D + c) =
          make_uint2(bf16_pair(a0 * inv, a1 * inv), bf16_pair(a2 * inv, a3 * inv));
      if (c == 0 && p.lse) store_lse(r, l2);
    }
  }
}

// O = sum_s 2^(lse_s - lse) O_s, lse = log2 sum_s 2^lse_s for one packed (row,
// head) per CTA: D / 4 threads cover the head and the CTA's groups of them take
// every GROUPS-th part, so that a row of many parts is read in a few rounds.
// A part without a key has lse = -inf and its O is not read.  Launched so that
// its start overlaps the end of the attention kernel, whose results it waits for.
template <int D>
__global__ void __launch_bounds__(256) attn_paged_merge_kernel(const PagedParams p, int batch) {
  constexpr int LANES = D / 4, GROUPS = 256 / LANES;
  __shared__ float w[128];
  __shared__ float sums[2];
  __shared__ float4 part[GROUPS][LANES];
  const int64_t g = blockIdx.x;
  const int64_t rows = static_cast<int64_t>(p.total_q) * p.hq;
  const int64_t t = g / p.hq;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (t < p.cu[0] || t >= p.cu[batch]) return;
  const int tid = threadIdx.x, n = p.num_splits;
  if (tid < 32) {
    float ls[4], top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int s = i * 32 + tid;
      ls[i] = s < n ? p.part_lse[s * rows + g] : -INFINITY;
      top = fmaxf(top, ls[i]);
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      ls[i] = pg_ex2(ls[i] - base);  // NaN where a part is NaN: its row is NaN
      sum += ls[i];
      w[i * 32 + tid] = ls[i];
    }
#pragma unroll
    for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
    if (tid == 0) {
      sums[0] = sum == 0.f ? 0.f : 1.f / sum;
      if (p.lse)
        p.lse[(g - t * p.hq) * static_cast<int64_t>(p.total_q) + t] =
            sum == 0.f ? -INFINITY : (base + pg_lg2(sum)) * 0.6931471805599453f;
    }
  }
  __syncthreads();
  const int c = tid % LANES, grp = tid / LANES;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = grp; s < n; s += GROUPS) {
    const float f = w[s];
    if (f == 0.f) continue;
    const float4 v = *reinterpret_cast<const float4*>(p.part_o + (s * rows + g) * D + c * 4);
    a.x += f * v.x, a.y += f * v.y, a.z += f * v.z, a.w += f * v.w;
  }
  part[grp][c] = a;
  __syncthreads();
  if (grp == 0) {
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) {
      const float4 v = part[i][c];
      a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
    }
    const float inv = sums[0];
    *reinterpret_cast<uint2*>(p.out + g * D + c * 4) =
        make_uint2(bf16_pair(a.x * inv, a.y * inv), bf16_pair(a.z * inv, a.w * inv));
  }
}

}  // namespace attn
