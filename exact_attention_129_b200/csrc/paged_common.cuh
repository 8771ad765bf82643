// paged_common.cuh -- what the kernels of attention over a paged cache share: the
// parameters, a CTA's place in the problem, the asynchronous loads of a tile of
// keys and values, the queries' layout, and the merge of parts.
//
// A CTA serves one key/value head, RT packed query rows of one sequence (row r =
// query row r / G of head r % G of the head's group) and one part of the keys.
// Rows of pages are found through the block table one 16-byte piece at a time,
// so any page size, pool order and page end inside a tile is one path.  Keys past
// the sequence (or masked for every row of the CTA) are filled with zeros and
// never read, so what a page holds there cannot reach the result.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "paged_append.cuh"
#include "ptx.cuh"

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
  const int32_t* only;  // [batch]: sequences with 0 are left out; null: none is
};

// keys of sequence b: what its row of the block table can hold, and under 2^29
// so that bounds and offsets add up in 32 bits
__device__ __forceinline__ int paged_length(const PagedParams& p, int b) {
  const int64_t room = static_cast<int64_t>(p.pages_per_seq) << p.page_shift;
  const int64_t most = room < (1 << 29) ? room : (1 << 29);
  return static_cast<int>(min(static_cast<int64_t>(max(p.seqlens[b], 0)), most));
}

__device__ __forceinline__ float pg_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float pg_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
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

// Softcap c of a score x, both in log2 units: c log2(e) tanh(y) with y = x / (c log2(e)).
// For |y| <= 1/2 it is x times the polynomial of tanh(y) / y (ptx.cuh), off by some 2^-23 of
// x however large c is; above that the identity tanh(y) = 1 - 2 / (1 + e^2y), whose error
// is absolute, some 2^-23 of c, and so of a score that is not far below c.
constexpr float kCapY = 0.34657359f;  // y = (2 / c) x kCapY: ln(2) / 2
__device__ __forceinline__ float pg_cap_ratio(float y) {  // tanh(y) / y
  const float u = y * y;
  float r = __fmaf_rn(tanhpoly::kA4, u, tanhpoly::kA3);
  r = __fmaf_rn(r, u, tanhpoly::kA2);
  r = __fmaf_rn(r, u, tanhpoly::kA1);
  return __fmaf_rn(r, u, tanhpoly::kA0);
}
__device__ __forceinline__ float pg_cap(float x, float cap_mul, float cap_log2) {
  const float x2 = x * cap_mul, y = x2 * kCapY;
  return fabsf(y) <= tanhpoly::kY0
             ? x * pg_cap_ratio(y)
             : cap_log2 * (1.f - __fdividef(2.f, 1.f + pg_ex2(x2)));
}

// a CTA's part of the problem
struct PagedPlace {
  int h, tile, split, b;      // key/value head, row tile, part, sequence
  int c0, nq, r0, rows;       // first packed row and rows of the sequence; of the CTA
  int nk, delta;
  int klo, khi;               // keys [klo, khi) are seen by some row,
  int in_lo, in_hi;           // [in_lo, in_hi) by every row
  int kb, ke;                 // this part: [kb, ke)
  int64_t row_base;

  __device__ int row_hi(const PagedParams& p, int i) const {
    return p.hi_off >= kPagedNoBound ? nk - 1 : min(nk - 1, i + delta + p.hi_off);
  }
  __device__ int row_lo(const PagedParams& p, int i) const {
    return p.lo_off >= kPagedNoBound ? 0 : max(0, i + delta - p.lo_off);
  }
  // packed (token, head) index of the CTA's row r
  __device__ int64_t row_index(const PagedParams& p, int r) const {
    const int g = r0 + r, i = g / p.group;
    return row_base + static_cast<int64_t>(i) * p.hq + (g - i * p.group);
  }
  __device__ void store_lse(const PagedParams& p, int r, float l2) const {  // natural log
    const int64_t g = row_index(p, r);
    const int64_t t = g / p.hq;
    p.lse[(g - t * p.hq) * static_cast<int64_t>(p.total_q) + t] = l2 * 0.6931471805599453f;
  }
  // false: the CTA is left out, has no rows, or no keys (its outputs are then written
  // here); parts begin at multiples of ALIGN
  template <int D, int RT, int THREADS, int ALIGN = 16>
  __device__ bool find(const PagedParams& p) {
    const int tid = threadIdx.x;
    // heads fastest: CTAs that run together read neighbouring rows of a token-major pool
    int64_t id = blockIdx.x;
    h = static_cast<int>(id % p.hkv);
    id /= p.hkv;
    tile = static_cast<int>(id % p.row_tiles);
    id /= p.row_tiles;
    split = static_cast<int>(id % p.num_splits);
    b = static_cast<int>(id / p.num_splits);
    if (p.only && p.only[b] == 0) return false;
    c0 = p.cu[b];
    nq = p.cu[b + 1] - c0;
    r0 = tile * RT;
    const int64_t all_rows = static_cast<int64_t>(nq) * p.group;
    if (r0 >= all_rows) return false;
    rows = static_cast<int>(all_rows - r0 < RT ? all_rows - r0 : RT);
    nk = paged_length(p, b);
    delta = nk - nq;
    const int i_first = r0 / p.group, i_last = (r0 + rows - 1) / p.group;
    klo = row_lo(p, i_first);
    khi = row_hi(p, i_last) + 1;
    in_lo = row_lo(p, i_last);
    in_hi = row_hi(p, i_first) + 1;
    const int64_t kb64 =
        static_cast<int64_t>(klo & ~(ALIGN - 1)) + static_cast<int64_t>(split) * p.chunk;
    ke = khi;
    if (split + 1 < p.num_splits && kb64 + p.chunk < khi) ke = static_cast<int>(kb64 + p.chunk);
    row_base = static_cast<int64_t>(c0) * p.hq + static_cast<int64_t>(h) * p.group;
    // the merge may be put on the SMs as they empty; it waits for this grid's end
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (kb64 < ke) {
      kb = static_cast<int>(kb64);
      return true;
    }
    if (p.num_splits > 1) {
      if (tid < rows)
        p.part_lse[static_cast<int64_t>(split) * p.total_q * p.hq + row_index(p, tid)] = -INFINITY;
    } else {
      for (int x = tid; x < rows * (D / 8); x += THREADS)
        *reinterpret_cast<uint4*>(p.out + row_index(p, x / (D / 8)) * D + (x % (D / 8)) * 8) =
            make_uint4(0, 0, 0, 0);
      if (p.lse && tid < rows) store_lse(p, tid, -INFINITY);
    }
    return false;
  }
};

// byte offset of piece c of a row in a tile, such that the 8 rows of an ldmatrix
// lie in different banks
template <int ROWB>
__device__ __forceinline__ uint32_t pg_swizzle(int row, int c) {
  if constexpr (ROWB >= 128) {
    return row * ROWB + ((c ^ (row & 7)) << 4);
  } else {
    const uint32_t o = row * ROWB + (c << 4);
    return o ^ (((o >> 7) & 7) << 4);
  }
}

// Asynchronous loads of tile t (BK keys from kb on) into its stage: K, V, for e4m3
// the scales of its 16-key blocks.  The pages of the blocks come through shared
// memory some tiles ahead, so that no load waits for the block table.  Addresses are
// 32-bit products of a page or slot with a stride, added to 64-bit bases.
template <class C>
struct PagedLoader {
  static constexpr int COPIES = C::BK * C::CPR / C::THREADS;
  static constexpr int STEP = C::THREADS / C::CPR;  // rows between a thread's copies
  static constexpr int BLOCKS = C::BK / 16;
  static_assert(C::THREADS % C::CPR == 0 && C::BK % STEP == 0 && C::THREADS >= 2 * BLOCKS);
  const uint8_t *kbase, *vbase;
  const int32_t* table;
  const float *kscale, *vscale;
  uint32_t stage0;
  static constexpr int RING = 2 * C::STAGES;
  const int32_t* pages;  // [RING][BLOCKS] in shared memory: tile t's at t % RING
  uint32_t pages_at;
  int klo, ke, kb, slot_mask, last;

  __device__ PagedLoader(const PagedParams& p, const PagedPlace& w, uint8_t* smem, int pages_off) {
    const int c = threadIdx.x % C::CPR;
    kbase = p.kc.p + p.kc.s_head * C::ESZ * w.h + c * 16;
    vbase = p.vc.p + p.vc.s_head * C::ESZ * w.h + c * 16;
    table = p.table + w.b * p.table_stride;
    kscale = p.kc.scale + w.h;
    vscale = p.vc.scale + w.h;
    stage0 = static_cast<uint32_t>(__cvta_generic_to_shared(smem));
    pages = reinterpret_cast<const int32_t*>(smem + pages_off);
    pages_at = stage0 + pages_off;
    klo = w.klo, ke = w.ke, kb = w.kb;
    slot_mask = (1 << p.page_shift) - 1;
    last = (w.ke - 1) >> p.page_shift;  // last entry of the table that is read
    int32_t* first = reinterpret_cast<int32_t*>(smem + pages_off);
    for (int i = threadIdx.x; i < RING * BLOCKS; i += C::THREADS)
      first[i] = __ldg(table + min((kb + i * 16) >> p.page_shift, last));
    __syncthreads();
  }
  __device__ void issue(const PagedParams& p, int t) const {
    const int row0 = threadIdx.x / C::CPR, c = threadIdx.x % C::CPR;
    const int at = t % C::STAGES;
    const uint32_t st = stage0 + at * C::STAGE;
    const int key0 = kb + t * C::BK;
    const int32_t* ids = pages + (t % RING) * BLOCKS;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) {
      const int row = row0 + i * STEP;
      const int key = key0 + row;
      // STEP and 16 divide one another, so a copy's block is i's, plus row0's
      uint32_t page = ids[STEP >= 16 ? i * (STEP / 16) + row0 / 16 : i * STEP / 16];
      const bool live = static_cast<uint32_t>(key - klo) < static_cast<uint32_t>(ke - klo) &&
                        page < static_cast<uint32_t>(p.num_pages);
      if (!live) page = 0;
      const uint32_t slot = key & slot_mask;
      const uint32_t dst = st + pg_swizzle<C::ROWB>(row, c);
      pg_cp16(dst,
              kbase + static_cast<uint64_t>(page) * p.k_page +
                  static_cast<uint64_t>(slot) * p.k_token,
              live);
      pg_cp16(dst + C::TILE,
              vbase + static_cast<uint64_t>(page) * p.v_page +
                  static_cast<uint64_t>(slot) * p.v_token,
              live);
    }
    const int tid = threadIdx.x;
    if (tid < 2 * BLOCKS) {
      if constexpr (C::ESZ == 1) {
        uint32_t page = ids[tid >> 1];  // a block of 16 keys lies in one page
        const bool live = key0 + (tid >> 1) * 16 < ke && page < static_cast<uint32_t>(p.num_pages);
        if (!live) page = 0;
        pg_cp4(st + 2 * C::TILE + tid * 4,
               ((tid & 1) ? vscale : kscale) + static_cast<int64_t>(page) * p.hkv, live);
      }
    }
  }
  // In iteration t >= 1, with the group that loads tile t + STAGES - 1: the pages of
  // tile t + RING - 1 over those of tile t - 1, which was issued long ago.  They are
  // used in iteration t + STAGES, when that group has completed.
  __device__ void next_pages(const PagedParams& p, int t) const {
    const int tid = threadIdx.x, u = t + RING - 1;
    if (t > 0 && tid < BLOCKS)
      pg_cp4(pages_at + ((u % RING) * BLOCKS + tid) * 4,
             table + min((kb + u * C::BK + tid * 16) >> p.page_shift, last), true);
  }
};

// The CTA's query rows into shared memory in the MMA's type, and the factor of
// each row's products (scale log2(e), times what undoes the row's own scaling).
// e4m3 caches multiply in f16: each row is scaled by a power of two so that its
// largest element is near 2^14, which keeps all 8 bits of elements down to 2^-31
// of it.
template <int D, bool FP8, int RT, int QROW, int THREADS>
__device__ __forceinline__ void paged_queries(const PagedParams& p, const PagedPlace& w,
                                              uint16_t* qs, float* fac) {
  constexpr int EPL = D / 32;  // elements per lane
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < RT; r += THREADS / 32) {
    uint32_t x[EPL / 2];
#pragma unroll
    for (int i = 0; i < EPL / 2; ++i) x[i] = 0;
    if (r < w.rows) {
      const uint16_t* src = p.q + w.row_index(p, r) * D + lane * EPL;
#pragma unroll
      for (int i = 0; i < EPL / 2; ++i) x[i] = *reinterpret_cast<const uint32_t*>(src + 2 * i);
    }
    float f = p.scale_log2;
    if constexpr (FP8) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < EPL / 2; ++i) m = max(m, max(x[i] & 0x7fffu, (x[i] >> 16) & 0x7fffu));
      m = __reduce_max_sync(0xffffffffu, m);
      // exponent of the row's largest element; rows that are not finite stay as
      // they are (their scores are not finite either), and tiny ones stop at 2^-100
      const int e = m >= 0x7f80u ? 14 : max(static_cast<int>(m >> 7) - 127, -100);
      const float up = exp2_int(14 - e);
      f *= exp2_int(e - 14);
#pragma unroll
      for (int i = 0; i < EPL / 2; ++i)
        x[i] = pg_f16_pair(bf16_lo(x[i]) * up, bf16_hi(x[i]) * up);
    }
#pragma unroll
    for (int i = 0; i < EPL / 2; ++i)
      *reinterpret_cast<uint32_t*>(qs + r * QROW + lane * EPL + 2 * i) = x[i];
    if (lane == 0) fac[r] = f;
  }
}

// one k16 step of 8 query rows as the MMA's second operand; `row` is the lane's
// (row lane / 4 of the 8).  For e4m3 the columns are in the order the codes come in.
template <bool FP8>
__device__ __forceinline__ void pg_query_frag(const uint16_t* row, int s, int quad, uint32_t& b0,
                                              uint32_t& b1) {
  const uint16_t* src = row + s * 16;
  if constexpr (FP8) {
    const uint2 x = *reinterpret_cast<const uint2*>(src + 4 * quad);
    b0 = x.x, b1 = x.y;
  } else {
    b0 = *reinterpret_cast<const uint32_t*>(src + 2 * quad);
    b1 = *reinterpret_cast<const uint32_t*>(src + 8 + 2 * quad);
  }
}

// 4 bytes of 2 keys x 2 head columns (ldmatrix.trans) -> the two columns' pairs of keys, f16
__device__ __forceinline__ void pg_value_frag(uint32_t w, uint32_t& first, uint32_t& second) {
  const uint32_t x = __byte_perm(w, 0, 0x3120);
  first = pg_f16_lo(x);
  second = pg_f16_hi(x);
}

// a block's scales as the softmax uses them: factor of K, log2 and inverse of V's.
// The pages outside the pool have zeros: their keys count as x = 0 and V = 0.
struct PagedScales {
  float ks, lv, iv;
  __device__ explicit PagedScales(float2 s) {
    ks = s.x == 0.f ? 1.f : s.x;
    const float v = s.y == 0.f ? 1.f : s.y;
    lv = pg_lg2(v);
    iv = pg_rcp(v);
  }
  __device__ PagedScales() : ks(1.f), lv(0.f), iv(1.f) {}
};

// one f16 (e4m3 caches) or bf16 in the low half of h
template <bool FP8>
__device__ __forceinline__ float pg_weight(uint32_t h) {
  if constexpr (FP8) {
    float f;
    asm("{.reg .b16 a, b; mov.b32 {a, b}, %1; cvt.f32.f16 %0, a;}" : "=f"(f) : "r"(h));
    return f;
  } else {
    return __uint_as_float(h << 16);
  }
}

// element d of a row of a loaded tile
template <bool FP8, int ROWB>
__device__ __forceinline__ float pg_tile_value(const uint8_t* tile, int row, int d) {
  const int byte = FP8 ? d : 2 * d;
  const uint8_t* p = tile + pg_swizzle<ROWB>(row, byte >> 4) + (byte & 15);
  if constexpr (FP8)
    return pg_weight<true>(pg_f16_lo(*p));
  else
    return pg_weight<false>(*reinterpret_cast<const uint16_t*>(p));
}

// whether one of two packed 16-bit values (f16 made of codes, or bf16) is not finite
template <bool FP8>
__device__ __forceinline__ bool pg_not_finite16(uint32_t w) {
  constexpr uint32_t E = FP8 ? 0x7c00u : 0x7f80u;
  return (w & E) == E || (w & (E << 16)) == (E << 16);
}
// the same of four codes (NaN is 0x7f with a sign), or of two bf16
template <bool FP8>
__device__ __forceinline__ bool pg_not_finite(uint32_t w) {
  if constexpr (FP8) return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
  return pg_not_finite16<false>(w);
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
