// paged_gather.cuh -- a paged cache's keys and values as packed bf16 rows, for
// calls with many query rows per sequence: those are bound by the tensor cores,
// so the keys are brought once into the layout of attn_fwd, whose tcgen05
// kernels run several times the rate of the mma.sync kernel in paged_attn.cuh.
// The pass reads a code (1 or 2 bytes) and writes 2 bytes per element: HBM-bound, 38 us
// for 2 x 16K tokens of 8 heads of 128 in e4m3 (5.3 TB/s; 50 us with pieces of 16
// elements, whose stores are half lines, one at a time).
//
// e4m3: code * scale rounded to bf16, exact for a power-of-two scale (a code has
// 4 significant bits).
//
// Sequence b becomes segment 2b of the packed problem, followed by segment
// 2b + 1 of no queries and kGatherPad zero rows.  attn_fwd reads whole blocks of
// up to 128 keys, multiplying those behind a segment's end by zero weights: they
// are these zeros and never another sequence's rows, whose NaN would survive
// the product.  Within a sequence such a value, behind the mask of some rows and not of
// others, would still reach them all, and a NaN score would be lost in the merge of parts.
// So sequences whose rows, keys or values are not finite are noted here, and the call
// computes them once more over their pages (paged_tc.cuh), whose rule is that a value
// reaches the rows that see it.  (Where none is noted the CTAs of that launch end at once:
// with the look at the rows 11 us of 522 for 2 x 1024 rows of 32 heads of 128 over 16K
// keys in e4m3.)  Under a window the rows more than 128 below the first visible
// key are not needed and not copied.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "paged_common.cuh"

namespace attn {

constexpr int kGatherPad = 128;
constexpr int kGatherThreads = 256;
constexpr int kGatherDeep = 8;

struct GatherParams {
  PagedParams a;       // cache, table, lengths, lo_off
  int batch, max_k;
  uint16_t* k;         // [rows][hkv][D]
  uint16_t* v;
  int32_t* cu_q;       // [2 batch + 1]
  int32_t* cu_k;
  int32_t* odd;        // [batch], zero before: 1 where something is not finite
};

__device__ __forceinline__ int gather_length(const GatherParams& p, int b) {
  return min(paged_length(p.a, b), p.max_k);
}

// the larger of the bf16 bits in each half, without the signs
__device__ __forceinline__ uint32_t gather_top(uint32_t top, const uint4& w) {
  constexpr uint32_t M = 0x7fff7fffu;
  top = __vmaxu2(top, __vmaxu2(w.x & M, w.y & M));
  return __vmaxu2(top, __vmaxu2(w.z & M, w.w & M));
}
__device__ __forceinline__ void gather_note(const GatherParams& p, int b, uint32_t top) {
  if ((top & 0xffffu) >= 0x7f80u || (top >> 16) >= 0x7f80u) p.odd[b] = 1;
}

// grid: (pages and pad of the longest sequence, sequences, K, V and a look at the queries)
template <int D, bool FP8>
__global__ void __launch_bounds__(kGatherThreads) attn_paged_gather_kernel(const GatherParams p) {
  const int b = blockIdx.y, tid = threadIdx.x;
  uint32_t top = 0;
  if (blockIdx.z == 2) {
    const int64_t c0 = p.a.cu[b];
    const int64_t pieces = (p.a.cu[b + 1] - c0) * p.a.hq * (D / 8);
    const uint4* q = reinterpret_cast<const uint4*>(p.a.q + c0 * p.a.hq * D);
    const int64_t step = static_cast<int64_t>(gridDim.x) * kGatherThreads;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kGatherThreads + tid; i < pieces; i += step)
      top = gather_top(top, q[i]);
    gather_note(p, b, top);
    return;
  }
  const int n = gather_length(p, b);
  const int page_size = 1 << p.a.page_shift;
  const int first = blockIdx.x * page_size;
  const bool header = blockIdx.x == 0 && blockIdx.z == 0;
  if (first >= n + kGatherPad && !header) return;
  // packed row of the sequence's first key
  __shared__ int64_t part[kGatherThreads / 32];
  int64_t sum = 0;
  for (int i = tid; i < b; i += kGatherThreads) sum += gather_length(p, i) + kGatherPad;
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if ((tid & 31) == 0) part[tid >> 5] = sum;
  __syncthreads();
  int64_t row0 = 0;
#pragma unroll
  for (int i = 0; i < kGatherThreads / 32; ++i) row0 += part[i];
  if (header && tid == 0) {
    p.cu_q[2 * b] = p.a.cu[b];
    p.cu_q[2 * b + 1] = p.a.cu[b + 1];
    p.cu_k[2 * b] = static_cast<int32_t>(row0);
    p.cu_k[2 * b + 1] = static_cast<int32_t>(row0 + n);
    if (b == p.batch - 1) {
      p.cu_q[2 * b + 2] = p.a.cu[b + 1];
      p.cu_k[2 * b + 2] = static_cast<int32_t>(row0 + n + kGatherPad);
    }
  }
  const int nq = p.a.cu[b + 1] - p.a.cu[b];
  if (nq <= 0) return;  // no row reads these keys
  int low = 0;
  if (p.a.lo_off < kPagedNoBound) low = max(0, n - nq - p.a.lo_off - 128);
  const int last = min(first + page_size, n + kGatherPad);
  if (last <= low) return;
  const bool is_v = blockIdx.z != 0;
  const CacheView& c = is_v ? p.a.vc : p.a.kc;
  int page = -1;
  if (first < n) page = p.a.table[b * p.a.table_stride + blockIdx.x];
  const bool known = static_cast<unsigned>(page) < static_cast<unsigned>(p.a.num_pages);
  constexpr int PIECES = D / 8;  // 8 elements each: stores of a warp are whole lines
  const int items = (last - first) * p.a.hkv * PIECES;
  uint16_t* out = (is_v ? p.v : p.k) + (row0 + first) * p.a.hkv * D;
  // kGatherDeep pieces of a thread in flight
  for (int x0 = tid; x0 < items; x0 += kGatherDeep * kGatherThreads) {
    uint4 w[kGatherDeep];  // e4m3: codes in x, y
    float scale[kGatherDeep];
#pragma unroll
    for (int i = 0; i < kGatherDeep; ++i) {
      const int x = x0 + i * kGatherThreads;
      const int piece = x % PIECES, rh = x / PIECES;
      const int h = rh % p.a.hkv, slot = rh / p.a.hkv;
      w[i] = make_uint4(0, 0, 0, 0);
      scale[i] = 0.f;
      if (x < items && first + slot < n && known) {
        const int64_t at = page * c.s_page + slot * c.s_token + h * c.s_head + piece * 8;
        if constexpr (FP8) {
          const uint2 codes = *reinterpret_cast<const uint2*>(c.p + at);
          w[i].x = codes.x, w[i].y = codes.y;
          scale[i] = c.scale[static_cast<int64_t>(page) * p.a.hkv + h];
        } else {
          w[i] = *reinterpret_cast<const uint4*>(c.p + at * 2);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kGatherDeep; ++i) {
      const int x = x0 + i * kGatherThreads;
      if (x >= items) break;
      if constexpr (FP8) {
        auto two = [&](uint32_t f16x2) {
          float f0, f1;
          asm("{.reg .b16 a, b; mov.b32 {a, b}, %2; cvt.f32.f16 %0, a; cvt.f32.f16 %1, b;}"
              : "=f"(f0), "=f"(f1) : "r"(f16x2));
          return bf16_pair(f0 * scale[i], f1 * scale[i]);
        };
        w[i] = make_uint4(two(pg_f16_lo(w[i].x)), two(pg_f16_hi(w[i].x)),
                          two(pg_f16_lo(w[i].y)), two(pg_f16_hi(w[i].y)));
      }
      top = gather_top(top, w[i]);
      *reinterpret_cast<uint4*>(out + static_cast<int64_t>(x) * 8) = w[i];
    }
  }
  gather_note(p, b, top);
}

}  // namespace attn
