// serve_api.cu -- the C ABI of rotary positions and of the paged key/value
// cache: argument checks, kernel choice and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "attn.h"
#include "paged_append.cuh"
#include "paged_attn.cuh"
#include "paged_gather.cuh"
#include "paged_tc.cuh"
#include "rotary.cuh"

namespace attn {

// api.cu
uint32_t* device_error_word();
uint64_t device_wait_timeout_ns();
void* tensor_map_encoder();

namespace {

constexpr int kServeDevices = 64;
constexpr int64_t kMaxGrid = 0x7fffffff;
constexpr int64_t kMaxStride = int64_t(1) << 31;  // elements: the kernels' bytes fit 32 bits

struct ServeDevice {
  int major = 0, sms = 0;
};

// compute capability and SM count of the current device; null if there is none
const ServeDevice* serve_device() {
  static ServeDevice state[kServeDevices];
  static bool known[kServeDevices];  // the values never change: a race rewrites the same ones
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kServeDevices) return nullptr;
  if (!__atomic_load_n(&known[dev], __ATOMIC_ACQUIRE)) {
    ServeDevice d;
    if (cudaDeviceGetAttribute(&d.major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return nullptr;
    __atomic_store_n(&state[dev].major, d.major, __ATOMIC_RELAXED);
    __atomic_store_n(&state[dev].sms, d.sms, __ATOMIC_RELAXED);
    __atomic_store_n(&known[dev], true, __ATOMIC_RELEASE);
  }
  return &state[dev];
}

attn_status_t device_ready(const ServeDevice** out) {
  const ServeDevice* d = serve_device();
  if (!d) return ATTN_ERR_CUDA;
  if (d->major != 10) return ATTN_ERR_UNSUPPORTED;
  *out = d;
  return ATTN_OK;
}

bool on16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool on4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// strides of bf16 rows: 16-byte accesses at every head of every token
bool row_strides(int64_t st, int64_t sh) { return st % 8 == 0 && sh % 8 == 0; }

bool head_dim_ok(int32_t d) { return d == 64 || d == 128 || d == 256; }

attn_status_t rope_args(const double* inv_freq, int32_t num_freqs, int32_t interleaved,
                        float mscale, int32_t inverse, int32_t d, RopeParams* r) {
  if (num_freqs < 0 || (num_freqs > 0 && !inv_freq)) return ATTN_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(inv_freq) & 7u) != 0) return ATTN_ERR_INVALID_ARG;
  if (num_freqs % 8 != 0 || 2 * static_cast<int64_t>(num_freqs) > d) return ATTN_ERR_INVALID_ARG;
  if (!std::isfinite(mscale)) return ATTN_ERR_INVALID_ARG;
  r->inv_freq = inv_freq;
  r->half = num_freqs;
  r->interleaved = interleaved != 0;
  r->mscale = mscale;
  r->sign = inverse ? -1.f : 1.f;
  return ATTN_OK;
}

attn_status_t launched() {
  return cudaGetLastError() == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA;
}

int page_shift_of(int32_t page_size) {
  for (int s = 4; s <= 7; ++s)
    if (page_size == (1 << s)) return s;
  return -1;
}

// the checks that every use of a cache shares
attn_status_t check_cache(const attn_paged_cache_t* c) {
  if (!c || !c->k || !c->v || !c->block_table || !on16(c->k) || !on16(c->v) ||
      !on4(c->block_table))
    return ATTN_ERR_INVALID_ARG;
  if (c->type != ATTN_CACHE_BF16 && c->type != ATTN_CACHE_E4M3) return ATTN_ERR_INVALID_ARG;
  if (!head_dim_ok(c->head_dim)) return ATTN_ERR_UNSUPPORTED;
  if (page_shift_of(c->page_size) < 0) return ATTN_ERR_UNSUPPORTED;
  const bool e4m3 = c->type == ATTN_CACHE_E4M3;
  if (e4m3 && (!c->k_scale || !c->v_scale || !on4(c->k_scale) || !on4(c->v_scale)))
    return ATTN_ERR_INVALID_ARG;
  const int64_t step = e4m3 ? 16 : 8;  // 16-byte accesses everywhere
  for (int64_t s : {c->k_s_page, c->k_s_token, c->k_s_head, c->v_s_page, c->v_s_token,
                    c->v_s_head})
    if (s % step != 0 || s < 0 || s >= kMaxStride) return ATTN_ERR_INVALID_ARG;
  if (c->num_pages < 1 || c->pages_per_seq < 0 || c->nheads_kv < 1 || c->nheads_kv > 65535)
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

CacheView cache_view(const attn_paged_cache_t* c, bool v) {
  CacheView r;
  r.p = static_cast<uint8_t*>(v ? c->v : c->k);
  r.scale = c->type == ATTN_CACHE_E4M3 ? (v ? c->v_scale : c->k_scale) : nullptr;
  r.s_page = v ? c->v_s_page : c->k_s_page;
  r.s_token = v ? c->v_s_token : c->k_s_token;
  r.s_head = v ? c->v_s_head : c->k_s_head;
  return r;
}

// ---------------------------------------------------------------------------
// rotary
// ---------------------------------------------------------------------------
template <int D>
attn_status_t launch_rotary(const RotaryParams& p, int64_t blocks, int groups, cudaStream_t s) {
  attn_rotary_kernel<D><<<dim3(static_cast<unsigned>(blocks), groups), kRotaryThreads, 0, s>>>(p);
  return launched();
}

// ---------------------------------------------------------------------------
// append
// ---------------------------------------------------------------------------
template <int D, bool E4M3>
attn_status_t launch_append_few(const AppendParams& p, cudaStream_t s) {
  constexpr int L = D / 16;
  const int64_t groups = static_cast<int64_t>(p.batch) * p.page_bound * 2 * p.hkv +
                         (p.q.p ? static_cast<int64_t>(p.total) * p.hq : 0);
  const int64_t blocks = (groups * L + 127) / 128;
  if (blocks > kMaxGrid) return ATTN_ERR_INVALID_ARG;
  attn_append_few_kernel<D, E4M3><<<static_cast<unsigned>(blocks), 128, 0, s>>>(p);
  return launched();
}

template <int D, bool E4M3, int IPT>
attn_status_t launch_append_page_n(const AppendParams& p, int items, dim3 grid, cudaStream_t s) {
  attn_append_page_kernel<D, E4M3, IPT><<<grid, items / IPT, 0, s>>>(p);
  return launched();
}

template <int D, bool E4M3>
attn_status_t launch_append_page(AppendParams p, int sms, cudaStream_t s) {
  const int64_t units = static_cast<int64_t>(p.batch) * p.page_bound;
  if (units > kMaxGrid) return ATTN_ERR_INVALID_ARG;
  // A CTA walks over as many heads, up to 8, as leave two CTAs for every SM: the
  // cosines and sines are then computed once for all of them.  16384 tokens of 32
  // + 8 + 8 heads of 128 into e4m3: 75 us (5.3 TB/s); 4 CTAs an SM 78, 16 86.
  auto per_cta = [&](int heads) {
    int64_t groups = (2ll * sms + units - 1) / units;
    groups = std::min<int64_t>(std::max<int64_t>(groups, (heads + 7) / 8), heads);
    return static_cast<int>((heads + groups - 1) / groups);
  };
  p.heads_per_cta = per_cta(p.hkv);
  p.kv_groups = (p.hkv + p.heads_per_cta - 1) / p.heads_per_cta;
  p.q_heads_per_cta = p.q.p ? per_cta(p.hq) : 1;
  const int q_groups = p.q.p ? (p.hq + p.q_heads_per_cta - 1) / p.q_heads_per_cta : 0;
  if (p.kv_groups + q_groups > 65535) return ATTN_ERR_INVALID_ARG;
  const dim3 grid(static_cast<unsigned>(units), p.kv_groups + q_groups);
  const int items = (D / 16) << p.page_shift;  // 64 .. 2048
  if (items <= 512) return launch_append_page_n<D, E4M3, 1>(p, items, grid, s);
  if constexpr (D >= 128)
    if (items == 1024) return launch_append_page_n<D, E4M3, 2>(p, items, grid, s);
  if constexpr (D == 256)
    if (items == 2048) return launch_append_page_n<D, E4M3, 4>(p, items, grid, s);
  return ATTN_ERR_UNSUPPORTED;
}

template <int D>
attn_status_t launch_append(const AppendParams& p, bool e4m3, int max_seqlen, int sms,
                            cudaStream_t s) {
  if (max_seqlen <= kAppendFew)
    return e4m3 ? launch_append_few<D, true>(p, s) : launch_append_few<D, false>(p, s);
  return e4m3 ? launch_append_page<D, true>(p, sms, s) : launch_append_page<D, false>(p, sms, s);
}

// ---------------------------------------------------------------------------
// attention over the cache
// ---------------------------------------------------------------------------
constexpr int kPagedMaxSplits = 128;

// How a call is cut into CTAs, a pure function of the arguments and the device.
// Two ways are open: the paged kernel over parts of the keys (with a merge), and
// packed bf16 copies (paged_gather.cuh) with attn_fwd.  Both are estimated from
// rates measured on a B200 and the quicker one is taken.
struct PagedPlan {
  bool dense;
  int splits;          // parts of the keys (dense: of attn_fwd_split)
  // paged kernel
  int rt;              // query rows per CTA
  int row_tiles;
  int chunk;           // keys of a part
  size_t lse_off;      // workspace: partial O, then partial LSE
  // dense
  int64_t key_rows;    // of the packed copies
  size_t v_off, cu_q_off, cu_k_off, odd_off, split_off, split_bytes;
  size_t bytes;        // of the workspace
};

size_t align256(size_t n) { return (n + 255) / 256 * 256; }

constexpr double kHbmBytesPerNs = 6500.0;   // measured copy rate
constexpr int64_t kDenseBytes = int64_t(4) << 30;  // the packed copies may take so much

// Query rows per CTA: 8, and in e4m3 16, of the mma.sync kernel; 32, 64 or 128 of the
// tcgen05 kernel.  512 CTAs of 16 rows of head_dim 64, 128, 256: e4m3 24, 32, 61 ns a key
// in the mma.sync kernel, 29, 36, 67 in the other; bf16 29, 46, 120 and 29, 44, 82.
constexpr int kPagedRows[5] = {8, 16, 32, 64, 128};
// ns per key of one CTA, by type, head_dim and rows, where HBM does not set the pace.
// (Between what a CTA takes alone over 128K keys and what it takes in a full round of
// 4096: e4m3, head_dim 128, 8 / 16 / 32 / 64 / 128 rows 9.3 / 11.2 / 6.7 / 9.1 / 15.1 and
// 18.4 / 16.7 / 11.2 / 13.7 / 20.9.)
constexpr double kPagedNsPerKey[2][3][5] = {{{9., 0., 6., 7., 11.},
                                             {15., 0., 7.7, 8.2, 12.},
                                             {23., 0., 14.2, 15., 16.2}},
                                            {{8.4, 10.2, 7.7, 9.6, 17.6},
                                             {11., 14., 9.8, 12., 21.},
                                             {20.5, 25., 18., 19.5, 23.}}};
// ns per key of one CTA of attn_fwd (its query tile against one key)
constexpr double kDenseNsPerKey[3] = {15., 17.7, 21.};

struct PagedShape {
  int64_t batch, units, group, rows, max_k, span, total_q, hq;
  int d, d_index, key_bytes;  // key_bytes: of K and V of one key and head
};

constexpr double kRoundNs[2] = {3000.0, 6000.0};  // a CTA's set-up and drain: mma.sync, tcgen05
constexpr double kEqualBatches = 0.45;
constexpr double kSpread[2] = {0.2, 0.0};  // of a CTA's time: mma.sync kernel, tcgen05 kernel
constexpr double kMergeCopies = 2.0;  // the parts of O cross HBM or L2 about so often

// one round of k CTAs of chunk keys side by side
double round_ns(int64_t k, double chunk, double ns_per_key, double key_bytes, double fixed) {
  return fixed + std::max(chunk * ns_per_key, k * chunk * key_bytes / kHbmBytesPerNs);
}
// n CTAs of equal length: whole rounds of `slots`, then the rest
double rounds_ns(int64_t n, int64_t slots, double chunk, double ns_per_key, double key_bytes,
                 double fixed) {
  const int64_t full = n / slots, rest = n % slots;
  return full * round_ns(slots, chunk, ns_per_key, key_bytes, fixed) +
         (rest ? round_ns(rest, chunk, ns_per_key, key_bytes, fixed) : 0.0);
}
// n CTAs of differing lengths: a free slot takes the next one, half a CTA is left over
double ragged_ns(double n, int64_t slots, double chunk, double ns_per_key, double key_bytes,
                 double fixed) {
  if (n <= slots) return round_ns(static_cast<int64_t>(n), chunk, ns_per_key, key_bytes, fixed);
  return n / slots * round_ns(slots, chunk, ns_per_key, key_bytes, fixed) +
         0.5 * round_ns(slots / 2, chunk, ns_per_key, key_bytes, fixed);
}

double paged_plan_tiles(const PagedShape& x, int want, int sms, PagedPlan* pl) {
  const bool e4m3 = x.key_bytes == 2 * x.d;
  const int ri =
      x.rows <= 8 ? 0 : e4m3 && x.rows <= 16 ? 1 : x.rows <= 32 ? 2 : x.rows <= 64 ? 3 : 4;
  const int rt = kPagedRows[ri];
  pl->rt = rt;
  pl->row_tiles = static_cast<int>((x.rows + rt - 1) / rt);
  const int64_t per_part = x.units * pl->row_tiles;
  // CTAs that share an SM
  const int64_t slots = static_cast<int64_t>(sms) * (ri > 1 || x.key_bytes > 512 ? 1 : 3 - ri);
  const double key = kPagedNsPerKey[e4m3][x.d_index][ri], fixed = kRoundNs[ri > 1];
  auto chunk_of = [&](int64_t splits) {  // whole tiles of every kernel
    return std::max<int64_t>(128, ((x.span + splits - 1) / splits + 127) / 128 * 128);
  };
  double best = 0;
  int64_t splits = 0;
  for (int s = want ? want : 1; s <= (want ? want : kPagedMaxSplits); s += 1 + s / 8) {
    const int64_t chunk = chunk_of(s), parts = (x.span + chunk - 1) / chunk;
    const double c = static_cast<double>(chunk);
    // max_k bounds the lengths, which are not known here: as if nearly half of the batches
    // were of equal sequences and the others of sequences of 0.6 of it on average.  (0.35
    // against 0.45: 32 equal sequences of 4K with 8 rows 69 and 59 us, 128 ragged ones of up
    // to 8K 312 and 314.)
    const int64_t n = per_part * parts;
    double t = rounds_ns(n, slots, c, key, x.key_bytes, fixed);
    if (x.batch > 1)
      t = kEqualBatches * t +
          (1. - kEqualBatches) * ragged_ns(0.6 * n, slots, c, key, x.key_bytes, fixed);
    // CTAs side by side do not end together: 16 sequences of 64K take 334 us with one
    // long CTA per slot when all goes well, 356 to 390 in most runs, with 16 parts 333 to
    // 375.  The same holds where one CTA of the mma.sync kernel fills an SM (bf16 with
    // head_dim 256): 128 sequences of 16K 814 us with the parts this term leads to, 868
    // without, 3 of 64K 315 and 341, though 16 of 1000 keys 37 and 32.  (The tcgen05
    // kernel does not gain: drafts 74 us without this term, 88 with 0.2.)
    t += 4000. + kSpread[ri > 1] * round_ns(std::min(n, slots), c, key, x.key_bytes, 0.);
    if (parts > 1)
      t += 2000. + kMergeCopies * 8. * parts * x.total_q * x.hq * x.d / kHbmBytesPerNs;
    if (!splits || t < best) best = t, splits = parts;
  }
  const int64_t chunk = chunk_of(want ? want : splits);
  pl->splits = static_cast<int>((x.span + chunk - 1) / chunk);
  pl->chunk = static_cast<int>(chunk);
  const size_t rows_all = static_cast<size_t>(pl->splits) * x.total_q * x.hq;
  pl->lse_off = align256(rows_all * x.d * 4);
  pl->bytes = pl->splits > 1 ? pl->lse_off + rows_all * 4 : 0;
  return best;
}

// ATTN_PAGED_PACK=0: the packed copies are not used; 1: they are, for any number of rows
// and num_splits, wherever their sizes fit.  Read on every call, for tests and for
// callers without the memory.  -1: not set
int paged_pack_switch() {
  const char* e = std::getenv("ATTN_PAGED_PACK");
  return !e ? -1 : e[0] == '0' ? 0 : e[0] == '1' ? 1 : -1;
}

// false: not open for this call, or no quicker than `limit`; forced: whatever the estimate
bool paged_plan_dense(const PagedShape& x, int hkv, int sms, int want, double limit, bool forced,
                      PagedPlan* pl) {
  const int64_t key_rows = x.batch * (x.max_k + kGatherPad);
  const int64_t copy = key_rows * hkv * x.d * 2;
  if (x.batch > 32767 || 2 * copy > kDenseBytes || key_rows >= (1 << 30)) return false;
  if (!forced && (x.rows < 128 || x.max_k < 512)) return false;
  if (x.units * ((x.rows + 127) / 128) > kMaxGrid) return false;  // the launch over the pages
  // code read, copy written and read; three launches more
  const double gather = 16000. + key_rows * hkv * (x.key_bytes + 8. * x.d) / kHbmBytesPerNs;
  const int64_t tile = x.d == 256 ? 128 : 256;
  const int64_t ctas = x.units * ((x.rows + tile - 1) / tile);
  double best = 0;
  int splits = 0;
  const int first = want ? want : 1, most = want ? want : 16;
  // (attn_fwd's grid: segments times parts)
  for (int s = first; s <= most && 2 * x.batch * s <= 65535 && (s == first || x.max_k >= 512 * s);
       s *= 2) {
    double t = gather + rounds_ns(ctas * s, sms, static_cast<double>(x.span) / s,
                                  kDenseNsPerKey[x.d_index], 0.0, kRoundNs[0]);
    if (s > 1) t += 4000. + kMergeCopies * 8. * s * x.total_q * x.hq * x.d / kHbmBytesPerNs;
    if (!splits || t < best) best = t, splits = s;
  }
  if (!splits || (!forced && best >= limit)) return false;
  pl->dense = true;
  pl->splits = splits;
  pl->key_rows = key_rows;
  pl->v_off = align256(copy);
  pl->cu_q_off = pl->v_off + align256(copy);
  pl->cu_k_off = pl->cu_q_off + align256((2 * static_cast<size_t>(x.batch) + 1) * 4);
  pl->odd_off = pl->cu_k_off + align256((2 * static_cast<size_t>(x.batch) + 1) * 4);
  pl->split_off = pl->odd_off + align256(static_cast<size_t>(x.batch) * 4);
  pl->split_bytes = splits > 1 ? attn_fwd_split_workspace_size(static_cast<int32_t>(x.total_q),
                                                               static_cast<int32_t>(x.hq), x.d,
                                                               splits)
                               : 0;
  pl->bytes = pl->split_off + pl->split_bytes;
  return true;
}

PagedPlan paged_plan(const attn_paged_cache_t* c, int batch, int total_q, int max_q, int max_k,
                     int hq, int hi_off, int lo_off, int want, int sms) {
  PagedPlan pl{};
  PagedShape x;
  x.batch = batch;
  x.units = static_cast<int64_t>(batch) * c->nheads_kv;
  x.group = hq / c->nheads_kv;
  x.rows = x.group * max_q;
  x.max_k = max_k;
  x.total_q = total_q;
  x.hq = hq;
  x.d = c->head_dim;
  x.d_index = x.d == 64 ? 0 : x.d == 128 ? 1 : 2;
  x.key_bytes = 2 * x.d * (c->type == ATTN_CACHE_E4M3 ? 1 : 2);
  // keys a CTA's rows can see: with both bounds, the window and the rows' spread;
  // parts begin at a multiple of 16 or 128
  x.span = max_k;
  if (lo_off < kPagedNoBound && hi_off < kPagedNoBound)
    x.span = std::min<int64_t>(x.span, static_cast<int64_t>(lo_off) + hi_off + 2 +
                                           (64 + x.group - 1) / x.group);
  if (lo_off < kPagedNoBound) x.span += 127;
  x.span = std::max<int64_t>(x.span, 1);
  const double t = paged_plan_tiles(x, want, sms, &pl);
  PagedPlan dense{};
  const int pack = paged_pack_switch();
  if ((pack < 0 ? want == 0 : pack) &&
      paged_plan_dense(x, c->nheads_kv, sms, want, t, pack == 1, &dense))
    return dense;
  return pl;
}

template <int D, bool FP8>
attn_status_t launch_gather(const GatherParams& p, cudaStream_t s) {
  const int page = 1 << p.a.page_shift;
  const int64_t pages = (static_cast<int64_t>(p.max_k) + kGatherPad + page - 1) / page;
  attn_paged_gather_kernel<D, FP8>
      <<<dim3(static_cast<unsigned>(pages), p.batch, 3), kGatherThreads, 0, s>>>(p);
  return launched();
}

struct PagedMask {
  int hi_off, lo_off;
};
PagedMask paged_mask(int32_t causal, int32_t wl, int32_t wr) {
  PagedMask m;
  m.hi_off = causal ? 0 : (wr >= 0 ? std::min(wr, kPagedNoBound) : kPagedNoBound);
  m.lo_off = wl >= 0 ? std::min(wl, kPagedNoBound) : kPagedNoBound;
  return m;
}

attn_status_t paged_sizes(const attn_paged_cache_t* c, int32_t batch, int32_t total_q,
                          int32_t max_q, int32_t max_k, int32_t hq, int32_t num_splits) {
  attn_status_t st = check_cache(c);
  if (st != ATTN_OK) return st;
  if (batch < 1 || total_q < 0 || max_q < 0 || max_k < 0 || max_k > (1 << 29) || hq < 1 ||
      hq > 65535 || hq % c->nheads_kv != 0 || num_splits < 0 || num_splits > kPagedMaxSplits)
    return ATTN_ERR_INVALID_ARG;
  if (static_cast<int64_t>(total_q) * hq * c->head_dim >= (int64_t(1) << 40))
    return ATTN_ERR_INVALID_ARG;
  return ATTN_OK;
}

// raises a kernel's shared memory limit once per device, launches it and, for
// keys in parts, the merge
template <int D, auto Kernel, int THREADS, int SMEM, class... Args>
attn_status_t launch_paged(const PagedParams& p, int batch, cudaStream_t s, const Args&... args) {
  static bool ready[kServeDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return ATTN_ERR_CUDA;
  if (!__atomic_load_n(&ready[dev], __ATOMIC_ACQUIRE)) {
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM) !=
        cudaSuccess)
      return ATTN_ERR_CUDA;
    __atomic_store_n(&ready[dev], true, __ATOMIC_RELEASE);
  }
  const int64_t ctas = static_cast<int64_t>(batch) * p.num_splits * p.row_tiles * p.hkv;
  if (ctas > kMaxGrid) return ATTN_ERR_INVALID_ARG;
  Kernel<<<static_cast<unsigned>(ctas), THREADS, SMEM, s>>>(args...);
  attn_status_t st = launched();
  if (st != ATTN_OK || p.num_splits == 1) return st;
  const int64_t rows = static_cast<int64_t>(p.total_q) * p.hq;
  if (rows > kMaxGrid) return ATTN_ERR_INVALID_ARG;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(rows));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_paged_merge_kernel<D>, p, batch) == cudaSuccess
             ? ATTN_OK
             : ATTN_ERR_CUDA;
}

// a pool as (columns, token, head, page) with boxes of box_cols x tokens of one page
// and head
bool pool_map(CUtensorMap* map, const CacheView& c, const PagedParams& p, int d, int esz,
              int box_cols, int tokens, CUtensorMapSwizzle swizzle) {
  using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  const Encode encode = reinterpret_cast<Encode>(tensor_map_encoder());
  if (!encode) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), cuuint64_t(1) << p.page_shift,
                              static_cast<cuuint64_t>(p.hkv),
                              static_cast<cuuint64_t>(p.num_pages)};
  // (the stride of a dimension of 1 is never used, and may be anything)
  auto stride = [&](int64_t s, cuuint64_t n) {
    return static_cast<cuuint64_t>(n > 1 ? s * esz : static_cast<int64_t>(d) * esz);
  };
  const cuuint64_t strides[3] = {stride(c.s_token, dims[1]), stride(c.s_head, dims[2]),
                                 stride(c.s_page, dims[3])};
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(tokens), 1,
                             1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return encode(map, esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                c.p, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool FP8, int KG>
attn_status_t launch_tc(const PagedParams& p, int batch, cudaStream_t s) {
  using C = PagedTcCfg<D, FP8, KG>;
  const PagedTcParams tp{p, device_error_word(), device_wait_timeout_ns()};
  if (!tp.err) return ATTN_ERR_CUDA;
  const int tokens = std::min(1 << p.page_shift, C::BK);
  CUtensorMap k, v;
  if (!pool_map(&k, p.kc, p, D, C::ESZ, C::KROW / C::ESZ, tokens,
                C::KROW == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B) ||
      !pool_map(&v, p.vc, p, D, C::ESZ, FP8 ? D : 64, tokens,
                FP8 ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B))
    return ATTN_ERR_CUDA;
  return launch_paged<D, attn_paged_tc_kernel<D, FP8, KG>, C::THREADS, C::SMEM>(p, batch, s, k, v,
                                                                               tp);
}

template <int D, bool FP8>
attn_status_t launch_paged_rows(const PagedParams& p, const PagedPlan& pl, int batch,
                                cudaStream_t s) {
  switch (pl.rt) {
    case 8:
      return launch_paged<D, attn_paged_kernel<D, FP8, 1>, 128, PagedCfg<D, FP8, 1>::SMEM>(
          p, batch, s, p);
    case 16:
      if constexpr (FP8)
        return launch_paged<D, attn_paged_kernel<D, FP8, 2>, 128, PagedCfg<D, FP8, 2>::SMEM>(
            p, batch, s, p);
    case 32: return launch_tc<D, FP8, 4>(p, batch, s);
    case 64: return launch_tc<D, FP8, 2>(p, batch, s);
    default: return launch_tc<D, FP8, 1>(p, batch, s);
  }
}

}  // namespace
}  // namespace attn

using namespace attn;

extern "C" attn_status_t attn_rotary(
    const void* q, int64_t q_st, int64_t q_sh, const void* k, int64_t k_st, int64_t k_sh,
    void* q_out, int64_t qo_st, int64_t qo_sh, void* k_out, int64_t ko_st, int64_t ko_sh,
    const double* inv_freq, int32_t num_freqs, int32_t interleaved, float mscale, int32_t inverse,
    const int32_t* positions, const int32_t* cu_seqlens, const int32_t* offsets, int32_t batch,
    int32_t zero_outside, int32_t total, int32_t nheads_q, int32_t nheads_kv, int32_t head_dim,
    attn_stream_t stream) {
  RotaryParams p;
  if (!q || !q_out || (k == nullptr) != (k_out == nullptr) || !on16(q) || !on16(q_out) ||
      !on16(k) || !on16(k_out))
    return ATTN_ERR_INVALID_ARG;
  if (!head_dim_ok(head_dim)) return ATTN_ERR_UNSUPPORTED;
  if (!row_strides(q_st, q_sh) || !row_strides(qo_st, qo_sh) || !row_strides(k_st, k_sh) ||
      !row_strides(ko_st, ko_sh))
    return ATTN_ERR_INVALID_ARG;
  if (total < 0 || nheads_q < 1 || nheads_kv < 0 || (k ? nheads_kv < 1 : nheads_kv != 0) ||
      nheads_q > 65535 || nheads_kv > 65535)
    return ATTN_ERR_INVALID_ARG;
  if (!on4(positions) || !on4(cu_seqlens) || !on4(offsets) || (cu_seqlens && batch < 1) ||
      (offsets && !cu_seqlens) || (positions && cu_seqlens))
    return ATTN_ERR_INVALID_ARG;
  attn_status_t st = rope_args(inv_freq, num_freqs, interleaved, mscale, inverse, head_dim, &p.rope);
  if (st != ATTN_OK) return st;
  const ServeDevice* dev = nullptr;
  if ((st = device_ready(&dev)) != ATTN_OK) return st;
  if (total == 0) return ATTN_OK;
  p.q = {static_cast<const uint16_t*>(q), q_st, q_sh};
  p.k = {static_cast<const uint16_t*>(k), k_st, k_sh};
  p.qo = {static_cast<uint16_t*>(q_out), qo_st, qo_sh};
  p.ko = {static_cast<uint16_t*>(k_out), ko_st, ko_sh};
  p.positions = positions;
  p.cu = cu_seqlens;
  p.offsets = offsets;
  p.zero_outside = zero_outside != 0;
  p.batch = batch;
  p.total = total;
  p.hq = nheads_q;
  p.heads = nheads_q + nheads_kv;
  const int64_t blocks =
      (static_cast<int64_t>(total) * (head_dim / 16) + kRotaryThreads - 1) / kRotaryThreads;
  if (blocks > kMaxGrid) return ATTN_ERR_INVALID_ARG;
  // Heads per thread: up to 16, which share the angles' cost, where that leaves
  // every SM 16 blocks; down to 1 for few tokens.  16384 tokens of 40 heads of 128:
  // 56 us with 8 heads a thread, 58 with 4 or 16; 131072 of 9 heads of 256: 189 us
  // with all 9, 204 with 8 and 1, 212 with 4.
  const int64_t want = std::max<int64_t>(1, (16ll * dev->sms + blocks - 1) / blocks);
  p.heads_per_thread = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>(16, p.heads / std::min<int64_t>(want, p.heads))));
  const int groups = (p.heads + p.heads_per_thread - 1) / p.heads_per_thread;
  if (groups > 65535) return ATTN_ERR_INVALID_ARG;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (head_dim) {
    case 64: return launch_rotary<64>(p, blocks, groups, s);
    case 128: return launch_rotary<128>(p, blocks, groups, s);
    default: return launch_rotary<256>(p, blocks, groups, s);
  }
}

extern "C" attn_status_t attn_paged_append(
    const attn_paged_cache_t* cache, const void* k, int64_t k_st, int64_t k_sh, const void* v,
    int64_t v_st, int64_t v_sh, const void* q, int64_t q_st, int64_t q_sh, void* q_out,
    int64_t qo_st, int64_t qo_sh, const int32_t* cu_seqlens, const int32_t* seqlens_k,
    int32_t batch, int32_t total, int32_t max_seqlen, int32_t nheads_q, const double* inv_freq,
    int32_t num_freqs, int32_t interleaved, float mscale, attn_stream_t stream) {
  attn_status_t st = check_cache(cache);
  if (st != ATTN_OK) return st;
  if (!k || !v || !on16(k) || !on16(v) || (q == nullptr) != (q_out == nullptr) || !on16(q) ||
      !on16(q_out))
    return ATTN_ERR_INVALID_ARG;
  if (!row_strides(k_st, k_sh) || !row_strides(v_st, v_sh) || !row_strides(q_st, q_sh) ||
      !row_strides(qo_st, qo_sh))
    return ATTN_ERR_INVALID_ARG;
  if (!cu_seqlens || !seqlens_k || !on4(cu_seqlens) || !on4(seqlens_k) || batch < 1 ||
      total < 0 || max_seqlen < 0 || nheads_q < 0 || (q ? nheads_q < 1 : nheads_q != 0) ||
      nheads_q > 65535)
    return ATTN_ERR_INVALID_ARG;
  AppendParams p;
  st = rope_args(inv_freq, num_freqs, interleaved, mscale, 0, cache->head_dim, &p.rope);
  if (st != ATTN_OK) return st;
  const ServeDevice* dev = nullptr;
  if ((st = device_ready(&dev)) != ATTN_OK) return st;
  max_seqlen = std::min(max_seqlen, total);
  if (max_seqlen == 0) return ATTN_OK;
  p.k = {static_cast<const uint16_t*>(k), k_st, k_sh};
  p.v = {static_cast<const uint16_t*>(v), v_st, v_sh};
  p.q = {static_cast<const uint16_t*>(q), q_st, q_sh};
  p.qo = {static_cast<uint16_t*>(q_out), qo_st, qo_sh};
  p.kc = cache_view(cache, false);
  p.vc = cache_view(cache, true);
  p.table = cache->block_table;
  p.table_stride = cache->table_stride;
  p.cu = cu_seqlens;
  p.seqlens = seqlens_k;
  p.batch = batch;
  p.total = total;
  p.hq = nheads_q;
  p.hkv = cache->nheads_kv;
  p.page_shift = page_shift_of(cache->page_size);
  p.num_pages = cache->num_pages;
  p.pages_per_seq = cache->pages_per_seq;
  p.page_bound = static_cast<int>(
      (static_cast<int64_t>(max_seqlen) + cache->page_size - 2) / cache->page_size + 1);
  const bool e4m3 = cache->type == ATTN_CACHE_E4M3;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (cache->head_dim) {
    case 64: return launch_append<64>(p, e4m3, max_seqlen, dev->sms, s);
    case 128: return launch_append<128>(p, e4m3, max_seqlen, dev->sms, s);
    default: return launch_append<256>(p, e4m3, max_seqlen, dev->sms, s);
  }
}

extern "C" size_t attn_paged_workspace_size(const attn_paged_cache_t* cache, int32_t batch,
                                            int32_t total_q, int32_t max_seqlen_q,
                                            int32_t max_seqlen_k, int32_t nheads_q, int32_t causal,
                                            int32_t window_left, int32_t window_right,
                                            int32_t num_splits) {
  if (paged_sizes(cache, batch, total_q, max_seqlen_q, max_seqlen_k, nheads_q, num_splits) !=
      ATTN_OK)
    return 0;
  const ServeDevice* dev = serve_device();
  if (!dev || total_q == 0 || max_seqlen_q == 0) return 0;
  const PagedMask m = paged_mask(causal, window_left, window_right);
  return paged_plan(cache, batch, total_q, std::min(max_seqlen_q, total_q), max_seqlen_k, nheads_q,
                    m.hi_off, m.lo_off, num_splits, dev->sms)
      .bytes;
}

extern "C" attn_status_t attn_paged_fwd(
    const attn_paged_cache_t* cache, const void* q, const int32_t* cu_seqlens_q,
    const int32_t* seqlens_k, int32_t batch, int32_t total_q, int32_t max_seqlen_q,
    int32_t max_seqlen_k, int32_t nheads_q, float scale, int32_t causal, int32_t window_left,
    int32_t window_right, float softcap, int32_t num_splits, int32_t return_lse, void* out,
    float* lse, void* workspace, size_t workspace_bytes, attn_stream_t stream) {
  attn_status_t st = paged_sizes(cache, batch, total_q, max_seqlen_q, max_seqlen_k, nheads_q,
                                 num_splits);
  if (st != ATTN_OK) return st;
  if (!q || !on16(q) || !out || !on16(out) || !cu_seqlens_q || !seqlens_k ||
      !on4(cu_seqlens_q) || !on4(seqlens_k) || (return_lse && (!lse || !on4(lse))))
    return ATTN_ERR_INVALID_ARG;
  if (!(std::isfinite(scale) && scale > 0.f) || !std::isfinite(softcap) || softcap < 0.f)
    return ATTN_ERR_INVALID_ARG;
  const ServeDevice* dev = nullptr;
  if ((st = device_ready(&dev)) != ATTN_OK) return st;
  if (total_q == 0 || max_seqlen_q == 0) return ATTN_OK;
  const PagedMask m = paged_mask(causal, window_left, window_right);
  PagedPlan pl = paged_plan(cache, batch, total_q, std::min(max_seqlen_q, total_q), max_seqlen_k,
                            nheads_q, m.hi_off, m.lo_off, num_splits, dev->sms);
  if (pl.bytes > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) ||
                       workspace_bytes < pl.bytes))
    return ATTN_ERR_INVALID_ARG;
  PagedParams p;
  p.q = static_cast<const uint16_t*>(q);
  p.kc = cache_view(cache, false);
  p.vc = cache_view(cache, true);
  p.table = cache->block_table;
  p.table_stride = cache->table_stride;
  p.cu = cu_seqlens_q;
  p.seqlens = seqlens_k;
  p.out = static_cast<uint16_t*>(out);
  p.lse = return_lse ? lse : nullptr;
  p.part_o = static_cast<float*>(workspace);
  p.part_lse = pl.bytes ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + pl.lse_off)
                        : nullptr;
  p.total_q = total_q;
  p.hq = nheads_q;
  p.hkv = cache->nheads_kv;
  p.group = nheads_q / cache->nheads_kv;
  p.page_shift = page_shift_of(cache->page_size);
  p.num_pages = cache->num_pages;
  p.pages_per_seq = cache->pages_per_seq;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.cap_mul = softcap > 0.f ? 2.f / softcap : 0.f;
  p.cap_log2 = softcap * 1.4426950408889634f;
  p.hi_off = m.hi_off;
  p.lo_off = m.lo_off;
  p.num_splits = pl.splits;
  p.chunk = pl.chunk;
  p.row_tiles = pl.row_tiles;
  const uint32_t esz = cache->type == ATTN_CACHE_E4M3 ? 1 : 2;
  p.k_page = static_cast<uint32_t>(cache->k_s_page) * esz;
  p.k_token = static_cast<uint32_t>(cache->k_s_token) * esz;
  p.v_page = static_cast<uint32_t>(cache->v_s_page) * esz;
  p.v_token = static_cast<uint32_t>(cache->v_s_token) * esz;
  p.only = nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool e4m3 = cache->type == ATTN_CACHE_E4M3;
  if (pl.dense) {
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    GatherParams g;
    g.a = p;
    g.batch = batch;
    g.max_k = max_seqlen_k;
    g.k = reinterpret_cast<uint16_t*>(ws);
    g.v = reinterpret_cast<uint16_t*>(ws + pl.v_off);
    g.cu_q = reinterpret_cast<int32_t*>(ws + pl.cu_q_off);
    g.cu_k = reinterpret_cast<int32_t*>(ws + pl.cu_k_off);
    g.odd = reinterpret_cast<int32_t*>(ws + pl.odd_off);
    if (cudaMemsetAsync(g.odd, 0, static_cast<size_t>(batch) * 4, s) != cudaSuccess)
      return ATTN_ERR_CUDA;
    switch (cache->head_dim) {
      case 64: st = e4m3 ? launch_gather<64, true>(g, s) : launch_gather<64, false>(g, s); break;
      case 128: st = e4m3 ? launch_gather<128, true>(g, s) : launch_gather<128, false>(g, s); break;
      default: st = e4m3 ? launch_gather<256, true>(g, s) : launch_gather<256, false>(g, s);
    }
    if (st != ATTN_OK) return st;
    st = attn_fwd_split(q, g.k, g.v, g.cu_q, g.cu_k, 2 * batch, total_q,
                        static_cast<int32_t>(pl.key_rows), max_seqlen_q, max_seqlen_k, nheads_q,
                        cache->nheads_kv, cache->head_dim, scale, causal, window_left,
                        window_right, softcap, pl.splits, return_lse, out, lse,
                        ws + pl.split_off, pl.split_bytes, stream);
    if (st != ATTN_OK) return st;
    // the sequences that the copies do not serve, over their pages
    p.only = g.odd;
    pl.rt = 128;
    p.num_splits = 1;
    p.chunk = max_seqlen_k;
    const int64_t rows = static_cast<int64_t>(p.group) * std::min(max_seqlen_q, total_q);
    p.row_tiles = static_cast<int>((rows + pl.rt - 1) / pl.rt);
  }
  switch (cache->head_dim) {
    case 64:
      return e4m3 ? launch_paged_rows<64, true>(p, pl, batch, s)
                  : launch_paged_rows<64, false>(p, pl, batch, s);
    case 128:
      return e4m3 ? launch_paged_rows<128, true>(p, pl, batch, s)
                  : launch_paged_rows<128, false>(p, pl, batch, s);
    default:
      return e4m3 ? launch_paged_rows<256, true>(p, pl, batch, s)
                  : launch_paged_rows<256, false>(p, pl, batch, s);
  }
}
