// libiqkv: the paged 8-bit cache's bookkeeping (host) and the kernels that
// fill, read, share and move its pages.
//
// Values held: for a page of one kv head, code = e4m3(x * 2^-e) with the page's
// exponent e, so that the page's largest element lands in (224, 448] (or in
// [-40, 60] at the limits).  A power of two, because then decoding is exact in
// bfloat16, a page whose exponent grows moves its codes by whole binades (exact
// above e4m3's subnormals), and the attention can fold the scale into exponents.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <new>

#include "iq_paged.cuh"

namespace iq {
namespace paged {

// ------------------------------------------------------------------ append

// One contiguous run of pages of one entry: `rows` rows of the call, from row
// `row0`, go to positions pos .. pos + rows - 1 of the slot, which lie in pages
// page, page + 1, ...; the rows that the first page already holds come from
// page `from` (another one when the page was shared and is being copied).
struct Segment {
  int entry, slot, row0, rows, pos, page, from;
};
constexpr int kSegments = 256;  // per launch, by value

struct AppendParams {
  const uint16_t* keys;
  const uint16_t* values;
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scales;
  float* v_scales;
  int* table;
  unsigned* status;
  int heads, n, max_pages;
  Segment seg[kSegments];
};

// NaN: 0; infinity: the largest value of its sign.
__device__ __forceinline__ uint32_t drop_non_finite(uint32_t w) {
#pragma unroll
  for (int s = 0; s < 32; s += 16) {
    const uint32_t h = (w >> s) & 0x7FFFu;
    if (h >= 0x7F80u) w = (w & ~(0x7FFFu << s)) | ((h == 0x7F80u ? 0x7F7Fu : 0u) << s);
  }
  return w;
}
// The larger magnitude of both halves of eight bf16 values (they order as integers).
__device__ __forceinline__ uint32_t magnitude(const uint4& x) {
  const uint32_t m = 0x7FFF7FFFu;
  const uint32_t t = __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
  return max(t & 0xFFFFu, t >> 16);
}

// One CTA per (page of a segment, kv head, keys or values): 8 warps, a warp per
// row, a lane per 8 dims, the page's new rows (32 KB at most) held in registers
// between the maximum and the rounding, so every row is read once and written
// once.  Bound by HBM: 32 x 2 x 4096 rows and their read-back take 115 us, 805 MB
// at 7.0 TB/s (a copy's measured rate is 6.8); one row for each of 32 slots and
// its read-back 4.3 us.  Looking at every element for NaN and infinity before the
// maximum cost 143 us instead of 54; the maximum of the magnitudes tells both.
// The page ids of a segment come by value, so that no launch for table entries,
// and no read of the table, precedes it.
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ AppendParams p) {
  wait_for_last_kernel();
  const Segment sg = p.seg[blockIdx.z];
  const int k = blockIdx.x, h = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int off = sg.pos % kPage;                 // rows of the segment's first page before it
  const int begin = k == 0 ? off : 0;             // this page's new rows: [begin, end)
  const int end = min(kPage, off + sg.rows - k * kPage);
  if (end <= begin) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int page = sg.page + k, from = k == 0 ? sg.from : page;
  const long long at = static_cast<long long>(page) * p.heads + h, at_from = static_cast<long long>(from) * p.heads + h;
  uint8_t* codes = (is_v ? p.v_codes : p.k_codes) + at * kPageBytes + lane * 8;
  float* scales = is_v ? p.v_scales : p.k_scales;
  const int row0 = sg.row0 + k * kPage - off;     // the call's row of this page's row 0
  const uint16_t* in = (is_v ? p.values : p.keys) +
                       ((static_cast<long long>(sg.entry) * p.heads + h) * p.n + row0) * kHeadDim + lane * 8;

  uint4 x[8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = warp + 8 * i;
    x[i] = make_uint4(0, 0, 0, 0);
    if (r >= begin && r < end) x[i] = __ldcs(reinterpret_cast<const uint4*>(in + static_cast<long long>(r) * kHeadDim));
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, magnitude(x[i]));
  bool odd = top >= 0x7F80u;
  if (odd) {  // rare: make this thread's values finite, and find their maximum again
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = make_uint4(drop_non_finite(x[i].x), drop_non_finite(x[i].y), drop_non_finite(x[i].z), drop_non_finite(x[i].w));
      top = max(top, magnitude(x[i]));
    }
  }
  __shared__ uint32_t tops[8];
  top = __reduce_max_sync(0xFFFFFFFFu, top);
  if (lane == 0) tops[warp] = top;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, tops[i]);

  // top = 1.m * 2^x:  448 * 2^e = 1.75 * 2^(8+e) is reached from e = x - 8 on, or x - 7 where 1.m is above 1.75
  int e = kEMin;
  if (top >= 0x80u) e = static_cast<int>(top >> 7) - 127 - 8 + ((top & 0x7Fu) > 0x60u ? 1 : 0);
  odd |= e > kEMax;
  e = min(max(e, kEMin), kEMax);
  const int old = begin > 0 ? exponent_of(scales[at_from]) : e;
  e = max(e, old);
  const float inv = power2(-e);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int r = warp + 8 * i;
    if (r < begin || r >= end) continue;
    const uint32_t* w = reinterpret_cast<const uint32_t*>(&x[i]);
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) c[j] = e4m3x2(bf16_to_f32(w[j] & 0xFFFFu) * inv, __uint_as_float(w[j] & 0xFFFF0000u) * inv);
    *reinterpret_cast<uint2*>(codes + r * kHeadDim) = make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  }
  // rows that were there: moved to this page, rescaled to the grown exponent
  if (begin > 0 && (from != page || e > old)) {
    const uint8_t* src = (is_v ? p.v_codes : p.k_codes) + at_from * kPageBytes + lane * 8;
    const float f = power2(max(old - e, -126));
    for (int r = warp; r < begin; r += 8) {
      uint2 c = *reinterpret_cast<const uint2*>(src + r * kHeadDim);
      if (e > old) {
        uint32_t* w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 lo = f16x2_to_f32(e4m3x2_to_f16x2(w[j] & 0xFFFFu)), hi = f16x2_to_f32(e4m3x2_to_f16x2(w[j] >> 16));
          w[j] = e4m3x2(lo.x * f, lo.y * f) | e4m3x2(hi.x * f, hi.y * f) << 16;
        }
      }
      *reinterpret_cast<uint2*>(codes + r * kHeadDim) = c;
    }
  }
  // a page that is new to its slot: the rows behind are zero, so that whole
  // pages can enter matrix products before they are full
  if (begin == 0 || from != page)
    for (int r = warp; r < kPage; r += 8)
      if (r >= end) *reinterpret_cast<uint2*>(codes + r * kHeadDim) = make_uint2(0, 0);
  if (odd) atomicOr(p.status, IQ_STATUS_RANGE);
  __syncthreads();  // the old scale has been read by every thread
  if (threadIdx.x == 0) {
    scales[at] = power2(e);
    if (blockIdx.y == 0) p.table[static_cast<long long>(sg.slot) * p.max_pages + sg.pos / kPage + k] = page;
  }
}

// ------------------------------------------------------------------ read

struct ReadParams {
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const float* k_scales;
  const float* v_scales;
  const int* table;
  unsigned* status;
  uint16_t* keys;
  uint16_t* values;
  int heads, n, max_pages, pages;
  int slot[IQ_MAX_BATCH], start[IQ_MAX_BATCH], len[IQ_MAX_BATCH];
};

// A warp per row of (entry, kv head), keys and values; a lane per 8 dims.  Bound
// by HBM (32 x 2 x 4096 rows: 61 us, 403 MB at 6.6 TB/s).
__global__ void __launch_bounds__(256) paged_read_kernel(const __grid_constant__ ReadParams p) {
  wait_for_last_kernel();
  const int lane = threadIdx.x & 31, h = blockIdx.y, i = blockIdx.z;
  const long long row = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (row >= p.n) return;
  const long long t = p.start[i] + row;
  uint4 kv[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (t < p.len[i]) {
    const int page = page_in_pool(p.table[static_cast<long long>(p.slot[i]) * p.max_pages + t / kPage], p.pages, p.status);
    const long long at = static_cast<long long>(page) * p.heads + h;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint2 c = __ldcs(reinterpret_cast<const uint2*>((w ? p.v_codes : p.k_codes) + at * kPageBytes +
                                                            (t % kPage) * kHeadDim + lane * 8));
      const float s = (w ? p.v_scales : p.k_scales)[at];
      uint32_t* o = reinterpret_cast<uint32_t*>(&kv[w]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = f16x2_to_f32(e4m3x2_to_f16x2((j < 2 ? c.x : c.y) >> (16 * (j & 1)) & 0xFFFFu));
        o[j] = __float_as_uint(f.x * s) >> 16 | (__float_as_uint(f.y * s) & 0xFFFF0000u);  // exact in bf16
      }
    }
  }
  const long long to = ((static_cast<long long>(i) * p.heads + h) * p.n + row) * kHeadDim + lane * 8;
  __stcs(reinterpret_cast<uint4*>(p.keys + to), kv[0]);
  __stcs(reinterpret_cast<uint4*>(p.values + to), kv[1]);
}

// ------------------------------------------------------------------ fork

struct ForkParams {
  int* table;
  int max_pages, count;
  int src[IQ_MAX_BATCH], dst[IQ_MAX_BATCH], n[IQ_MAX_BATCH];  // n: pages of src
};

// A CTA takes 32 columns of the table for every pair: all sources are read
// before any row is written, so a permutation of slots needs no second table.
__global__ void __launch_bounds__(256) paged_fork_kernel(const __grid_constant__ ForkParams p) {
  wait_for_last_kernel();
  __shared__ int rows[IQ_MAX_BATCH][32];
  const int lane = threadIdx.x & 31, col = blockIdx.x * 32 + lane;
  for (int i = threadIdx.x >> 5; i < p.count; i += 8)
    if (col < p.n[i]) rows[i][lane] = p.table[static_cast<long long>(p.src[i]) * p.max_pages + col];
  __syncthreads();
  for (int i = threadIdx.x >> 5; i < p.count; i += 8)
    if (col < p.n[i]) p.table[static_cast<long long>(p.dst[i]) * p.max_pages + col] = rows[i][lane];
}

// ------------------------------------------------------------------ compact

// Runs of consecutive ids: pages src .. src + n - 1 become dst .. dst + n - 1
// (first: how many pages the runs before it hold), and table entries
// at .. at + n - 1 become id .. id + n - 1.
constexpr int kRuns = 320;
struct CompactParams {
  const uint8_t* k_from;
  const uint8_t* v_from;
  const float* ks_from;
  const float* vs_from;
  uint8_t* k_to;
  uint8_t* v_to;
  float* ks_to;
  float* vs_to;
  int* table;
  int heads, pages, page_runs, table_runs;  // pages: in all page runs
  int src[kRuns], dst[kRuns], first[kRuns];
  long long at[kRuns];
  int id[kRuns], n[kRuns];
};

// Blocks [0, pages * 2 * heads): 16 KB each, a page of one kv head, keys or
// values, and its scale.  The blocks behind them: a run of table entries each.
// Bound by HBM: 3818 pages of two kv heads in 73 us, 501 MB at 6.8 TB/s.
__global__ void __launch_bounds__(256) paged_compact_kernel(const __grid_constant__ CompactParams p) {
  wait_for_last_kernel();
  const long long copies = static_cast<long long>(p.pages) * 2 * p.heads;
  if (blockIdx.x >= copies) {
    const int r = static_cast<int>(blockIdx.x - copies);
    for (int j = threadIdx.x; j < p.n[r]; j += 256) p.table[p.at[r] + j] = p.id[r] + j;
    return;
  }
  const int part = static_cast<int>(blockIdx.x % (2 * p.heads)), j = static_cast<int>(blockIdx.x / (2 * p.heads));
  int lo = 0, hi = p.page_runs - 1;  // the last run that begins at or before page j
  while (lo < hi) {
    const int mid = (lo + hi + 1) / 2;
    if (p.first[mid] <= j) lo = mid;
    else hi = mid - 1;
  }
  const int k = j - p.first[lo], h = part >> 1;
  const bool is_v = part & 1;
  const long long from = static_cast<long long>(p.src[lo] + k) * p.heads + h, to = static_cast<long long>(p.dst[lo] + k) * p.heads + h;
  const uint4* s = reinterpret_cast<const uint4*>((is_v ? p.v_from : p.k_from) + from * kPageBytes);
  uint4* d = reinterpret_cast<uint4*>((is_v ? p.v_to : p.k_to) + to * kPageBytes);
  uint4 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = __ldcs(s + threadIdx.x + 256 * i);
#pragma unroll
  for (int i = 0; i < 4; ++i) __stcs(d + threadIdx.x + 256 * i, x[i]);
  if (threadIdx.x == 0) (is_v ? p.vs_to : p.ks_to)[to] = (is_v ? p.vs_from : p.ks_from)[from];
}
static_assert(kPageBytes == 4 * 256 * 16, "four 16-byte pieces per thread");

// ------------------------------------------------------------------ bookkeeping

int check_slots(const iq_paged* c, const int32_t* slots, int n, bool distinct) {
  if (n < 0 || n > IQ_MAX_BATCH) return fail(IQ_ERR_INVALID_ARG, "bad number of slots");
  if (!slots) return n <= c->slots ? IQ_OK : fail(IQ_ERR_INVALID_ARG, "more entries than slots");
  bool seen[IQ_MAX_BATCH] = {};
  for (int i = 0; i < n; ++i) {
    if (slots[i] < 0 || slots[i] >= c->slots) return fail(IQ_ERR_INVALID_ARG, "slot out of range");
    if (distinct && seen[slots[i]]) return fail(IQ_ERR_INVALID_ARG, "a slot is given twice");
    seen[slots[i]] = true;
  }
  return IQ_OK;
}

namespace {

int32_t* row_of(const iq_paged* c, int slot) { return c->table_host + static_cast<long long>(slot) * c->max_pages; }

int take_page(iq_paged* c) {  // the lowest free id; there is one
  int p = c->first_free;
  while (c->refs[p] != 0) ++p;
  c->refs[p] = 1;
  c->first_free = p + 1;
  --c->free_pages;
  return p;
}
void drop_page(iq_paged* c, int p) {
  if (--c->refs[p] > 0) return;
  ++c->free_pages;
  c->first_free = std::min(c->first_free, p);
}
void drop_from(iq_paged* c, int slot, int keep) {  // the slot's pages from index `keep` on
  int32_t* row = row_of(c, slot);
  for (int j = pages_for(c->lens[slot]) - 1; j >= keep; --j) drop_page(c, row[j]);
}

// What an append of the entries needs, checked without a change.
int check_append(iq_paged* c, const void* keys, const void* values, int n, const int32_t* slots, const int32_t* counts,
                 int n_slots) {
  int st = iq_paged_check(c);
  if (st != IQ_OK) return st;
  st = check_slots(c, slots, n_slots, true);
  if (st != IQ_OK) return st;
  if (n < 0) return fail(IQ_ERR_INVALID_ARG, "negative token count");
  if (n > 0 && n_slots > 0) {
    if (!keys || !values) return fail(IQ_ERR_INVALID_ARG, "null keys/values");
    if (misaligned(keys) || misaligned(values)) return fail(IQ_ERR_INVALID_ARG, "keys/values not 16-byte aligned");
  }
  if (counts)
    for (int i = 0; i < n_slots; ++i)
      if (counts[i] < 0 || counts[i] > n) return fail(IQ_ERR_INVALID_ARG, "counts[i] outside [0, n]");
  long long need = 0;
  for (int i = 0; i < n_slots; ++i) {
    const int s = slot_of(slots, i);
    const long long total = static_cast<long long>(c->lens[s]) + (counts ? counts[i] : n);
    if (total > static_cast<long long>(c->max_pages) * kPage) return fail(IQ_ERR_CAPACITY, "append past a slot's max_pages");
    need += pages_for(total) - pages_for(c->lens[s]);
  }
  for (int i = 0; i < n_slots; ++i) {  // shared last pages are copied, whoever else goes on in them
    const int s = slot_of(slots, i);
    if ((counts ? counts[i] : n) > 0 && c->lens[s] % kPage && c->refs[row_of(c, s)[c->lens[s] / kPage]] > 1) ++need;
  }
  return need <= c->free_pages ? IQ_OK : fail(IQ_ERR_CAPACITY, "the pool has too few free pages");
}

// The checked append: takes pages, launches, and puts everything back if a launch
// fails.  What changes a page or a table entry that a slot lives on (a run that
// begins in a partly full page: it rescales the rows there, or moves them to a copy
// and names that one) goes with the last launch; the launches before it write
// pages that are still free to anyone who looks at the host's arrays.
int do_append(iq_paged* c, const void* keys, const void* values, int n, const int32_t* slots, const int32_t* counts,
              int n_slots, iq_stream_t stream) {
  AppendParams p;
  p.keys = static_cast<const uint16_t*>(keys);
  p.values = static_cast<const uint16_t*>(values);
  p.k_codes = c->k_codes;
  p.v_codes = c->v_codes;
  p.k_scales = c->k_scales;
  p.v_scales = c->v_scales;
  p.table = c->table;
  p.status = c->status;
  p.heads = c->kv_heads;
  p.n = n;
  p.max_pages = c->max_pages;
  int segs = 0, widest = 0, done = 0, begun = 0;
  Segment last_ones[IQ_MAX_BATCH];  // one per entry at most
  static_assert(IQ_MAX_BATCH <= kSegments, "they fit one launch");
  int was[IQ_MAX_BATCH];  // the shared page that entry i's own copy replaced
  cudaError_t err = cudaSuccess;
  auto launch = [&]() {
    if (segs && err == cudaSuccess) {
      void* args[] = {&p};
      err = launch_after(reinterpret_cast<const void*>(&paged_append_kernel), dim3(widest, 2 * c->kv_heads, segs), 256, 0,
                         static_cast<cudaStream_t>(stream), args);
    }
    segs = widest = 0;
  };
  auto add = [&](const Segment& sg) {
    p.seg[segs++] = sg;
    widest = std::max(widest, (sg.pos % kPage + sg.rows + kPage - 1) / kPage);
  };
  for (; done < n_slots && err == cudaSuccess; ++done) {
    const int s = slot_of(slots, done), len = c->lens[s], cnt = counts ? counts[done] : n;
    was[done] = -1;
    if (cnt == 0) continue;
    int32_t* row = row_of(c, s);
    const int last = pages_for(static_cast<long long>(len) + cnt);
    int j = len / kPage;
    int from = -1;
    if (len % kPage) {  // the last page goes on
      from = row[j];
      if (c->refs[from] > 1) {  // let go of only after the launch: other entries read it there too
        was[done] = from;
        row[j] = take_page(c);
      }
    }
    for (int k = pages_for(len); k < last; ++k) row[k] = take_page(c);
    for (int pos = len; j < last;) {
      int m = 1;
      while (j + m < last && row[j + m] == row[j] + m) ++m;
      const int stop = std::min((j + m) * static_cast<long long>(kPage), static_cast<long long>(len) + cnt);
      const Segment sg{done, s, pos - len, stop - pos, pos, row[j], from >= 0 ? from : row[j]};
      if (from >= 0) {
        last_ones[begun++] = sg;
      } else {
        if (segs == kSegments) launch();
        add(sg);
      }
      pos = stop;
      j += m;
      from = -1;
    }
  }
  if (segs + begun > kSegments) launch();
  for (int i = 0; i < begun; ++i) add(last_ones[i]);
  launch();
  if (err != cudaSuccess) {
    for (int i = 0; i < done; ++i) {
      const int s = slot_of(slots, i), len = c->lens[s], cnt = counts ? counts[i] : n;
      if (cnt == 0) continue;
      int32_t* row = row_of(c, s);
      for (int k = pages_for(len); k < pages_for(static_cast<long long>(len) + cnt); ++k) drop_page(c, row[k]);
      if (was[i] >= 0) {
        drop_page(c, row[len / kPage]);
        row[len / kPage] = was[i];
      }
    }
    return cuda_fail(err, "paged append");
  }
  for (int i = 0; i < n_slots; ++i) {
    if (was[i] >= 0) drop_page(c, was[i]);
    c->lens[slot_of(slots, i)] += counts ? counts[i] : n;
  }
  return IQ_OK;
}

}  // namespace
}  // namespace paged
}  // namespace iq

using namespace iq;
using namespace iq::paged;

extern "C" {

int iq_paged_debug_fail(int launch) {
  clear_error();
  launch_to_fail = launch < 0 ? -1 : launch;
  return IQ_OK;
}

int iq_paged_debug_stall(void) {
  clear_error();
  stall_next = true;
  return IQ_OK;
}

int iq_paged_bytes(int slots, int kv_heads, int head_dim, int pages, int max_pages, size_t out_bytes[6]) {
  clear_error();
  if (!out_bytes) return fail(IQ_ERR_INVALID_ARG, "null out_bytes");
  if (slots <= 0 || kv_heads <= 0 || head_dim <= 0 || pages <= 0 || max_pages <= 0)
    return fail(IQ_ERR_INVALID_ARG, "slots, kv_heads, head_dim, pages and max_pages must be positive");
  if (head_dim != kHeadDim) return fail(IQ_ERR_UNSUPPORTED, "only head_dim 256 is built");
  if (slots > IQ_MAX_BATCH) return fail(IQ_ERR_UNSUPPORTED, "slots above IQ_MAX_BATCH");
  if (kv_heads > 1024) return fail(IQ_ERR_UNSUPPORTED, "kv_heads above 1024");
  if (static_cast<long long>(pages) * kv_heads * kPage >= (1LL << 31))
    return fail(IQ_ERR_UNSUPPORTED, "pages * kv_heads * IQ_PAGE exceeds 2^31");
  if (max_pages > (1 << 25) - 1) return fail(IQ_ERR_UNSUPPORTED, "max_pages * IQ_PAGE exceeds 2^31");
  const size_t rows = static_cast<size_t>(pages) * kv_heads;
  out_bytes[0] = out_bytes[1] = rows * kPageBytes;
  out_bytes[2] = out_bytes[3] = rows * 4;
  out_bytes[4] = static_cast<size_t>(slots) * max_pages * 4;
  out_bytes[5] = IQ_WORKSPACE_HEAD_BYTES;
  return IQ_OK;
}

int iq_paged_check(const iq_paged* c) {
  clear_error();
  if (!c) return fail(IQ_ERR_INVALID_ARG, "null cache");
  size_t bytes[6];
  const int st = iq_paged_bytes(c->slots, c->kv_heads, c->head_dim, c->pages, c->max_pages, bytes);
  if (st != IQ_OK) return st;
  const void* ptrs[6] = {c->k_codes, c->v_codes, c->k_scales, c->v_scales, c->table, c->status};
  for (const void* ptr : ptrs) {
    if (!ptr) return fail(IQ_ERR_INVALID_ARG, "null cache buffer");
    if (misaligned(ptr)) return fail(IQ_ERR_INVALID_ARG, "cache buffer not 16-byte aligned");
  }
  if (!c->lens || !c->table_host || !c->refs) return fail(IQ_ERR_INVALID_ARG, "null host array");
  if (c->free_pages < 0 || c->free_pages > c->pages || c->first_free < 0 || c->first_free > c->pages)
    return fail(IQ_ERR_INVALID_ARG, "free_pages or first_free outside the pool");
  for (int s = 0; s < c->slots; ++s)
    if (c->lens[s] < 0 || c->lens[s] > static_cast<long long>(c->max_pages) * kPage)
      return fail(IQ_ERR_INVALID_ARG, "lens[s] outside [0, max_pages * IQ_PAGE]");
  return IQ_OK;
}

int iq_paged_alloc(iq_paged* c, int slots, int kv_heads, int head_dim, int pages, int max_pages, void* const buffers[6],
                   int32_t* lens, int32_t* table_host, int32_t* refs) {
  clear_error();
  if (!c || !buffers || !lens || !table_host || !refs) return fail(IQ_ERR_INVALID_ARG, "null cache, buffers or host array");
  size_t bytes[6];
  int st = iq_paged_bytes(slots, kv_heads, head_dim, pages, max_pages, bytes);
  if (st != IQ_OK) return st;
  iq_paged d;
  std::memset(&d, 0, sizeof(d));
  d.slots = slots;
  d.kv_heads = kv_heads;
  d.head_dim = head_dim;
  d.pages = d.free_pages = pages;
  d.max_pages = max_pages;
  d.k_codes = static_cast<uint8_t*>(buffers[0]);
  d.v_codes = static_cast<uint8_t*>(buffers[1]);
  d.k_scales = static_cast<float*>(buffers[2]);
  d.v_scales = static_cast<float*>(buffers[3]);
  d.table = static_cast<int32_t*>(buffers[4]);
  d.status = static_cast<uint32_t*>(buffers[5]);
  d.lens = lens;
  d.table_host = table_host;
  d.refs = refs;
  std::memset(lens, 0, sizeof(int32_t) * slots);
  st = iq_paged_check(&d);
  if (st != IQ_OK) return st;
  std::memset(table_host, 0, bytes[4]);
  std::memset(refs, 0, sizeof(int32_t) * pages);
  *c = d;
  return IQ_OK;
}

int iq_paged_append(iq_paged* c, const void* keys, const void* values, int n, const int32_t* slots,
                    const int32_t* counts, int n_slots, iq_stream_t stream) {
  const int st = check_append(c, keys, values, n, slots, counts, n_slots);
  return st != IQ_OK ? st : do_append(c, keys, values, n, slots, counts, n_slots, stream);
}

int iq_paged_append_attend(iq_paged* c, const void* keys, const void* values, int n, const void* q, int q_heads,
                           int n_queries, const int32_t* slots, const int32_t* counts, int n_slots, float scale,
                           int causal, int window, int sinks, void* out, int out_f32, void* workspace,
                           size_t workspace_bytes, iq_stream_t stream) {
  int st = check_append(c, keys, values, n, slots, counts, n_slots);
  if (st != IQ_OK) return st;
  if (counts && n != n_queries) return fail(IQ_ERR_INVALID_ARG, "counts need as many rows as queries");
  st = check_attend(c, q, q_heads, n_queries, slots, counts, n_slots, n, scale, causal, window, sinks, out, out_f32, workspace,
                    workspace_bytes);
  if (st != IQ_OK) return st;
  st = do_append(c, keys, values, n, slots, counts, n_slots, stream);
  if (st != IQ_OK) return st;
  return iq_paged_attend(c, q, q_heads, n_queries, slots, counts, n_slots, scale, causal, window, sinks, out, out_f32,
                         workspace, workspace_bytes, stream);
}

int iq_paged_read(const iq_paged* c, const int32_t* slots, const int32_t* start, int n_slots, int n, void* keys_out,
                  void* values_out, iq_stream_t stream) {
  int st = iq_paged_check(c);
  if (st != IQ_OK) return st;
  st = check_slots(c, slots, n_slots, false);
  if (st != IQ_OK) return st;
  if (n < 0) return fail(IQ_ERR_INVALID_ARG, "negative row count");
  if (n == 0 || n_slots == 0) return IQ_OK;
  if (!start || !keys_out || !values_out) return fail(IQ_ERR_INVALID_ARG, "null start/keys_out/values_out");
  if (misaligned(keys_out) || misaligned(values_out)) return fail(IQ_ERR_INVALID_ARG, "outputs not 16-byte aligned");
  ReadParams p;
  std::memset(&p, 0, sizeof(p));
  p.k_codes = c->k_codes;
  p.v_codes = c->v_codes;
  p.k_scales = c->k_scales;
  p.v_scales = c->v_scales;
  p.table = c->table;
  p.status = c->status;
  p.keys = static_cast<uint16_t*>(keys_out);
  p.values = static_cast<uint16_t*>(values_out);
  p.heads = c->kv_heads;
  p.n = n;
  p.max_pages = c->max_pages;
  p.pages = c->pages;
  for (int i = 0; i < n_slots; ++i) {
    if (start[i] < 0) return fail(IQ_ERR_INVALID_ARG, "negative start");
    p.slot[i] = slot_of(slots, i);
    p.start[i] = start[i];
    p.len[i] = c->lens[p.slot[i]];
  }
  void* args[] = {&p};
  IQ_CUDA(launch_after(reinterpret_cast<const void*>(&paged_read_kernel), dim3((n + 7) / 8, c->kv_heads, n_slots), 256, 0,
                       static_cast<cudaStream_t>(stream), args));
  const size_t bytes = static_cast<size_t>(n_slots) * c->kv_heads * n * kHeadDim * 2;
  launched_outputs(stream, {keys_out, bytes}, {values_out, bytes});
  return IQ_OK;
}

int iq_paged_trim(iq_paged* c, const int32_t* slots, const int32_t* n, int n_slots, int32_t* trimmed) {
  int st = iq_paged_check(c);
  if (st != IQ_OK) return st;
  st = check_slots(c, slots, n_slots, true);
  if (st != IQ_OK) return st;
  if (!n) return fail(IQ_ERR_INVALID_ARG, "null counts");
  for (int i = 0; i < n_slots; ++i)
    if (n[i] < 0) return fail(IQ_ERR_INVALID_ARG, "negative trim count");
  for (int i = 0; i < n_slots; ++i) {
    const int s = slot_of(slots, i), t = std::min(n[i], c->lens[s]);
    drop_from(c, s, pages_for(c->lens[s] - t));
    c->lens[s] -= t;
    if (trimmed) trimmed[i] = t;
  }
  return IQ_OK;
}

int iq_paged_free(iq_paged* c, const int32_t* slots, int n_slots) {
  int32_t all[IQ_MAX_BATCH];
  std::fill(all, all + IQ_MAX_BATCH, INT32_MAX);
  return iq_paged_trim(c, slots, all, n_slots, nullptr);
}

int iq_paged_fork(iq_paged* c, const int32_t* src, const int32_t* dst, int count, iq_stream_t stream) {
  int st = iq_paged_check(c);
  if (st != IQ_OK) return st;
  if (count == 0) return IQ_OK;
  if (!src || !dst) return fail(IQ_ERR_INVALID_ARG, "null src/dst");
  st = check_slots(c, src, count, false);
  if (st != IQ_OK) return st;
  st = check_slots(c, dst, count, true);
  if (st != IQ_OK) return st;
  ForkParams p;
  p.table = c->table;
  p.max_pages = c->max_pages;
  p.count = count;
  int widest = 0;
  long long total = 0;
  for (int i = 0; i < count; ++i) {
    p.src[i] = src[i];
    p.dst[i] = dst[i];
    p.n[i] = pages_for(c->lens[src[i]]);
    widest = std::max(widest, p.n[i]);
    total += p.n[i];
  }
  // the sources' rows as they were: a source may be another pair's dst
  int32_t* rows = new (std::nothrow) int32_t[total + 1];
  if (!rows) return fail(IQ_ERR_CAPACITY, "no host memory for the forked rows");
  if (widest > 0) {
    void* args[] = {&p};
    const cudaError_t err =
        launch_after(reinterpret_cast<const void*>(&paged_fork_kernel), dim3((widest + 31) / 32), 256, 0, static_cast<cudaStream_t>(stream), args);
    if (err != cudaSuccess) {
      delete[] rows;
      return cuda_fail(err, "paged fork");
    }
  }
  int32_t lens[IQ_MAX_BATCH];
  int32_t* at = rows;
  for (int i = 0, same = 0; i < count; ++i) {  // the new holders first, so that no page is free in between
    std::memcpy(at, row_of(c, src[i]), sizeof(int32_t) * p.n[i]);
    ++same;
    if (i + 1 == count || src[i + 1] != src[i]) {  // a run of pairs with one source
      for (int j = 0; j < p.n[i]; ++j) c->refs[at[j]] += same;
      same = 0;
    }
    lens[i] = c->lens[src[i]];
    at += p.n[i];
  }
  for (int i = 0; i < count; ++i) drop_from(c, dst[i], 0);
  at = rows;
  for (int i = 0; i < count; ++i) {
    std::memcpy(row_of(c, dst[i]), at, sizeof(int32_t) * p.n[i]);
    c->lens[dst[i]] = lens[i];
    at += p.n[i];
  }
  delete[] rows;
  return IQ_OK;
}

int iq_paged_compact(const iq_paged* src, iq_paged* dst, iq_stream_t stream) {
  int st = iq_paged_check(src);
  if (st != IQ_OK) return st;
  st = iq_paged_check(dst);
  if (st != IQ_OK) return st;
  if (src->slots != dst->slots || src->kv_heads != dst->kv_heads || src->head_dim != dst->head_dim)
    return fail(IQ_ERR_INVALID_ARG, "src and dst shapes differ");
  if (src->k_codes == dst->k_codes || src->v_codes == dst->v_codes || src->k_codes == dst->v_codes ||
      src->v_codes == dst->k_codes || src->table == dst->table || src->k_scales == dst->k_scales ||
      src->v_scales == dst->v_scales || src->lens == dst->lens || src->table_host == dst->table_host || src->refs == dst->refs)
    return fail(IQ_ERR_INVALID_ARG, "src and dst share a buffer");
  for (int s = 0; s < src->slots; ++s)
    if (pages_for(src->lens[s]) > dst->max_pages) return fail(IQ_ERR_CAPACITY, "dst max_pages below a source slot's pages");
  if (src->pages - src->free_pages > dst->pages) return fail(IQ_ERR_CAPACITY, "dst has too few pages");
  int32_t* to = new (std::nothrow) int32_t[src->pages];
  if (!to) return fail(IQ_ERR_CAPACITY, "no host memory for the page map");
  std::fill(to, to + src->pages, -1);
  CompactParams p;
  p.k_from = src->k_codes;
  p.v_from = src->v_codes;
  p.ks_from = src->k_scales;
  p.vs_from = src->v_scales;
  p.k_to = dst->k_codes;
  p.v_to = dst->v_codes;
  p.ks_to = dst->k_scales;
  p.vs_to = dst->v_scales;
  p.table = dst->table;
  p.heads = dst->kv_heads;
  p.pages = p.page_runs = p.table_runs = 0;
  int run_page = 0, run_len = 0;  // the last page run: its first source page, its length
  cudaError_t err = cudaSuccess;
  bool begun = false;  // a launch has written dst's pages
  auto launch = [&]() {
    const long long blocks = static_cast<long long>(p.pages) * 2 * p.heads + p.table_runs;
    if (blocks && err == cudaSuccess) {
      void* args[] = {&p};
      err = launch_after(reinterpret_cast<const void*>(&paged_compact_kernel), dim3(static_cast<unsigned>(blocks)), 256, 0,
                         static_cast<cudaStream_t>(stream), args);
      begun |= err == cudaSuccess;
    }
    p.pages = p.page_runs = p.table_runs = run_len = 0;
  };
  int used = 0;
  for (int s = 0; s < src->slots; ++s) {
    const int32_t* row = row_of(src, s);
    for (int j = 0; j < pages_for(src->lens[s]); ++j) {
      const int page = row[j];
      const bool fresh = to[page] < 0;
      if (p.page_runs == kRuns || p.table_runs == kRuns) launch();
      if (fresh) {
        to[page] = used++;
        if (run_len > 0 && page == run_page + run_len) {
          ++run_len;
        } else {
          p.src[p.page_runs] = run_page = page;
          p.dst[p.page_runs] = to[page];
          p.first[p.page_runs++] = p.pages;
          run_len = 1;
        }
        ++p.pages;
      }
      const int t = p.table_runs - 1;
      const long long at = static_cast<long long>(s) * dst->max_pages + j;
      if (t >= 0 && p.at[t] + p.n[t] == at && p.id[t] + p.n[t] == to[page] && j > 0) {
        ++p.n[t];
      } else {
        p.at[t + 1] = at;
        p.id[t + 1] = to[page];
        p.n[t + 1] = 1;
        ++p.table_runs;
      }
    }
  }
  launch();
  if (err != cudaSuccess) {
    delete[] to;
    if (begun) {  // what dst held is lost
      std::memset(dst->lens, 0, sizeof(int32_t) * dst->slots);
      std::memset(dst->refs, 0, sizeof(int32_t) * dst->pages);
      dst->free_pages = dst->pages;
      dst->first_free = 0;
    }
    return cuda_fail(err, "paged compact");
  }
  std::memset(dst->refs, 0, sizeof(int32_t) * dst->pages);
  for (int s = 0; s < src->slots; ++s) {
    const int32_t* row = row_of(src, s);
    int32_t* new_row = row_of(dst, s);
    for (int j = 0; j < pages_for(src->lens[s]); ++j) {
      new_row[j] = to[row[j]];
      ++dst->refs[new_row[j]];
    }
    dst->lens[s] = src->lens[s];
  }
  dst->free_pages = dst->pages - used;
  dst->first_free = used;
  delete[] to;
  return IQ_OK;
}

}  // extern "C"
