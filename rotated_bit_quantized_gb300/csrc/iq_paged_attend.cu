// libiqkv: attention over the paged 8-bit cache.
//
// Two kernels.  Calls with at most 32 query rows per kv head (decode, verify)
// run paged_split_kernel (its CTAs: iq_paged_split.cuh): the keys are the matrix
// products' M dimension, the codes go from HBM through shared memory into tcgen05.mma
// untouched, and the keys of all (slot, kv head) pairs are split evenly over the GPU.
// More rows run paged_prefill_kernel (iq_paged_prefill.cu).
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <cstring>
#include <mutex>

#include "iq_paged_split.cuh"

namespace iq {
namespace paged {

// ------------------------------------------------------------------ decode and verify

template <int NR>
__global__ void __launch_bounds__(split::Shape<NR>::kThreads, 1) paged_split_kernel(const __grid_constant__ AttendParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzled operands need it; no room to align by hand
  split::run<NR>(p, {0, p.entries, p.cost, p.total, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x)}, smem);
}

// Joins the partial results of the units that ranges cut, in the order of the
// ranges.  CTA (g, y) takes `rows` rows of the unit that range g's end cuts, 8 /
// rows warps each, a lane per 8 dims: one row where the partials are many
// (eight warps share them, then add up through shared memory), eight where the
// rows are.  Latency: 5 us for 32 partials of 16 rows, 11 us for 150 cut units of
// 128 rows (39 MB, L2).
struct JoinParams {
  const float* part_o;
  const float2* part_ml;
  const Cut* cuts;
  void* out;
  int out_f32, heads, rep, nq, unit_rows, rows;
  short entry[IQ_MAX_BATCH];
  int count[IQ_MAX_BATCH];
};
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ JoinParams p) {
  wait_for_last_kernel();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.last < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, share = 8 / p.rows;
  const int x = blockIdx.y * p.rows + warp / share, r = cut.z * p.unit_rows + x, j = r / p.rep;
  const bool live = x < p.unit_rows && r < p.count[cut.e] * p.rep;
  auto row = [&](int g) { return static_cast<long long>(g == static_cast<int>(blockIdx.x) ? cut.slot : 2 * g) * p.unit_rows + x; };
  __shared__ float part[8][kHeadDim + 2];
  float m = kUnset, sum = 0.0f, o[8] = {};
  if (live) {
    for (int g = blockIdx.x + lane; g <= cut.last; g += 32) m = fmaxf(m, __ldcg(&p.part_ml[row(g)]).x);  // every lane a partial
#pragma unroll
    for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, d));
#pragma unroll 4
    for (int g = blockIdx.x + warp % share; g <= cut.last; g += share) {
      const long long i = row(g);
      const float2 ml = __ldcg(&p.part_ml[i]);
      const float4* v = reinterpret_cast<const float4*>(p.part_o + i * kHeadDim + lane * 8);
      const float4 v0 = __ldcg(v), v1 = __ldcg(v + 1);
      const float f = ex2_approx(ml.x - m);
      sum = fmaf(f, ml.y, sum);
      o[0] = fmaf(f, v0.x, o[0]), o[1] = fmaf(f, v0.y, o[1]), o[2] = fmaf(f, v0.z, o[2]), o[3] = fmaf(f, v0.w, o[3]);
      o[4] = fmaf(f, v1.x, o[4]), o[5] = fmaf(f, v1.y, o[5]), o[6] = fmaf(f, v1.z, o[6]), o[7] = fmaf(f, v1.w, o[7]);
    }
  }
  if (share > 1) {
#pragma unroll
    for (int d = 0; d < 8; ++d) part[warp][d * 32 + lane] = o[d];
    if (lane == 0) part[warp][kHeadDim] = sum;
    __syncthreads();
    if (warp != 0) return;
    for (int w = 1; w < 8; ++w) {
#pragma unroll
      for (int d = 0; d < 8; ++d) o[d] += part[w][d * 32 + lane];
      sum += part[w][kHeadDim];
    }
  }
  if (!live) return;
  const long long to = static_cast<long long>((p.entry[cut.e] * p.heads + cut.h) * p.rep + r - j * p.rep) * p.nq + j;
  store_out8(p.out, p.out_f32, to * kHeadDim + lane * 8, o, sum == 0.0f ? 0.0f : 1.0f / sum);
}

// Rows of entries without a key: zeros.
struct ZeroParams {
  void* out;
  int q_heads, nq, out_bytes;
  short entry[IQ_MAX_BATCH];
  int count[IQ_MAX_BATCH];
};
__global__ void __launch_bounds__(256) paged_zero_kernel(const __grid_constant__ ZeroParams p) {
  wait_for_last_kernel();
  const int pieces = kHeadDim * p.out_bytes / 16;
  const long long n = static_cast<long long>(p.count[blockIdx.y]) * pieces;
  for (int h = 0; h < p.q_heads; ++h) {
    uint4* out = static_cast<uint4*>(p.out) + (static_cast<long long>(p.entry[blockIdx.y]) * p.q_heads + h) * p.nq * pieces;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) out[i] = make_uint4(0, 0, 0, 0);
  }
}

namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// Up to 32 query rows per kv head the split kernel, beyond the prefill kernel.
// Measured over 8 x 131072 tokens (and 4 x 16384, 1 x 4096 with 8 kv heads): 32 rows
// 173.5 us split (28.3, 20.3); 33 rows 194.6 prefill (29.4, 21.0); a split kernel of
// 64 rows, which spills and stores its weights byte by byte, took 255.5 us at 33
// rows (37.7, 24.7) and 265.6 at 64 (45.9, 33.0), the prefill kernel 197.0 (31.2, 22.7).
constexpr int kMaxSplitRows = 32;
int unit_rows(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : rows <= kMaxSplitRows ? 32 : 128; }

// The tiles of one head of an entry whose units hold `each` rows, and how many units those are.
long long tiles_of_entry(int len, int count, int rep, int each, int causal, int window, int sinks, int* units) {
  long long n = 0;
  const int all = count * rep;
  *units = 0;
  for (long long r = 0; r < all; r += each, ++*units)
    n += tiles_of(len, len - count + static_cast<int>(r) / rep, len - count + (static_cast<int>(std::min<long long>(r + each, all)) - 1) / rep,
                  causal, window, sinks).n;
  return n;
}
// What a unit's beginning and end take, in tiles, where a range has 8 tiles or
// more (shorter ones are left at a tile's grain).  Measured, 0 / 1 / 2 / 4 / 6:
// 4 x 1531 prompts - / 137 / 131 / 138 / 145 us; batched decode under a window
// of 4096 - / 34.5 / 33.9 / 32.9 / - us.
constexpr int unit_cost(int each) { return each == 128 ? 2 : 4; }

template <int NR>
cudaError_t launch_split(const AttendParams& p, int grid, cudaStream_t stream) {
  using C = split::Shape<NR>;
  static std::atomic<uint64_t> seen{0};
  const void* kernel = reinterpret_cast<const void*>(&paged_split_kernel<NR>);
  const cudaError_t e = allow_smem(kernel, C::kSmem, seen);
  void* args[] = {const_cast<AttendParams*>(&p)};
  return e == cudaSuccess ? launch_after(kernel, dim3(grid), C::kThreads, C::kSmem, stream, args) : e;
}

}  // namespace

thread_local int launch_to_fail = -1;
thread_local bool stall_next = false;

cudaError_t launch_after(const void* kernel, dim3 grid, int threads, int smem, cudaStream_t stream, void** args) {
  if (launch_to_fail >= 0 && launch_to_fail-- == 0) return cudaErrorLaunchFailure;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, kernel, args);
}

cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& seen) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && seen.load(std::memory_order_relaxed) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) seen.fetch_or(1ull << dev, std::memory_order_relaxed);
  return e;
}

bool code_map(CUtensorMap* map, const uint8_t* codes, long long rows, int box_rows) {
  const cuuint64_t dims[2] = {kHeadDim, static_cast<cuuint64_t>(rows)}, strides[1] = {kHeadDim};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, unit[2] = {1, 1};
  auto fn = encode_fn();
  return fn && fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(codes), dims, strides, box, unit,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int store_zeros(const iq_paged* c, int q_heads, int n_queries, const int32_t* slots, const int32_t* counts, int n_slots, void* out,
                int out_f32, iq_stream_t stream) {
  ZeroParams z;
  z.out = out;
  z.q_heads = q_heads;
  z.nq = n_queries;
  z.out_bytes = out_f32 ? 4 : 2;
  int n = 0, most = 0;
  for (int i = 0; i < n_slots; ++i) {
    const int count = counts ? counts[i] : n_queries;
    if (count == 0 || c->lens[slot_of(slots, i)] > 0) continue;
    z.entry[n] = static_cast<short>(i);
    z.count[n++] = count;
    most = std::max(most, count);
  }
  if (n == 0) return IQ_OK;
  void* args[] = {&z};
  IQ_CUDA(launch_after(reinterpret_cast<const void*>(&paged_zero_kernel), dim3(std::min(64, (most + 7) / 8), n), 256, 0,
                       static_cast<cudaStream_t>(stream), args));
  launched_outputs(stream, {out, static_cast<size_t>(n_slots) * q_heads * n_queries * kHeadDim * (out_f32 ? 4 : 2)});
  return IQ_OK;
}

int check_attend(const iq_paged* c, const void* q, int q_heads, int n_queries, const int32_t* slots,
                 const int32_t* counts, int n_slots, int added, float scale, int causal, int window, int sinks,
                 const void* out, int out_f32, const void* workspace, size_t workspace_bytes) {
  size_t need = 0;
  int st = iq_paged_attend_workspace(c, q_heads, n_queries, n_slots, &need);
  if (st != IQ_OK) return st;
  st = check_slots(c, slots, n_slots, false);
  if (st != IQ_OK) return st;
  if (causal != 0 && causal != 1) return fail(IQ_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (window < 0 || sinks < 0) return fail(IQ_ERR_INVALID_ARG, "negative window or sinks");
  if (window > 0 && !causal) return fail(IQ_ERR_INVALID_ARG, "a window needs causal attention");
  if (sinks > 0 && window == 0) return fail(IQ_ERR_INVALID_ARG, "sinks need a window");
  if (out_f32 != 0 && out_f32 != 1) return fail(IQ_ERR_INVALID_ARG, "out_f32 must be 0 or 1");
  if (!(scale - scale == 0.0f)) return fail(IQ_ERR_INVALID_ARG, "scale is not finite");
  if (counts)
    for (int i = 0; i < n_slots; ++i)
      if (counts[i] < 0 || counts[i] > n_queries) return fail(IQ_ERR_INVALID_ARG, "counts[i] outside [0, n_queries]");
  if (n_slots == 0 || n_queries == 0) return IQ_OK;
  if (!q || !out) return fail(IQ_ERR_INVALID_ARG, "null q/out");
  if (misaligned(q) || misaligned(out)) return fail(IQ_ERR_INVALID_ARG, "q/out not 16-byte aligned");
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return fail(IQ_ERR_WORKSPACE, "workspace missing or too small");
    if (misaligned(workspace, 256)) return fail(IQ_ERR_WORKSPACE, "workspace not 256-byte aligned");
  }
  // the slots of all units stay below 2^31: told by a bound, counted where that passes it
  const int rep = q_heads / c->kv_heads, each = unit_rows(n_queries * rep);
  for (int exact = 0; exact < 2; ++exact) {
    long long total = 0;
    for (int i = 0; i < n_slots; ++i) {
      const int count = counts ? counts[i] : n_queries, len = c->lens[slot_of(slots, i)] + (counts && added ? counts[i] : added);
      if (len <= 0 || count <= 0) continue;
      int units = (count * rep + each - 1) / each;
      const long long tiles = exact ? tiles_of_entry(len, count, rep, each, causal, window, sinks, &units)
                                    : static_cast<long long>(units) * (len / kTile + 1);
      total += (tiles + static_cast<long long>(units) * unit_cost(each)) * c->kv_heads;
    }
    if (total < (1LL << 31)) return IQ_OK;
  }
  return fail(IQ_ERR_UNSUPPORTED, "too many queries and keys for one call");
}

}  // namespace paged
}  // namespace iq

using namespace iq;
using namespace iq::paged;

extern "C" {

int iq_paged_attend_workspace(const iq_paged* c, int q_heads, int n_queries, int n_slots, size_t* bytes) {
  int st = iq_paged_check(c);
  if (st != IQ_OK) return st;
  if (!bytes) return fail(IQ_ERR_INVALID_ARG, "null bytes");
  if (q_heads <= 0 || n_queries < 0 || n_slots < 0) return fail(IQ_ERR_INVALID_ARG, "bad q_heads, n_queries or n_slots");
  if (n_slots > IQ_MAX_BATCH) return fail(IQ_ERR_INVALID_ARG, "bad number of slots");
  if (q_heads % c->kv_heads) return fail(IQ_ERR_UNSUPPORTED, "q_heads must be a multiple of kv_heads");
  if (q_heads / c->kv_heads > kMaxRep) return fail(IQ_ERR_UNSUPPORTED, "at most 64 query heads per kv head");
  if (static_cast<long long>(n_queries) * (q_heads / c->kv_heads) >= (1LL << 30)) return fail(IQ_ERR_UNSUPPORTED, "too many query rows");
  const int rows = n_queries * (q_heads / c->kv_heads);
  const size_t parts = rows > 0 && n_slots > 0 ? 2 * static_cast<size_t>(num_sms()) * unit_rows(rows) : 0;
  *bytes = parts ? parts * (kHeadDim * sizeof(float) + sizeof(float2)) + num_sms() * sizeof(Cut) : 0;
  if (rows > kMaxSplitRows) {  // the queries' two parts and factors
    const size_t all = static_cast<size_t>(n_slots) * q_heads * n_queries;
    if (all >= (1u << 30)) return fail(IQ_ERR_UNSUPPORTED, "too many query rows");
    *bytes += all * (2 * kHeadDim + sizeof(float));
  }
  return IQ_OK;
}

int iq_paged_attend(const iq_paged* c, const void* q, int q_heads, int n_queries, const int32_t* slots,
                    const int32_t* counts, int n_slots, float scale, int causal, int window, int sinks, void* out,
                    int out_f32, void* workspace, size_t workspace_bytes, iq_stream_t stream) {
  const int st = check_attend(c, q, q_heads, n_queries, slots, counts, n_slots, 0, scale, causal, window, sinks, out, out_f32,
                              workspace, workspace_bytes);
  if (st != IQ_OK || n_slots == 0 || n_queries == 0) return st;
  const int rep = q_heads / c->kv_heads, rows = rep * n_queries;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const Range written{out, static_cast<size_t>(n_slots) * q_heads * n_queries * kHeadDim * (out_f32 ? 4 : 2)};
  int longest = 0;
  for (int i = 0; i < n_slots; ++i) longest = std::max(longest, c->lens[slot_of(slots, i)]);
  if (window >= longest) window = sinks = 0;  // nothing is out of it, and positions less a window stay in 32 bits
  const int zeroed = store_zeros(c, q_heads, n_queries, slots, counts, n_slots, out, out_f32, stream);
  if (zeroed != IQ_OK) return zeroed;
  AttendParams p;
  std::memset(&p, 0, sizeof(p));
  p.unit_rows = unit_rows(rows);
  long long tiles = 0, per[IQ_MAX_BATCH];
  int units[IQ_MAX_BATCH];
  for (int i = 0; i < n_slots; ++i) {
    const int len = c->lens[slot_of(slots, i)], count = counts ? counts[i] : n_queries;
    per[i] = units[i] = 0;
    if (len > 0 && count > 0) tiles += (per[i] = tiles_of_entry(len, count, rep, p.unit_rows, causal, window, sinks, &units[i])) * c->kv_heads;
  }
  const int grid = static_cast<int>(std::min<long long>(num_sms(), tiles));
  if (grid == 0) return IQ_OK;
  p.cost = tiles >= 8ll * grid ? unit_cost(p.unit_rows) : 0;
  long long total = 0;
  for (int i = 0; i < n_slots; ++i) {
    const int s = slot_of(slots, i), len = c->lens[s], count = counts ? counts[i] : n_queries;
    if (count == 0 || len == 0) continue;
    const int e = p.entries++;
    p.entry[e] = static_cast<short>(i);
    p.slot[e] = static_cast<short>(s);
    p.len[e] = len;
    p.count[e] = count;
    p.cum[e] = static_cast<int>(total);
    per[i] += static_cast<long long>(units[i]) * p.cost;
    total += per[i] * c->kv_heads;
    p.per[e] = static_cast<int>(per[i]);
  }
  p.cum[p.entries] = p.total = static_cast<int>(total);
  const long long pool_rows = static_cast<long long>(c->pages) * c->kv_heads * kPage;
  if (!code_map(&p.k_map, c->k_codes, pool_rows) || !code_map(&p.v_map, c->v_codes, pool_rows))
    return fail(IQ_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  p.k_scales = c->k_scales;
  p.v_scales = c->v_scales;
  p.table = c->table;
  p.status = c->status;
  p.q = static_cast<const uint16_t*>(q);
  p.out = out;
  p.out_f32 = out_f32;
  p.heads = c->kv_heads;
  p.rep = rep;
  while ((2 << p.rep_shift) <= rep) ++p.rep_shift;
  if (rep & (rep - 1)) p.rep_mul = static_cast<unsigned>(((1ull << (32 + p.rep_shift)) + rep - 1) / rep);
  p.nq = n_queries;
  p.pages = c->pages;
  p.max_pages = c->max_pages;
  p.causal = causal;
  p.window = window;
  p.sinks = sinks;
  p.scale = scale;
  p.stall = stall_next ? 1 : 0;
  stall_next = false;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = reinterpret_cast<float2*>(p.part_o + 2ll * num_sms() * p.unit_rows * kHeadDim);
  p.cuts = reinterpret_cast<Cut*>(p.part_ml + 2ll * num_sms() * p.unit_rows);
  int all_counts[IQ_MAX_BATCH];
  if (p.unit_rows == 128) {
    const long long all = static_cast<long long>(n_slots) * q_heads * n_queries;
    p.cut = reinterpret_cast<uint8_t*>(p.cuts + num_sms());  // 16-byte aligned
    p.factors = reinterpret_cast<float*>(p.cut + all * 2 * kHeadDim);
    p.slots_n = n_slots;
    for (int i = 0; i < n_slots; ++i) all_counts[i] = counts ? counts[i] : n_queries;
    if (!code_map(&p.q_map, p.cut, 2 * all, 128)) return fail(IQ_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  }
  cudaError_t err = p.unit_rows == 8    ? launch_split<8>(p, grid, cs)
                    : p.unit_rows == 16 ? launch_split<16>(p, grid, cs)
                    : p.unit_rows == 32 ? launch_split<32>(p, grid, cs)
                                        : launch_prefill(p, all_counts, grid, cs);
  if (err == cudaSuccess && grid > 1) {
    const int each = p.unit_rows == 128 ? 8 : 1, most = std::min(p.unit_rows, rows);
    JoinParams j;
    j.part_o = p.part_o;
    j.part_ml = p.part_ml;
    j.cuts = p.cuts;
    j.out = p.out;
    j.out_f32 = p.out_f32;
    j.heads = p.heads;
    j.rep = p.rep;
    j.nq = p.nq;
    j.unit_rows = p.unit_rows;
    j.rows = each;
    std::memcpy(j.entry, p.entry, sizeof(j.entry));
    std::memcpy(j.count, p.count, sizeof(j.count));
    void* args[] = {&j};
    err = launch_after(reinterpret_cast<const void*>(&paged_join_kernel), dim3(grid - 1, (most + each - 1) / each), 256, 0, cs, args);
  }
  if (err != cudaSuccess) return cuda_fail(err, "paged attention");
  launched_outputs(stream, written);
  return IQ_OK;
}

}  // extern "C"
