// libiqkv: attention over the paged 8-bit cache.
//
// First form: a warp per query row, online softmax over the keys that the row
// sees (at most two runs of them: the sinks and the window), every key's codes
// decoded in registers.  float32 throughout.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>

#include "iq_paged.cuh"

namespace iq {
namespace paged {

struct AttendParams {
  const uint8_t* k_codes;
  const uint8_t* v_codes;
  const float* k_scales;
  const float* v_scales;
  const int* table;
  unsigned* status;
  const uint16_t* q;
  void* out;
  int out_f32, heads, rep, nq, pages, max_pages, causal, window, sinks;
  float scale;
  int slot[IQ_MAX_BATCH], len[IQ_MAX_BATCH], count[IQ_MAX_BATCH];
};

__device__ __forceinline__ void load8(const uint8_t* codes, float s, float (&x)[8]) {
  const uint2 c = *reinterpret_cast<const uint2*>(codes);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = f16x2_to_f32(e4m3x2_to_f16x2((j < 2 ? c.x : c.y) >> (16 * (j & 1)) & 0xFFFFu));
    x[2 * j] = f.x * s;
    x[2 * j + 1] = f.y * s;
  }
}

__global__ void __launch_bounds__(256) paged_attend_simple(const __grid_constant__ AttendParams p) {
  const int lane = threadIdx.x & 31, i = blockIdx.z, hq = blockIdx.y, h = hq / p.rep;
  const int j = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (j >= p.count[i]) return;
  const int len = p.len[i], pos = len - p.count[i] + j;
  const long long row = ((static_cast<long long>(i) * p.heads * p.rep + hq) * p.nq + j) * kHeadDim + lane * 8;
  float q[8], o[8] = {};
  const uint4 raw = *reinterpret_cast<const uint4*>(p.q + row);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int d = 0; d < 8; ++d) q[d] = bf16_to_f32(w[d / 2] >> (16 * (d & 1)) & 0xFFFFu) * p.scale;
  const int stop = p.causal ? pos + 1 : len;
  const int low = p.window && pos >= p.window ? pos - p.window + 1 : 0;  // first key of the window
  float m = -__builtin_huge_valf(), l = 0.0f;
  for (int t = min(p.sinks, low) > 0 ? 0 : low; t < stop; ++t) {
    if (t == p.sinks && t < low) t = low;
    const int page = page_in_pool(p.table[static_cast<long long>(p.slot[i]) * p.max_pages + t / kPage], p.pages, p.status);
    const long long at = static_cast<long long>(page) * p.heads + h, byte = at * kPageBytes + (t % kPage) * kHeadDim + lane * 8;
    float x[8], s = 0.0f;
    load8(p.k_codes + byte, p.k_scales[at], x);
#pragma unroll
    for (int d = 0; d < 8; ++d) s = fmaf(q[d], x[d], s);
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
    const float m2 = fmaxf(m, s), f = __expf(m - m2), e = __expf(s - m2);
    load8(p.v_codes + byte, p.v_scales[at], x);
#pragma unroll
    for (int d = 0; d < 8; ++d) o[d] = fmaf(o[d], f, e * x[d]);
    l = fmaf(l, f, e);
    m = m2;
  }
  const float inv = stop > 0 ? 1.0f / l : 0.0f;
  if (p.out_f32) {
    float* out = static_cast<float*>(p.out) + row;
#pragma unroll
    for (int d = 0; d < 8; ++d) out[d] = o[d] * inv;
  } else {
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + row);
#pragma unroll
    for (int d = 0; d < 4; ++d) out[d] = f32_to_bf16_bits(o[2 * d] * inv) | f32_to_bf16_bits(o[2 * d + 1] * inv) << 16;
  }
}

int check_attend(const iq_paged* c, const void* q, int q_heads, int n_queries, const int32_t* slots,
                 const int32_t* counts, int n_slots, float scale, int causal, int window, int sinks,
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
  return IQ_OK;
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
  *bytes = 0;
  return IQ_OK;
}

int iq_paged_attend(const iq_paged* c, const void* q, int q_heads, int n_queries, const int32_t* slots,
                    const int32_t* counts, int n_slots, float scale, int causal, int window, int sinks, void* out,
                    int out_f32, void* workspace, size_t workspace_bytes, iq_stream_t stream) {
  const int st = check_attend(c, q, q_heads, n_queries, slots, counts, n_slots, scale, causal, window, sinks, out, out_f32,
                              workspace, workspace_bytes);
  if (st != IQ_OK || n_slots == 0 || n_queries == 0) return st;
  AttendParams p;
  std::memset(&p, 0, sizeof(p));
  p.k_codes = c->k_codes;
  p.v_codes = c->v_codes;
  p.k_scales = c->k_scales;
  p.v_scales = c->v_scales;
  p.table = c->table;
  p.status = c->status;
  p.q = static_cast<const uint16_t*>(q);
  p.out = out;
  p.out_f32 = out_f32;
  p.heads = c->kv_heads;
  p.rep = q_heads / c->kv_heads;
  p.nq = n_queries;
  p.pages = c->pages;
  p.max_pages = c->max_pages;
  p.causal = causal;
  p.window = window;
  p.sinks = sinks;
  p.scale = scale;
  for (int i = 0; i < n_slots; ++i) {
    p.slot[i] = slot_of(slots, i);
    p.len[i] = c->lens[p.slot[i]];
    p.count[i] = counts ? counts[i] : n_queries;
  }
  paged_attend_simple<<<dim3((n_queries + 7) / 8, q_heads, n_slots), 256, 0, static_cast<cudaStream_t>(stream)>>>(p);
  IQ_CUDA(cudaGetLastError());
  return IQ_OK;
}

}  // extern "C"
