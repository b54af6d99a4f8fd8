// libiqkv: attention of many query rows per kv head (prompts and their chunks)
// over the paged 8-bit cache.  What its CTAs do: iq_paged_rows.cuh.
#include <cuda_runtime.h>

#include "iq_paged_rows.cuh"

namespace iq {
namespace paged {
namespace {

// The queries' two parts and factors, a warp per four rows, before the kernel
// below: cut inside it, by warps of its own, they slowed the row threads by a
// third around every unit's begin (the conversions share a pipe), 260 against
// 214 us for 8191 queries under a window of 1023.
struct CutParams {
  const uint16_t* q;
  uint8_t* cut;
  float* factors;
  int heads, rep, nq, total;
  float scale;
  int count[IQ_MAX_BATCH];
};
__global__ void __launch_bounds__(256) paged_cut_kernel(const __grid_constant__ CutParams p) {
  wait_for_last_kernel();
  const int lane = threadIdx.x & 31, w0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * 4, rows = p.nq * p.rep;
  uint4 raw[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int w = min(w0 + k, p.total - 1), eh = w / rows, r = w - eh * rows, j = r / p.rep, e = eh / p.heads;
    raw[k] = make_uint4(0, 0, 0, 0);
    if (j < p.count[e])  // row r of (entry, kv head): query j of query head eh * rep + r % rep
      raw[k] = __ldcs(reinterpret_cast<const uint4*>(p.q + ((static_cast<long long>(eh) * p.rep + r - j * p.rep) * p.nq + j) * kHeadDim) + lane);
  }
  if (p.scale < 0.0f) {  // the factors are positive, so that the largest product is the largest score
#pragma unroll
    for (int k = 0; k < 4; ++k)
      raw[k] = make_uint4(raw[k].x ^ 0x80008000u, raw[k].y ^ 0x80008000u, raw[k].z ^ 0x80008000u, raw[k].w ^ 0x80008000u);
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint2 hi, lo;
    const float f = split_query<1>(raw[k], hi, lo);
    const long long w = w0 + k;
    if (w >= p.total) break;
    reinterpret_cast<uint2*>(p.cut + w * kHeadDim)[lane] = hi;
    reinterpret_cast<uint2*>(p.cut + (p.total + w) * kHeadDim)[lane] = lo;
    if (lane == 0) p.factors[w] = fminf(f * (fabsf(p.scale) * kLog2e), 3e38f);
  }
}

__global__ void __launch_bounds__(rows::kThreads, 1) paged_prefill_kernel(const __grid_constant__ AttendParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];  // the swizzled operands need it; no room to align by hand
  rows::run(p, {0, p.entries, p.cost, p.total, static_cast<int>(blockIdx.x), static_cast<int>(gridDim.x)}, smem);
}

}  // namespace

cudaError_t launch_prefill(const AttendParams& p, const int* counts, int grid, cudaStream_t stream) {
  static std::atomic<uint64_t> seen{0};
  const void* kernel = reinterpret_cast<const void*>(&paged_prefill_kernel);
  cudaError_t e = allow_smem(kernel, rows::kSmem, seen);
  CutParams c;
  c.q = p.q;
  c.cut = p.cut;
  c.factors = p.factors;
  c.heads = p.heads;
  c.rep = p.rep;
  c.nq = p.nq;
  c.total = p.slots_n * p.heads * p.rep * p.nq;
  c.scale = p.scale;
  for (int i = 0; i < p.slots_n; ++i) c.count[i] = counts[i];
  void* cut_args[] = {&c};
  void* args[] = {const_cast<AttendParams*>(&p)};
  if (e == cudaSuccess) e = launch_after(reinterpret_cast<const void*>(&paged_cut_kernel), dim3((c.total + 31) / 32), 256, 0, stream, cut_args);
  if (e == cudaSuccess) e = launch_after(kernel, dim3(grid), rows::kThreads, rows::kSmem, stream, args);
  return e;
}

}  // namespace paged
}  // namespace iq
