// The paged 8-bit cache, shared between its translation units: descriptor
// checks, e4m3 conversions and the page exponent.
#pragma once

#include <atomic>

#include "iq_common.cuh"

namespace iq {
namespace paged {

constexpr int kPage = IQ_PAGE;
constexpr int kPageBytes = kPage * kHeadDim;  // one page of one kv head, keys or values
constexpr int kEMin = -40, kEMax = 60;        // exponents of the page scales
constexpr int kMaxRep = 64;

// The slot list of a call: distinct, in range; NULL stands for 0 .. n-1.
int check_slots(const iq_paged* c, const int32_t* slots, int n, bool distinct);
inline int slot_of(const int32_t* slots, int i) { return slots ? slots[i] : i; }
inline int pages_for(long long tokens) { return static_cast<int>((tokens + kPage - 1) / kPage); }
inline bool misaligned(const void* p, uintptr_t to = 16) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// The arguments of an attention call, checked.  added: the rows that the call
// appends to every entry first (counts[i] of them, where counts are given).
int check_attend(const iq_paged* c, const void* q, int q_heads, int n_queries, const int32_t* slots,
                 const int32_t* counts, int n_slots, int added, float scale, int causal, int window, int sinks,
                 const void* out, int out_f32, const void* workspace, size_t workspace_bytes);

// A launch that may begin while the kernel before it ends; every kernel of the
// paged cache waits for that one itself, before it touches memory.  args: one
// pointer per parameter.
cudaError_t launch_after(const void* kernel, dim3 grid, int threads, int smem, cudaStream_t stream, void** args);
// Shared memory above 48 KB, allowed once per kernel and device (`seen`: the kernel's own).
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& seen);
extern thread_local int launch_to_fail;  // test hook (iq_paged_debug_fail): how many launches from now, < 0: none
extern thread_local bool stall_next;     // test hook (iq_paged_debug_stall)
__device__ __forceinline__ void wait_for_last_kernel() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
// For a kernel that takes tensor memory: it takes it between these two.  A kernel
// that holds some while it waits for another, which may still have to take its own
// on the same multiprocessor, could wait forever.
__device__ __forceinline__ void wait_only() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void release_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// Two floats to e4m3, to nearest even, saturating at +-448: `lo` in bits 0..7.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  unsigned short d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
// Two e4m3 codes (bits 0..15) to f16x2, exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t d;
  const unsigned short h = static_cast<unsigned short>(two);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(h));
  return d;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h2) {
  float2 r;
  asm("{\n.reg .b16 l, h;\nmov.b32 {l, h}, %2;\ncvt.f32.f16 %0, l;\ncvt.f32.f16 %1, h;\n}" : "=f"(r.x), "=f"(r.y) : "r"(h2));
  return r;
}
// 2^e for e in [-126, 127]
__device__ __forceinline__ float power2(int e) { return __int_as_float((e + 127) << 23); }
__device__ __forceinline__ int exponent_of(float p2) { return (__float_as_int(p2) >> 23) - 127; }

// A page id of the device table, kept inside the pool whatever it says.
__device__ __forceinline__ int page_in_pool(int id, int pages, unsigned* status) {
  if (static_cast<unsigned>(id) < static_cast<unsigned>(pages)) return id;
  atomicOr(status, IQ_STATUS_BAD_PAGE);
  return 0;
}

}  // namespace paged
}  // namespace iq
