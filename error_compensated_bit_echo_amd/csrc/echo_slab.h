// Slab pipeline of the product kernels: loads from global memory straight into LDS
// through buffer resources, the waits on them, and the workgroup barrier between
// K steps.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace echo {
namespace {

// Fourth word of a raw buffer resource: 32-bit data format (any nonzero format
// does for these loads; a zero format would make every load return zero).
constexpr int kBufferWord3 = 0x00020000;

// The non-temporal (nt) bit of the cache-policy operand: the lines are kept in
// the caches as streaming data, evicted first.
constexpr int kNonTemporal = 2;

// A raw buffer resource over `bytes` bytes from `base`, and one 16-byte-per-lane
// load through it straight into LDS (lane l's 16 bytes land at lds + 16 l bytes;
// an offset at or past `bytes` reads zeros).  The slab loads use these rather
// than global_load_lds: the compiler counts a global (FLAT-encoded) load into
// LDS as pending LDS traffic too, so every wait for fragment reads in the K loop
// also waited for the next slab's loads (measured 4-5 % slower).  The builtins
// exist only for the device; the host pass, which also compiles the kernel
// bodies, gets stand-ins it never runs.
struct BufRsrc {
  __amdgpu_buffer_rsrc_t r;
};
__device__ __forceinline__ BufRsrc buffer_rsrc(const void* base, int32_t bytes) {
#if defined(__HIP_DEVICE_COMPILE__)
  return BufRsrc{__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, bytes, kBufferWord3)};
#else
  (void)base;
  (void)bytes;
  return BufRsrc{};
#endif
}
// POLICY: the cache-policy operand of the load (0, or kNonTemporal).
template <int POLICY>
__device__ __forceinline__ void buffer_load_lds16(BufRsrc r, void* lds, uint32_t voffset, uint32_t soffset) {
#if defined(__HIP_DEVICE_COMPILE__)
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r.r, (__attribute__((address_space(3))) void*)lds, 16, voffset,
                                           soffset, 0, POLICY);
#else
  (void)r;
  (void)lds;
  (void)voffset;
  (void)soffset;
#endif
}

// s_waitcnt immediate that waits for every outstanding LDS access of this
// wavefront (lgkmcnt 0) and not for vector-memory operations or exports.
constexpr int kLdsDrained = 0xC07F;

// s_waitcnt immediate that waits until at most n vector-memory operations of
// this wavefront are outstanding (lgkm and export counts not waited on):
// vmcnt[3:0] in bits 3:0, vmcnt[5:4] in bits 15:14, expcnt 7, lgkmcnt 15.
constexpr int vmcnt_at_most(int n) { return (n & 15) | ((n >> 4) << 14) | (7 << 4) | (15 << 8); }
// The same, and every outstanding LDS access too (lgkmcnt 0).
constexpr int vmcnt_at_most_lds_drained(int n) { return vmcnt_at_most(n) & ~(15 << 8); }

// Workgroup barrier for the slab pipeline.  __syncthreads() would also make
// every wavefront wait for all its outstanding global loads (its release fence
// covers the loads that write LDS), which would drain the loads of the later
// slabs at every step; here each wavefront first waits, with vmcnt_at_most,
// for the loads of the slab about to be read only.  The empty asm statements
// keep the compiler from moving LDS accesses across the barrier.
__device__ __forceinline__ void slab_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

}  // namespace
}  // namespace echo
