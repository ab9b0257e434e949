// Element access of the layer operators: runs of 8 elements of fp32, bfloat16 or
// fp16 at any alignment of the element type (gfx950 loads and stores 16 bytes at
// any byte address; the compiler emits the wide access from a memcpy), widened to
// fp32, and rounded back to nearest, ties to even.
#pragma once

#pragma clang fp contract(off)

#include "echo_layer_internal.h"

namespace echo {
namespace {

// The launch arguments (the kernel's first parameter, at the start of the argument
// segment) where they lie in constant memory, so that a pointer picked by the rank,
// which is uniform, is one scalar load; indexing the parameter itself would make the
// compiler copy it to scratch memory.
#if defined(__HIP_DEVICE_COMPILE__)
template <typename Args>
__device__ __forceinline__ const __attribute__((address_space(4))) Args* kernel_args() {
  return (const __attribute__((address_space(4))) Args*)__builtin_amdgcn_kernarg_segment_ptr();
}
#else
template <typename Args>
__device__ const Args* kernel_args();  // never run: the host pass only parses the kernels
#endif

template <int E>
struct ElemOf;
template <>
struct ElemOf<kElemF32> {
  typedef float T;
};
template <>
struct ElemOf<kElemBf16> {
  typedef __bf16 T;
};
template <>
struct ElemOf<kElemF16> {
  typedef _Float16 T;
};

template <int E>
__device__ __forceinline__ void load8(const void* base, int64_t at, float v[8]) {
  typedef typename ElemOf<E>::T T;
  typedef T T8 __attribute__((ext_vector_type(8)));
  T8 x;
  __builtin_memcpy(&x, static_cast<const T*>(base) + at, sizeof(x));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = static_cast<float>(x[i]);
}

template <int E>
__device__ __forceinline__ float load1(const void* base, int64_t at) {
  return static_cast<float>(static_cast<const typename ElemOf<E>::T*>(base)[at]);
}

// An fp32 value to the element type.  For fp16 the value passes through an empty asm
// statement: the compiler would otherwise fold the fp32 operation before the
// conversion into one v_fma_mixlo_f16, which rounds once where the operations
// named round twice.
template <int E>
__device__ __forceinline__ typename ElemOf<E>::T narrow(float v) {
#if defined(__HIP_DEVICE_COMPILE__)
  if constexpr (E == kElemF16) asm("" : "+v"(v));
#endif
  return static_cast<typename ElemOf<E>::T>(v);
}

template <int E>
__device__ __forceinline__ void store8(void* base, int64_t at, const float v[8]) {
  typedef typename ElemOf<E>::T T;
  typedef T T8 __attribute__((ext_vector_type(8)));
  T8 x;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = narrow<E>(v[i]);
  __builtin_memcpy(static_cast<T*>(base) + at, &x, sizeof(x));
}

template <int E>
__device__ __forceinline__ void store1(void* base, int64_t at, float v) {
  typedef typename ElemOf<E>::T T;
  static_cast<T*>(base)[at] = narrow<E>(v);
}

}  // namespace
}  // namespace echo
