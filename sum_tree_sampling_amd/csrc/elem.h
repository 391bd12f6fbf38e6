// elem.h -- element types of the sequence operators: loads and stores of a
// few neighbouring values at the type's own alignment (gfx950 takes unaligned
// wide accesses), converted from and to f32.  The conversion to 16 bits is the
// hardware's, to nearest even.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace per {

typedef __bf16 bf16_t;
typedef _Float16 f16_t;

// N values of T as they lie in memory.
template <typename T, int N>
struct Pack {
  typedef T vec __attribute__((ext_vector_type(N)));
  vec v;
};
template <typename T>
struct Pack<T, 1> {
  T v;
};

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T* p) {
  Pack<T, N> r;
  __builtin_memcpy(&r, p, sizeof r);
  return r;
}

template <typename T, int N>
__device__ __forceinline__ void unpack(const Pack<T, N>& r, float (&out)[N]) {
  if constexpr (N == 1) {
    out[0] = (float)r.v;
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) out[i] = (float)r.v[i];
  }
}

template <typename T, int N>
__device__ __forceinline__ void store_vals(T* p, const float (&in)[N]) {
  Pack<T, N> r;
  if constexpr (N == 1) {
    r.v = (T)in[0];
  } else {
    typedef float fvec __attribute__((ext_vector_type(N)));
    fvec f;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = in[i];
    r.v = __builtin_convertvector(f, decltype(r.v));
  }
  __builtin_memcpy(p, &r, sizeof r);
}

// The same, past the caches: for output that this kernel does not read again.
template <typename T, int N>
__device__ __forceinline__ void store_once(T* p, const float (&in)[N]) {
  if constexpr (N == 1) {
    __builtin_nontemporal_store((T)in[0], p);
  } else {
    typedef float fvec __attribute__((ext_vector_type(N)));
    typedef T tvec __attribute__((ext_vector_type(N)));
    typedef tvec tvec_u __attribute__((aligned(sizeof(T))));
    fvec f;
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = in[i];
    __builtin_nontemporal_store(__builtin_convertvector(f, tvec), reinterpret_cast<tvec_u*>(p));
  }
}

// 16 bytes at a 16-byte aligned address that no later access is expected to
// find in a cache.
template <typename P>
__device__ __forceinline__ P load_once(const void* p) {
  typedef uint32_t u4 __attribute__((ext_vector_type(4)));
  const u4 u = __builtin_nontemporal_load(static_cast<const u4*>(p));
  P r;
  static_assert(sizeof(P) == 16, "16 bytes");
  __builtin_memcpy(&r, &u, 16);
  return r;
}

}  // namespace per
