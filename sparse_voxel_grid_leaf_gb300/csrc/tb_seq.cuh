// Device helpers shared by the sequence operators (tb_rotary.cu, tb_norm.cu,
// tb_linattn.cu): 16-byte vectors of the three row types, read and written as
// 32-bit floats.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cstdint>

namespace tb {

template <class T> struct RowType;
template <> struct RowType<float> {
  static constexpr int kVec = 4;
  __device__ static float to(float x) { return x; }
  __device__ static float from(float x) { return x; }
};
template <> struct RowType<__half> {
  static constexpr int kVec = 8;
  __device__ static float to(__half x) { return __half2float(x); }
  __device__ static __half from(float x) { return __float2half_rn(x); }
};
template <> struct RowType<__nv_bfloat16> {
  static constexpr int kVec = 8;
  __device__ static float to(__nv_bfloat16 x) { return __bfloat162float(x); }
  __device__ static __nv_bfloat16 from(float x) { return __float2bfloat16_rn(x); }
};

// V elements of T as one register vector: 16 bytes for V = RowType<T>::kVec,
// one element for V = 1.
template <class T, int V> struct alignas(V * sizeof(T)) Pack {
  T e[V];
};

template <class T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  if constexpr (V == 1) {
    Pack<T, 1> r;
    r.e[0] = *p;
    return r;
  } else {
    static_assert(sizeof(Pack<T, V>) == 16, "16-byte vectors");
    union {
      uint4 u;
      Pack<T, V> v;
    } r;
    r.u = *reinterpret_cast<const uint4*>(p);
    return r.v;
  }
}

template <class T, int V>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, V>& v) {
  if constexpr (V == 1) {
    *p = v.e[0];
  } else {
    union {
      uint4 u;
      Pack<T, V> v;
    } r;
    r.v = v;
    *reinterpret_cast<uint4*>(p) = r.u;
  }
}

template <class T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& v, float (&f)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = RowType<T>::to(v.e[i]);
}

template <class T, int V>
__device__ __forceinline__ Pack<T, V> pack(const float (&f)[V]) {
  Pack<T, V> r;
#pragma unroll
  for (int i = 0; i < V; ++i) r.e[i] = RowType<T>::from(f[i]);
  return r;
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
  return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int d = 16; d; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
  return x;
}

}  // namespace tb
