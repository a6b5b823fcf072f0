// Device helpers shared by the sequence operators (tb_rotary.cu, tb_norm.cu,
// tb_linattn.cu): 16-byte vectors of the three row types, read and written as
// 32-bit floats.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>
#include <cstring>

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

// V elements of T as they lie in memory, in whole registers (an array of
// 16-bit elements would take a register each): 16 bytes for V =
// RowType<T>::kVec, one element for V = 1.
template <class T, int V> struct Pack {
  static_assert(V * sizeof(T) == 16 || V * sizeof(T) == 8, "vectors of 16 or 8 bytes");
  uint32_t w[V * sizeof(T) / 4];
};
template <class T> struct Pack<T, 1> {
  T e;
};

template <class T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  Pack<T, V> r;
  if constexpr (V == 1) {
    r.e = *p;
  } else if constexpr (V * sizeof(T) == 8) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    r.w[0] = u.x, r.w[1] = u.y;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    r.w[0] = u.x, r.w[1] = u.y, r.w[2] = u.z, r.w[3] = u.w;
  }
  return r;
}

template <class T, int V>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, V>& v) {
  if constexpr (V == 1) *p = v.e;
  else if constexpr (V * sizeof(T) == 8) *reinterpret_cast<uint2*>(p) = make_uint2(v.w[0], v.w[1]);
  else *reinterpret_cast<uint4*>(p) = make_uint4(v.w[0], v.w[1], v.w[2], v.w[3]);
}

__device__ __forceinline__ float2 halves_of(uint32_t w, __half) {
  __half2 h;
  memcpy(&h, &w, 4);
  return __half22float2(h);
}
__device__ __forceinline__ float2 halves_of(uint32_t w, __nv_bfloat16) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ uint32_t word_of(float lo, float hi, __half) {
  const __half2 h = __floats2half2_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}
__device__ __forceinline__ uint32_t word_of(float lo, float hi, __nv_bfloat16) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &h, 4);
  return w;
}

template <class T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& v, float (&f)[V]) {
  if constexpr (V == 1) {
    f[0] = RowType<T>::to(v.e);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = __uint_as_float(v.w[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 x = halves_of(v.w[i], T());
      f[2 * i] = x.x;
      f[2 * i + 1] = x.y;
    }
  }
}

template <class T, int V>
__device__ __forceinline__ Pack<T, V> pack(const float (&f)[V]) {
  Pack<T, V> r;
  if constexpr (V == 1) {
    r.e = RowType<T>::from(f[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < V; ++i) r.w[i] = __float_as_uint(f[i]);
  } else {
#pragma unroll
    for (int i = 0; i < V / 2; ++i) r.w[i] = word_of(f[2 * i], f[2 * i + 1], T());
  }
  return r;
}

// A kernel that reads what the one before it in a call writes is launched while
// that one still runs (launch_early) and waits here for its end; the one before
// lets it start.  Both are no-ops in ordinary launches.
__device__ __forceinline__ void wait_for_last_kernel() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_kernel_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

template <class... P, class... A>
cudaError_t launch_early(void (*kernel)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, bool early, A&&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = grid;
  c.blockDim = block;
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = early ? 1 : 0;
  return cudaLaunchKernelEx(&c, kernel, P(args)...);
}

// Lets a kernel take up to `bytes` of dynamic shared memory.  The limit belongs
// to the kernel, not to the launch: it is set to the most that any call takes,
// once for each device, so that calls from several host threads never lower it
// under one another.  ready: the kernel's own.
constexpr int kMaxDevices = 64;
template <class K>
cudaError_t allow_shared(K* kernel, int bytes, std::atomic<bool> (&ready)[kMaxDevices]) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool known = dev >= 0 && dev < kMaxDevices;
  if (known && ready[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && known) ready[dev].store(true, std::memory_order_release);
  return e;
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
