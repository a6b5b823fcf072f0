// Linear attention with a decay for each head: the single-token step, and the
// recurrence over rows in 32-bit arithmetic (any row type and head size).
//
// Step: 8 bytes per state element and nothing else of size, so the bound is
// memory.  A block takes one state [key, value]; every thread keeps its loads
// of a column group in flight together, updates them, writes them back and
// adds its share of q S, which the block joins in shared memory.
//
// Recurrence: a warp holds the state columns of 16 values, each thread 2
// columns x a quarter of the keys in registers, and walks the rows, which the
// block stages in shared memory as floats.  Two multiply-adds and a multiply
// per state element and row in packed pairs (fma.rn.f32x2) bound it.
#include "tb_linattn.cuh"
#include "tb_seq.cuh"

namespace tb {
namespace {

// ---------------------------------------------------------------- one token

constexpr int kStepThreads = 256;
constexpr int kStepBatch = 16;  // state vectors in flight per thread

template <class T, int V>
__global__ void __launch_bounds__(kStepThreads) k_step(StepLaunch l) {
  const tb_linear_step_args& a = l.a;
  __shared__ float s_q[256], s_k[256];
  __shared__ float s_o[kStepThreads * V];
  const int64_t n = blockIdx.x / a.heads;
  const int h = (int)(blockIdx.x - n * a.heads);
  const int64_t slot = a.slots ? (int64_t)a.slots[n] : n;
  T* out = (T*)a.out + n * a.out_row + h * a.out_head;
  if (slot < 0 || slot >= a.num_slots) {
    for (int i = threadIdx.x; i < a.value; i += kStepThreads) out[i] = RowType<T>::from(0.f);
    return;
  }
  const int cols = a.value / V;               // column groups
  const int rows = kStepThreads / cols;       // state rows of one sweep
  const int col = threadIdx.x % cols, row = threadIdx.x / cols;
  const bool live = row < rows;
  float* state = a.state + ((slot * a.heads + h) * a.key) * (int64_t)a.value + col * V;
  const T* q = (const T*)a.q + n * a.q_row + h * a.q_head;
  const T* k = (const T*)a.k + n * a.k_row + h * a.k_head;
  const T* v = (const T*)a.v + n * a.v_row + h * a.v_head;
  for (int i = threadIdx.x; i < a.key; i += kStepThreads) {
    s_q[i] = RowType<T>::to(q[i]);
    s_k[i] = RowType<T>::to(k[i]);
  }
  const float decay = a.decay[h];
  float vv[V], o[V] = {};
#pragma unroll
  for (int j = 0; j < V; ++j) vv[j] = live ? RowType<T>::to(v[col * V + j]) : 0.f;
  bool first = true;
  for (int base = row; first || base < a.key; base += rows * kStepBatch) {
    Pack<float, V> x[kStepBatch];
#pragma unroll
    for (int i = 0; i < kStepBatch; ++i) {
      const int r = base + i * rows;
      if (live && r < a.key) x[i] = load_pack<float, V>(state + (int64_t)r * a.value);
    }
    if (first) __syncthreads();  // q and k are staged; the state's loads are on their way
    first = false;
#pragma unroll
    for (int i = 0; i < kStepBatch; ++i) {
      const int r = base + i * rows;
      if (live && r < a.key) {
        const float kk = s_k[r], qq = s_q[r];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          x[i].e[j] = fmaf(x[i].e[j], decay, kk * vv[j]);
          o[j] = fmaf(qq, x[i].e[j], o[j]);
        }
        store_pack<float, V>(state + (int64_t)r * a.value, x[i]);
      }
    }
  }
  if (live)
#pragma unroll
    for (int j = 0; j < V; ++j) s_o[row * a.value + col * V + j] = o[j];
  __syncthreads();
  for (int i = threadIdx.x; i < a.value; i += kStepThreads) {
    float sum = 0.f;
    for (int r = 0; r < rows; ++r) sum += s_o[r * a.value + i];
    out[i] = RowType<T>::from(sum * a.scale);
  }
}

template <class T>
cudaError_t go_step(const StepLaunch& l, cudaStream_t s) {
  const unsigned blocks = (unsigned)(l.a.streams * l.a.heads);
  if (l.a.value % 4 == 0) k_step<T, 4><<<blocks, kStepThreads, 0, s>>>(l);
  else k_step<T, 1><<<blocks, kStepThreads, 0, s>>>(l);
  return cudaGetLastError();
}

// ------------------------------------------------------------- the recurrence

typedef unsigned long long f32x2;
__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 halves(f32x2 x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

constexpr int kScanRows = 16;  // rows staged at a time

// KS: keys of one thread; 4 KS >= K.  A warp's four key slices interleave by
// four keys, so that their 16-byte reads of a staged row are consecutive.
template <class T, int KS>
__global__ void __launch_bounds__(256) k_scan(LinLaunch l) {
  constexpr int KP = 4 * KS;
  const LinProblem& p = l.p[blockIdx.z];
  __shared__ __align__(16) float s_a[kScanRows][KP], s_b[kScanRows][KP];
  __shared__ float s_c[kScanRows][128];
  const LinSegment seg = lin_segment(l, blockIdx.x);
  if (seg.grid < 0) return;
  const int h = blockIdx.y;
  const bool want_out = p.out && l.phase != 1;
  if (l.phase == 1 && seg.index + 1 == seg.count && !p.last) return;  // nobody reads this segment's state
  const float decay = l.decay[h];
  const int lane = threadIdx.x & 31, slice = lane & 3;
  const int v0 = (threadIdx.x >> 5) * 16 + (lane >> 2) * 2;
  const int64_t state_at = ((int64_t)seg.grid * l.heads + h) * p.K * p.V;
  float* seg_state = p.seg ? p.seg + ((int64_t)blockIdx.x * l.heads + h) * p.K * p.V : nullptr;

  f32x2 u[2][KS / 2];
  auto key = [&](int i) { return (i / 4 * 4 + slice) * 4 + i % 4; };
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < KS; i += 2) {
      float x[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = key(i + j), v = v0 + c;
        x[j] = 0.f;
        if (k < p.K && v < p.V) {
          if (l.phase == 2) x[j] = seg_state[(int64_t)k * p.V + v];
          else if (l.phase == 0 && p.first) x[j] = p.first[state_at + k * p.first_k + v * p.first_v];
        }
      }
      u[c][i / 2] = pair(x[0], x[1]);
    }

  const int64_t origin = p.reverse ? seg.end - 1 - seg.first : seg.begin + seg.first;
  const int64_t dir = p.reverse ? -1 : 1;
  const f32x2 fold = pair(p.fold, p.fold);
  for (int t0 = 0; t0 < seg.len; t0 += kScanRows) {
    const int nt = min(kScanRows, seg.len - t0);
    __syncthreads();
    for (int i = threadIdx.x; i < nt * KP; i += blockDim.x) {
      const int t = i / KP, k = i % KP;
      const int64_t row = origin + dir * (t0 + t);
      s_a[t][k] = want_out && k < p.K ? RowType<T>::to(((const T*)p.a)[row * p.a_row + h * p.a_head + k]) : 0.f;
      s_b[t][k] = k < p.K ? RowType<T>::to(((const T*)p.b)[row * p.b_row + h * p.b_head + k]) : 0.f;
    }
    for (int i = threadIdx.x; i < nt * 128; i += blockDim.x) {
      const int t = i / 128, v = i % 128;
      const int64_t row = origin + dir * (t0 + t);
      s_c[t][v] = v < p.V ? RowType<T>::to(((const T*)p.c)[row * p.c_row + h * p.c_head + v]) : 0.f;
    }
    __syncthreads();
    for (int t = 0; t < nt; ++t) {
      const float d = p.late && t0 + t == 0 ? 1.f : decay;
      const f32x2 d2 = pair(d, d);
      const f32x2 c0 = mul2(pair(s_c[t][v0], s_c[t][v0]), fold);
      const f32x2 c1 = mul2(pair(s_c[t][v0 + 1], s_c[t][v0 + 1]), fold);
      f32x2 o0 = 0ull, o1 = 0ull;
#pragma unroll
      for (int i = 0; i < KS; i += 4) {
        const float4 b = *reinterpret_cast<const float4*>(&s_b[t][(i + slice) * 4]);
        const f32x2 b0 = pair(b.x, b.y), b1 = pair(b.z, b.w);
        u[0][i / 2] = fma2(u[0][i / 2], d2, mul2(b0, c0));
        u[1][i / 2] = fma2(u[1][i / 2], d2, mul2(b0, c1));
        u[0][i / 2 + 1] = fma2(u[0][i / 2 + 1], d2, mul2(b1, c0));
        u[1][i / 2 + 1] = fma2(u[1][i / 2 + 1], d2, mul2(b1, c1));
        if (want_out) {
          const float4 a = *reinterpret_cast<const float4*>(&s_a[t][(i + slice) * 4]);
          const f32x2 a0 = pair(a.x, a.y), a1 = pair(a.z, a.w);
          o0 = fma2(a0, u[0][i / 2], o0);
          o1 = fma2(a0, u[1][i / 2], o1);
          o0 = fma2(a1, u[0][i / 2 + 1], o0);
          o1 = fma2(a1, u[1][i / 2 + 1], o1);
        }
      }
      if (want_out) {
        float x = halves(o0).x + halves(o0).y, y = halves(o1).x + halves(o1).y;
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        y += __shfl_xor_sync(0xffffffffu, y, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        y += __shfl_xor_sync(0xffffffffu, y, 2);
        const int v = v0 + slice;
        if (slice < 2 && v < p.V) {
          const int64_t row = origin + dir * (t0 + t);
          ((T*)p.out)[row * p.o_row + h * p.o_head + v] = RowType<T>::from((slice ? y : x) * p.mul);
        }
      }
    }
  }

  float* dst = l.phase == 1 ? seg_state : l.phase == 0 && p.last ? p.last + state_at : nullptr;
  if (!dst) return;
  const float leave = p.late && seg.len > 0 ? decay : 1.f;
#pragma unroll
  for (int c = 0; c < 2; ++c)
#pragma unroll
    for (int i = 0; i < KS; i += 2) {
      const float2 x = halves(u[c][i / 2]);
      const int v = v0 + c;
      if (v < p.V && key(i) < p.K) dst[(int64_t)key(i) * p.V + v] = x.x * leave;
      if (v < p.V && key(i + 1) < p.K) dst[(int64_t)key(i + 1) * p.V + v] = x.y * leave;
    }
}

constexpr int kCombineBatch = 16;

// Joins the segments of a split call: the state that enters each segment, in
// place of the segment's own, and the state that leaves the grid.
__global__ void __launch_bounds__(256) k_combine(LinLaunch l) {
  const LinProblem& p = l.p[blockIdx.z];
  const int b = blockIdx.x / l.heads, h = blockIdx.x % l.heads;
  const int slot0 = lin_first_slot(l, b);
  int64_t begin, end;
  lin_grid_rows(l, b, begin, end);
  const int n = lin_segments_of(l, end - begin);
  const float decay = l.decay[h];
  const float whole = lin_power(decay, (float)l.segment);
  const float rest = lin_power(decay, (float)(end - begin - (int64_t)(n - 1) * l.segment));
  const int size = p.K * p.V;
  const int64_t state_at = ((int64_t)b * l.heads + h) * size;
  const int i = blockIdx.y * blockDim.x + threadIdx.x;
  if (i >= size) return;
  float x = p.first ? p.first[state_at + i / p.V * p.first_k + i % p.V * p.first_v] : 0.f;
  float* at = p.seg + ((int64_t)slot0 * l.heads + h) * size + i;
  const int64_t next = (int64_t)l.heads * size;
  // the segments' own states are loaded ahead of the chain that joins them
  for (int s0 = 0; s0 < n; s0 += kCombineBatch) {
    float own[kCombineBatch];
#pragma unroll
    for (int j = 0; j < kCombineBatch; ++j)
      own[j] = s0 + j < n - (p.last ? 0 : 1) ? at[(s0 + j) * next] : 0.f;
#pragma unroll
    for (int j = 0; j < kCombineBatch; ++j)
      if (s0 + j < n) {
        at[(s0 + j) * next] = x;
        x = fmaf(x, s0 + j + 1 == n ? rest : whole, own[j]);
      }
  }
  if (p.last) p.last[state_at + i] = x;
}

template <class T>
cudaError_t go_scan(const LinLaunch& l, cudaStream_t s) {
  int K = 0, V = 0;
  for (int i = 0; i < l.n; ++i) {
    K = K > l.p[i].K ? K : l.p[i].K;
    V = V > l.p[i].V ? V : l.p[i].V;
  }
  const dim3 grid(l.segments, l.heads, l.n);
  const int threads = (V + 15) / 16 * 32;
  if (K <= 64) k_scan<T, 16><<<grid, threads, 0, s>>>(l);
  else k_scan<T, 32><<<grid, threads, 0, s>>>(l);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_step(const void* args, cudaStream_t s) {
  const StepLaunch& l = *(const StepLaunch*)args;
  switch (l.a.type) {
    case TB_TYPE_F32: return go_step<float>(l, s);
    case TB_TYPE_F16: return go_step<__half>(l, s);
    default: return go_step<__nv_bfloat16>(l, s);
  }
}

cudaError_t launch_linear_scan(const void* args, cudaStream_t s) {
  const LinLaunch& l = *(const LinLaunch*)args;
  switch (l.type) {
    case TB_TYPE_F32: return go_scan<float>(l, s);
    case TB_TYPE_F16: return go_scan<__half>(l, s);
    default: return go_scan<__nv_bfloat16>(l, s);
  }
}

cudaError_t launch_linear_combine(const void* args, cudaStream_t s) {
  const LinLaunch& l = *(const LinLaunch*)args;
  int size = 0;
  for (int i = 0; i < l.n; ++i) size = l.p[i].K * l.p[i].V > size ? l.p[i].K * l.p[i].V : size;
  const dim3 grid((unsigned)(l.grids * l.heads), (size + 255) / 256, l.n);
  k_combine<<<grid, 256, 0, s>>>(l);
  return cudaGetLastError();
}

}  // namespace tb
