// Linear attention with a decay for each head: the single-token step, the
// recurrence over rows (tb_linattn_scan.cuh) and the joining of segments.
//
// Step: 8 bytes per state element and nothing else of size, so the bound is
// memory.  A block takes one state [key, value]; every thread keeps its loads
// of a column group in flight together, updates them, writes them back and
// adds its share of q S, which the block joins in shared memory.  Measured:
// 256 streams of 16 heads of 128 x 128 in 82 us, 97% of copy bandwidth.
#include "tb_linattn.cuh"
#include "tb_linattn_scan.cuh"
#include "tb_seq.cuh"

namespace tb {
namespace {

// ---------------------------------------------------------------- one token

constexpr int kStepThreads = 256;

// kBatch: state vectors in flight per thread.
template <class T, int V, int kStepBatch>
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
        float f[V];
        unpack<float, V>(x[i], f);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          f[j] = fmaf(f[j], decay, kk * vv[j]);
          o[j] = fmaf(qq, f[j], o[j]);
        }
        store_pack<float, V>(state + (int64_t)r * a.value, pack<float, V>(f));
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
  // as many vectors as a thread has of the state, up to 8: with more the registers leave too few blocks
  const bool vec = l.a.value % 4 == 0;
  const int rows = kStepThreads / (vec ? l.a.value / 4 : l.a.value), sweep = (l.a.key + rows - 1) / rows;
  if (!vec) k_step<T, 1, 8><<<blocks, kStepThreads, 0, s>>>(l);
  else if (sweep <= 4) k_step<T, 4, 4><<<blocks, kStepThreads, 0, s>>>(l);
  else k_step<T, 4, 8><<<blocks, kStepThreads, 0, s>>>(l);
  return cudaGetLastError();
}

// ------------------------------------------------------------- the recurrence

template <class T, int KS>
__global__ void __launch_bounds__(256) k_scan(LinLaunch l) {
  __shared__ __align__(16) float s_rows[scan_floats(KS)];
  const LinProblem& p = l.p[blockIdx.z];
  const LinSegment seg = lin_segment(l, blockIdx.x);
  // the first grid's block has the rows before it, the last one's those past it: few, where grids are short (512 grids of 8
  // rows, 8 heads of 128 x 128: 97 us, 96 without)
  if ((blockIdx.x == 0 && seg.begin > 0) || (blockIdx.x + 1 == gridDim.x && seg.end < l.tokens))
    lin_zero_rows<typename LinBits<sizeof(T)>::type>(
        p, {seg.begin, seg.end}, blockIdx.x == 0 ? 0 : seg.begin,
        blockIdx.x + 1 == gridDim.x ? seg.begin + l.tokens - seg.end : seg.begin, blockIdx.y, 1, threadIdx.x, blockDim.x);
  scan_walk<T, KS>(l, p, seg, blockIdx.y, s_rows, blockDim.x);
}

constexpr int kCombineBatch = 8;

// Joins the segments of a split call: the state that enters each segment, in
// place of the segment's own, and the state that leaves the grid.  A thread
// takes N elements of a state, and loads a batch of the segments' own ahead of
// the chain that joins them: 40 MB of states in 18 us an element at a time.
template <int N>
__global__ void __launch_bounds__(256) k_combine(LinLaunch l) {
  let_next_kernel_start();
  const LinProblem& p = l.p[blockIdx.z];
  const int b = blockIdx.x / l.heads, h = blockIdx.x % l.heads;
  const int slot0 = lin_first_slot(l, b);
  int64_t begin, end;
  lin_grid_rows(l, b, begin, end);
  // offsets that decrease name rows twice: their segments are more than the slots, which bound the walk
  const int n = min(lin_segments_of(l, end - begin), max(0, l.segments - slot0));
  const float decay = l.decay[h];
  const float whole = lin_power(decay, (float)l.segment);
  const float rest = lin_power(decay, (float)(end - begin - (int64_t)(n - 1) * l.segment));
  const int size = p.K * p.V;
  const int64_t state_at = ((int64_t)b * l.heads + h) * size;
  const int i = (blockIdx.y * blockDim.x + threadIdx.x) * N;
  if (i >= size) return;
  wait_for_last_kernel();
  float x[N];
#pragma unroll
  for (int k = 0; k < N; ++k)
    x[k] = p.first ? p.first[state_at + (i + k) / p.V * p.first_k + (i + k) % p.V * p.first_v] : 0.f;
  float* at = p.seg + ((int64_t)slot0 * l.heads + h) * size + i;
  const int64_t next = (int64_t)l.heads * size;
  const int own_count = n - (p.last ? 0 : 1);  // the last segment's own state is made where it is asked for
  for (int s0 = 0; s0 < n; s0 += kCombineBatch) {
    Pack<float, N> own[kCombineBatch];
#pragma unroll
    for (int j = 0; j < kCombineBatch; ++j)
      if (s0 + j < own_count) own[j] = load_pack<float, N>(at + (s0 + j) * next);
#pragma unroll
    for (int j = 0; j < kCombineBatch; ++j)
      if (s0 + j < n) {
        store_pack<float, N>(at + (s0 + j) * next, pack<float, N>(x));
        float f[N];
        if (s0 + j < own_count) unpack<float, N>(own[j], f);
#pragma unroll
        for (int k = 0; k < N; ++k)
          x[k] = fmaf(x[k], s0 + j + 1 == n ? rest : whole, s0 + j < own_count ? f[k] : 0.f);
      }
  }
  if (p.last) store_pack<float, N>(p.last + state_at + i, pack<float, N>(x));
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
  bool vec = true;
  for (int i = 0; i < l.n; ++i) {
    size = l.p[i].K * l.p[i].V > size ? l.p[i].K * l.p[i].V : size;
    vec = vec && l.p[i].K * l.p[i].V % 4 == 0 && ((uintptr_t)l.p[i].last & 15) == 0;
  }
  const int n = vec ? 4 : 1;
  const dim3 grid((unsigned)(l.grids * l.heads), (size + 256 * n - 1) / (256 * n), l.n);
  return launch_early(vec ? k_combine<4> : k_combine<1>, grid, 256, 0, s, true, l);
}

}  // namespace tb
