// Selective scan: the joining of the segments of a split call, forward for the
// states and, in the gradient, backward for what the chunks carry.
#include "tb_scan.cuh"

namespace tb {
namespace {

constexpr int kBatch = 8;

// The state that each segment starts from (or what enters it from behind), in
// place of its own: X = exp(a sum) X + own along a grid.  A thread takes four
// states of a channel of a grid, and loads a batch of the segments' own ahead
// of the chain that joins them.  least: the first segment whose own joins;
// first, last: the state that enters and the place of the one that comes out,
// [grids, channels, states] or NULL.
template <bool kBack>
__device__ __forceinline__ void join(const ScanLaunch& l, float* seg, int b, int64_t i, const float* first, float* last) {
  const tb_scan_args& a = l.a;
  const int per_channel = l.pad / 4;
  const int64_t place = i / per_channel;
  if (place >= l.wide) return;
  const int s = (int)(i - place * per_channel) * 4, group = (int)(place / l.group_pad), in = (int)(place - (int64_t)group * l.group_pad);
  const int per = a.channels / a.groups;
  const int64_t c = (int64_t)group * per + in, state_at = ((int64_t)b * a.channels + c) * a.states + s;
  const int slot0 = scan_first_slot(l, b);
  int64_t begin, end;
  lin_grid_rows(l, b, begin, end);
  const int n = scan_segments_of(l, end - begin);
  float a2[4], x[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const bool is = in < per && s + k < a.states;
    a2[k] = is ? scan_rate(a.a[c * a.states + s + k]) : 0.f;
    x[k] = is && first ? first[state_at + k] : 0.f;
  }
  wait_for_last_kernel();
  const int64_t next = kBack ? -(int64_t)l.wide * l.pad : (int64_t)l.wide * l.pad;
  const int64_t from = slot0 + (kBack ? n - 1 : 0);
  float* at = seg + (from * l.wide + place) * l.pad + s;
  const float* sum = l.sum + from * l.wide + place;
  const int64_t next_sum = kBack ? -(int64_t)l.wide : (int64_t)l.wide;
  const int count = last ? n : n - 1;  // the last one's own is made where it is asked for
  for (int j0 = 0; j0 < n; j0 += kBatch) {
    float4 own[kBatch];
    float d[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (j0 + j < count) {
        own[j] = *reinterpret_cast<const float4*>(at + (j0 + j) * next);
        d[j] = sum[(j0 + j) * next_sum];
      }
    float most = 0.f;  // one question for a batch: its decays stay ahead of the chain
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (j0 + j < count)
#pragma unroll
        for (int k = 0; k < 4; ++k) most = fmaxf(most, scan_exponent(d[j], a2[k]));
    if (most > kMostExponent) {  // one by one, read again: few calls come here
#pragma unroll 1
      for (int j = j0; j < min(j0 + kBatch, n); ++j) {
        float f[4];
        if (j < count) read_numbers<4>(f, at + j * next);
        write_numbers<4>(at + j * next, x);
        if (j < count)
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = scan_carried(sum[j * next_sum], a2[k], x[k], f[k]);
      }
      continue;
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (j0 + j < n) {
        *reinterpret_cast<float4*>(at + (j0 + j) * next) = make_float4(x[0], x[1], x[2], x[3]);
        if (j0 + j < count) {
          const float f[4] = {own[j].x, own[j].y, own[j].z, own[j].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = fmaf(scan_decay(d[j], a2[k]), x[k], f[k]);
        }
      }
  }
  if (last && in < per)
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (s + k < a.states) last[state_at + k] = x[k];
}

constexpr int kThreads = 128;
__device__ __forceinline__ int64_t items(const ScanLaunch& l) { return (int64_t)l.wide * (l.pad / 4); }

__global__ void __launch_bounds__(kThreads) k_scan_join(ScanLaunch l) {
  let_next_kernel_start();
  const int blocks = (int)((items(l) + kThreads - 1) / kThreads);
  join<false>(l, l.seg, blockIdx.x / blocks, (int64_t)(blockIdx.x % blocks) * kThreads + threadIdx.x, l.a.state, nullptr);
}
__global__ void __launch_bounds__(kThreads) k_scan_back_join(ScanBackwardLaunch g) {
  let_next_kernel_start();
  const ScanLaunch& l = g.f;
  const int blocks = (int)((items(l) + kThreads - 1) / kThreads), b = blockIdx.x / blocks;
  const int64_t i = (int64_t)(blockIdx.x % blocks) * kThreads + threadIdx.x;
  if (blockIdx.y) join<true>(l, g.seg_back, b, i, g.g.dstate_out, g.g.dstate);
  else join<false>(l, l.seg, b, i, l.a.state, nullptr);
}
unsigned join_blocks(const ScanLaunch& l) {
  return (unsigned)(((int64_t)l.wide * (l.pad / 4) + kThreads - 1) / kThreads * l.grids);
}

}  // namespace

cudaError_t launch_scan_join(const void* args, cudaStream_t s) {
  const ScanLaunch& l = *(const ScanLaunch*)args;
  return launch_early(k_scan_join, join_blocks(l), kThreads, 0, s, true, l);
}
cudaError_t launch_scan_back_join(const void* args, cudaStream_t s) {
  const ScanBackwardLaunch& g = *(const ScanBackwardLaunch*)args;
  return launch_early(k_scan_back_join, dim3(join_blocks(g.f), 2), kThreads, 0, s, true, g);
}

}  // namespace tb
