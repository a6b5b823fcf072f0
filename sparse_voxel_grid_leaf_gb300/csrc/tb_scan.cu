// Selective scan: the walk over rows, the joining of segments and the step for
// single tokens (tb_selective_scan, tb_selective_scan_step).
//
//   h_t = exp(delta_t a) h_(t-1) + delta_t x_t b_t,  y_t = (c_t . h_t + d x_t) silu(z_t)
//
// The states stay in registers (tb_scan.cuh); rows come through shared memory,
// eight at a time, the next ones on their way while eight are walked.  A call
// with few grids and channels is split along the rows: the segments' own last
// states first (from zero), their joining, then the outputs.  A segment's decay
// as a whole is exp(a sum of delta), so joining needs the sum alone.
//
// A row of 64 channels and 16 states takes 148 instructions in the states' pass,
// 284 cycles a scheduler: of those 62 paired multiply-adds at their rate (2.45
// cycles each) would take 53%, 36 exponentials and quotients (4 cycles) 51%; the
// counters have the issue slots 56% and the exponentials 56% busy, and in the
// outputs' pass (205 instructions, 420 cycles, 36 bytes spilled a thread in 16
// bits) 54 and 41%.  Nothing is full; which wait leads was not measured.  A prompt
// of 65537 rows, 2048 channels in bf16 is 1.10 ms, where its bytes alone would be
// 0.16.
//
// Past 16 states a warp takes its channels' states in blocks of 16, in turn for
// every eight rows, and fewer warps run: a prompt of 16384 rows, 2048 channels
// 0.31 ms with 16 states, 0.64 with 32, 1.39 with 64, 2.83 with 128.
#include "tb_scan.cuh"

namespace tb {
namespace {

constexpr int CH = kScanChannels;

// One warp's shared memory.  kParts: rows whose sums wait for their outputs.
template <class T, int NN, int kParts>
struct alignas(16) WalkShared {
  T raw[2][kParts ? 3 : 2][kTileRows][CH];  // x, dt, z of two tiles
  float delta[kTileRows][CH], dx[kTileRows][CH];
  float b[kTileRows][2 * NN], c[kParts ? kTileRows : 1][2 * NN];
  float part[kParts ? kParts : 1][2][CH];  // c . h over a lane's states
};
template <int NN>
constexpr int kept_floats() { return 32 * 4 * NN; }  // of a warp's states of a pass

// What a walk does: the outputs from the states that the segments start from
// (kOut); the segments' own last states from zero and their sums of delta
// (kStates); and those before every tile as well, for the gradient (kTiles).
enum Walk { kOut, kStates, kTiles };

template <Walk kWalk, bool kMany>
constexpr int parts_rows() { return kWalk != kOut ? 0 : kMany ? kTileRows : kTileRows / 2; }

// kMany: more states than a pass takes; those of a tile wait in shared memory
// (after the warps' own part) while the others' pass.
template <class T, int NN, Walk kWalk, bool kMany>
__global__ void __launch_bounds__(128, kMany ? 2 : 4) k_scan(ScanLaunch l) {
  extern __shared__ __align__(16) char s_raw[];
  constexpr bool kGives = kWalk == kOut;
  constexpr int kParts = parts_rows<kWalk, kMany>(), kRows = kGives ? kParts : kTileRows;  // at a time
  typedef WalkShared<T, NN, kParts> Shared;
  let_next_kernel_start();
  const tb_scan_args& a = l.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Shared& s = reinterpret_cast<Shared*>(s_raw)[warp];
  const int blocks = kMany ? l.pad / (2 * NN) : 1;  // of states
  float* s_h = reinterpret_cast<float*>(s_raw + l.warps * sizeof(Shared)) + warp * blocks * kept_floats<NN>();
  const int slot = (int)(blockIdx.x / l.blocks_x), at = (int)(blockIdx.x % l.blocks_x) * l.warps + warp;
  const ScanTile t = scan_tile<CH>(l, at / l.group_tiles, at % l.group_tiles);
  if (t.group >= a.groups) return;
  const int c4 = lane / 2 * 4, s0 = lane % 2 * NN;
  const f32x2 bias = channel_pair<CH>(a.dt_bias, t), skip = channel_pair<CH>(kGives ? a.d : nullptr, t);
  float rate[4][NN];  // on their way while the segment is found
  if (!kMany) read_dense<NN>(rate, a.a, t, a.states, c4, s0);
  const LinSegment seg = scan_segment_of(l, slot);
  if (kGives) scan_zero_share<T, CH>(l, a.y, a.y_row, slot, t);
  if (seg.grid < 0 || (kWalk == kStates && seg.index + 1 == seg.count)) return;  // the last one's own state joins no other
  const int64_t row0 = seg.begin + seg.first, state_at = (int64_t)seg.grid * a.channels * a.states;
  const int64_t mine = (t.place + c4) * l.pad + s0;  // the lane's place in a slot of the workspace
  float* const own = l.seg + (int64_t)slot * l.wide * l.pad + mine;
  f32x2 h[4][NN / 2] = {}, a2[4][NN / 2];
  auto as_pairs = [&](f32x2(&p)[4][NN / 2], const float(&f)[4][NN]) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int n = 0; n < NN; n += 2) p[j][n / 2] = pair(f[j][n], f[j][n + 1]);
  };
  auto rates = [&](int n0) {
    if (kMany) read_dense<NN>(rate, a.a, t, a.states, c4, n0 + s0);
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int n = 0; n < NN; n += 2) a2[j][n / 2] = pair(scan_rate(rate[j][n]), scan_rate(rate[j][n + 1]));
  };
  auto first = [&](int n0) {
    if (!kGives) return;
    float f[4][NN];
    if (l.segment) {
#pragma unroll
      for (int j = 0; j < 4; ++j) read_numbers<NN>(f[j], own + n0 + j * l.pad);
    } else {
      read_dense<NN>(f, a.state ? a.state + state_at : nullptr, t, a.states, c4, n0 + s0);
    }
    as_pairs(h, f);
  };
  auto write = [&](float* to) {  // in the workspace
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int n = 0; n < NN / 2; n += 2) write_pairs(to + j * l.pad + 2 * n, h[j][n], h[j][n + 1]);
  };
  auto keep = [&](int k) {
#pragma unroll
    for (int i = 0; i < NN; ++i)
      write_pairs(s_h + k * kept_floats<NN>() + (i * 32 + lane) * 4, h[i * 2 / (NN / 2)][i * 2 % (NN / 2)], h[i * 2 / (NN / 2)][i * 2 % (NN / 2) + 1]);
  };
  auto kept = [&](int k) {
#pragma unroll
    for (int i = 0; i < NN; ++i) {
      f32x2 f[2];
      read_pairs<2>(f, s_h + k * kept_floats<NN>() + (i * 32 + lane) * 4);
      h[i * 2 / (NN / 2)][i * 2 % (NN / 2)] = f[0], h[i * 2 / (NN / 2)][i * 2 % (NN / 2) + 1] = f[1];
    }
  };
  const int tiles = (seg.len + kTileRows - 1) / kTileRows;
  auto fetch = [&](int i) {
    const int n = min(kTileRows, seg.len - i * kTileRows);
    if (n > 0) {
      const int64_t row = row0 + (int64_t)i * kTileRows;
      auto& raw = s.raw[i & 1];
      scan_fetch<T, CH>(&raw[0][0][0], a.x, a.x_row, row, n, t, l.vec);
      scan_fetch<T, CH>(&raw[1][0][0], a.dt, a.dt_row, row, n, t, l.vec);
      if constexpr (kGives)
        if (a.z) scan_fetch<T, CH>(&raw[2][0][0], a.z, a.z_row, row, n, t, l.vec);
    }
    copies_on_their_way();
  };
  ScanStates<T, 2 * NN> nb(a.b, a.b_row, t.group * a.b_group, row0, a.states, 0), nc(a.c, a.c_row, t.group * a.c_group, row0, a.states, 0);
  auto load_states = [&](int i, int n0) {
    const int n = min(kTileRows, seg.len - i * kTileRows);
    if (kMany) {
      nb = ScanStates<T, 2 * NN>(a.b, a.b_row, t.group * a.b_group, row0, a.states, n0);
      if (kGives) nc = ScanStates<T, 2 * NN>(a.c, a.c_row, t.group * a.c_group, row0, a.states, n0);
    }
    nb.load(i * kTileRows, n);
    if (kGives) nc.load(i * kTileRows, n);
  };
  PairOut<T, CH> out(a.y, a.y_row, row0, t);
  f32x2 total = 0;
  fetch(0);
  load_states(0, 0);
  if (kGives) wait_for_last_kernel();  // for what the segments start from; what is read above, no kernel of the call writes
  if (kMany) {
    for (int k = 0; k < blocks; ++k) {
      first(k * 2 * NN);
      keep(k);
    }
  } else {
    rates(0);
    first(0);
  }
  for (int i = 0; i < tiles; ++i) {
    const int n = min(kTileRows, seg.len - i * kTileRows);
    fetch(i + 1);
    if (kWalk == kTiles && i) {
      const int64_t tile = scan_tile_place(row0, i);
      if (!kMany) write(l.tile + tile * l.wide * l.pad + mine);
      *reinterpret_cast<f32x2*>(l.tile_sum + tile * l.wide + t.place + 2 * lane) = total;
    }
    wait_for_copies<1>();
    auto& raw = s.raw[i & 1];
#pragma unroll
    for (int r = 0; r < kTileRows; ++r) {
      f32x2 delta = scan_step_of(row_pair<T, CH>(raw[1][r]), bias, a.softplus);
      if (r >= n) delta = 0;
      total = add2(total, delta);
      pair_of<CH>(s.delta[r]) = delta;
      pair_of<CH>(s.dx[r]) = mul2(delta, row_pair<T, CH>(raw[0][r]));
    }
    auto walk = [&](int r, int k) {
      float d[4], x[4], y[4];
      f32x2 b[NN / 2], c[NN / 2];
      read_numbers<4>(d, &s.delta[r][c4]);
      read_numbers<4>(x, &s.dx[r][c4]);
      read_pairs<NN / 2>(b, &s.b[r][s0]);
      if constexpr (kGives) read_pairs<NN / 2>(c, &s.c[r][s0]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 dd = both(d[j]), xx = both(x[j]);
        f32x2 sum = 0;
#pragma unroll
        for (int m = 0; m < NN / 2; ++m) {
          h[j][m] = fma2(scan_decay(dd, a2[j][m]), h[j][m], mul2(xx, b[m]));
          if (kGives) sum = m ? fma2(c[m], h[j][m], sum) : mul2(c[m], h[j][m]);
        }
        const float2 f = halves(sum);
        y[j] = f.x + f.y;
      }
      if constexpr (kGives) {
        float* to = &s.part[r % kRows][lane % 2][c4];
        if (kMany && k) {
          float f[4];
          read_numbers<4>(f, to);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[j] += f[j];
        }
        write_numbers<4>(to, y);
      }
    };
    auto give = [&](int r) {
      f32x2 y = add2(pair_of<CH>(s.part[r % kRows][0]), pair_of<CH>(s.part[r % kRows][1]));
      y = fma2(skip, row_pair<T, CH>(raw[0][r]), y);
      if (a.z) y = mul2(y, scan_gate(row_pair<T, CH>(raw[2][r])));
      if (r < n) out.put(r, y);
    };
    for (int k = 0; k < blocks; ++k) {
      nb.store(s.b);
      if constexpr (kGives) nc.store(s.c);
      __syncwarp();
      if (kMany) {
        rates(k * 2 * NN);
        kept(k);
        if (kWalk == kTiles && i) write(l.tile + scan_tile_place(row0, i) * l.wide * l.pad + mine + k * 2 * NN);
      }
      if (kMany && k + 1 < blocks) load_states(i, (k + 1) * 2 * NN);
      else load_states(i + 1, 0);
#pragma unroll
      for (int r0 = 0; r0 < kTileRows; r0 += kRows) {
#pragma unroll
        for (int r = r0; r < r0 + kRows; ++r) walk(r, k);
        if (kMany) keep(k);
        __syncwarp();
        if (kGives && k + 1 == blocks) {
#pragma unroll
          for (int r = r0; r < r0 + kRows; ++r) give(r);
          __syncwarp();
        }
      }
    }
    out.at += kTileRows * out.stride;
  }
  wait_for_copies<0>();
  const bool ends = kGives && a.state_out && seg.index + 1 == seg.count;
  if (!kGives || ends)
    for (int k = 0; k < blocks; ++k) {
      if (kMany) kept(k);
      if (!kGives) {
        write(own + k * 2 * NN);
      } else {
        float f[4][NN];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int m = 0; m < NN / 2; ++m) {
            const float2 v = halves(h[j][m]);
            f[j][2 * m] = v.x, f[j][2 * m + 1] = v.y;
          }
        write_dense<NN>(a.state_out + state_at, f, t, a.states, c4, k * 2 * NN + s0);
      }
    }
  if (!kGives) *reinterpret_cast<f32x2*>(l.sum + (int64_t)slot * l.wide + t.place + 2 * lane) = total;
}

template <class T, int NN, Walk kWalk, bool kMany>
cudaError_t go(const ScanLaunch& l, cudaStream_t s) {
  size_t bytes = l.warps * sizeof(WalkShared<T, NN, parts_rows<kWalk, kMany>()>);
  if (kMany) bytes += (size_t)l.warps * (l.pad / (2 * NN)) * kept_floats<NN>() * sizeof(float);
  static std::atomic<bool> ready[kMaxDevices];
  const cudaError_t e = allow_shared(k_scan<T, NN, kWalk, kMany>, 227 * 1024, ready);
  if (e != cudaSuccess) return e;
  return launch_early(k_scan<T, NN, kWalk, kMany>, (unsigned)((int64_t)l.segments * l.blocks_x), 32 * l.warps, bytes, s,
                      kWalk == kOut && l.segment != 0, l);
}
template <class T, Walk kWalk>
cudaError_t pick(const ScanLaunch& l, cudaStream_t s) {
  if (l.pass == 8) return go<T, 4, kWalk, false>(l, s);
  return l.pad == 16 ? go<T, 8, kWalk, false>(l, s) : go<T, 8, kWalk, true>(l, s);
}
template <Walk kWalk>
cudaError_t by_type(const ScanLaunch& l, cudaStream_t s) {
  switch (l.a.type) {
    case TB_TYPE_F32: return pick<float, kWalk>(l, s);
    case TB_TYPE_F16: return pick<__half, kWalk>(l, s);
    default: return pick<__nv_bfloat16, kWalk>(l, s);
  }
}

// ---------------------------------------------------------------- one token
//
// 8 bytes a state and nothing else of size: the bound is memory.  Four lanes
// take a channel, four states at a time each, of four streams at once: a lane
// makes the step and the gate of one of the streams (by every lane they took
// more instructions than the states), and the states of all four are on their
// way together.  256 streams of 2048 channels and 16 states: 12.5 us, 5.7 TB/s
// (17.3 with each lane making every stream's step).  kVec: states, b and c by
// vectors of four, up to 16 states a channel (a lane's rates stay in registers);
// element by element 64 states of those streams take 108 us, where their bytes
// take 41.
constexpr int kStepThreads = 128;

template <class T, bool kVec>
__global__ void __launch_bounds__(kStepThreads) k_scan_step(ScanStepLaunch l) {
  const tb_scan_step_args& a = l.a;
  const int blocks_x = (a.channels + 31) / 32, lane = threadIdx.x % 4, s4 = lane * 4;
  const int c = (int)(blockIdx.x % blocks_x) * 32 + threadIdx.x / 4;
  const int64_t n0 = (int64_t)(blockIdx.x / blocks_x) * l.per_block, n1 = min(n0 + l.per_block, a.streams);
  const bool live = c < a.channels, mine = live && s4 < a.states;
  const int group = live ? c / (a.channels / a.groups) : 0;
  const float bias = live && a.dt_bias ? a.dt_bias[c] : 0.f, skip = live && a.d ? a.d[c] : 0.f;
  const float* rate = a.a + (int64_t)c * a.states;
  float a2[4] = {};
  if (kVec && mine) {
    unpack<float, 4>(load_pack<float, 4>(rate + s4), a2);
#pragma unroll
    for (int k = 0; k < 4; ++k) a2[k] = scan_rate(a2[k]);
  }
  for (int64_t n = n0; n < n1; n += 4) {
    // the lane's own stream of the four
    const int64_t own = n + lane;
    int64_t slot = own >= n1 || !live ? -1 : a.slots ? (int64_t)a.slots[own] : own;
    if (slot >= a.num_slots || slot < 0) slot = -1;
    int64_t at[4];  // of each one's states, -1: none
#pragma unroll
    for (int j = 0; j < 4; ++j) at[j] = __shfl_sync(0xffffffffu, slot, j, 4);
    Pack<float, 4> hp[4];
    Pack<T, 4> bp[4], cp[4];
    const T* const b = (const T*)a.b + n * a.b_row + group * a.b_group;
    const T* const cc = (const T*)a.c + n * a.c_row + group * a.c_group;
    if (kVec && mine) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (at[j] >= 0) {
          hp[j] = load_pack<float, 4>(a.state + (at[j] * a.channels + c) * (int64_t)a.states + s4);
          bp[j] = load_pack<T, 4>(b + j * a.b_row + s4);
          cp[j] = load_pack<T, 4>(cc + j * a.c_row + s4);
        }
    }
    float x = 0.f, delta = 0.f, z = 0.f;
    if (slot >= 0) {
      x = RowType<T>::to(((const T*)a.x)[own * a.x_row + c]);
      delta = RowType<T>::to(((const T*)a.dt)[own * a.dt_row + c]) + bias;
      if (a.z) z = RowType<T>::to(((const T*)a.z)[own * a.z_row + c]);
      if (a.softplus) delta = scan_softplus(delta);
    }
    const float dx = delta * x;
    float sum[4] = {};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float dj = __shfl_sync(0xffffffffu, delta, j, 4), xj = __shfl_sync(0xffffffffu, dx, j, 4);
      if (at[j] < 0) continue;
      float* const h = a.state + (at[j] * a.channels + c) * (int64_t)a.states;
      if (kVec) {
        if (mine) {
          float f[4], g[4], r[4];
          unpack<float, 4>(hp[j], f);
          unpack<T, 4>(bp[j], g);
          unpack<T, 4>(cp[j], r);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            f[k] = fmaf(scan_decay(dj, a2[k]), f[k], xj * g[k]);
            sum[j] = fmaf(r[k], f[k], sum[j]);
          }
          store_pack<float, 4>(h + s4, pack<float, 4>(f));
        }
      } else {
        for (int s = lane; s < a.states; s += 4) {
          const float f = fmaf(scan_decay(dj, scan_rate(rate[s])), h[s], xj * RowType<T>::to(b[j * a.b_row + s]));
          sum[j] = fmaf(RowType<T>::to(cc[j * a.c_row + s]), f, sum[j]);
          h[s] = f;
        }
      }
    }
    // to each lane the sum of its own stream
    float even = lane & 1 ? sum[1] : sum[0], odd = lane & 1 ? sum[3] : sum[2];
    even += __shfl_xor_sync(0xffffffffu, lane & 1 ? sum[0] : sum[1], 1);
    odd += __shfl_xor_sync(0xffffffffu, lane & 1 ? sum[2] : sum[3], 1);
    float y = lane & 2 ? odd : even;
    y += __shfl_xor_sync(0xffffffffu, lane & 2 ? even : odd, 2);
    if (live && own < n1) {
      y = fmaf(skip, x, y);
      if (a.z) y *= z * scan_sigmoid(z);
      ((T*)a.y)[own * a.y_row + c] = RowType<T>::from(slot >= 0 ? y : 0.f);
    }
  }
}

}  // namespace

cudaError_t launch_scan(const void* args, cudaStream_t s) { return by_type<kOut>(*(const ScanLaunch*)args, s); }
cudaError_t launch_scan_states(const void* args, cudaStream_t s) {
  const ScanLaunch& l = *(const ScanLaunch*)args;
  return l.tile ? by_type<kTiles>(l, s) : by_type<kStates>(l, s);
}

cudaError_t launch_scan_step(const void* args, cudaStream_t s) {
  const ScanStepLaunch& l = *(const ScanStepLaunch*)args;
  const int64_t blocks = (l.a.channels + 31) / 32 * ((l.a.streams + l.per_block - 1) / l.per_block);
  auto go = [&](auto four, auto one) {
    if (l.vec) four<<<(unsigned)blocks, kStepThreads, 0, s>>>(l);
    else one<<<(unsigned)blocks, kStepThreads, 0, s>>>(l);
    return cudaGetLastError();
  };
  switch (l.a.type) {
    case TB_TYPE_F32: return go(k_scan_step<float, true>, k_scan_step<float, false>);
    case TB_TYPE_F16: return go(k_scan_step<__half, true>, k_scan_step<__half, false>);
    default: return go(k_scan_step<__nv_bfloat16, true>, k_scan_step<__nv_bfloat16, false>);
  }
}

}  // namespace tb
