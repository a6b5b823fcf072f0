// The gradient of the selective scan (tb_selective_scan_backward).
//
// With ds = dy silu(z), s_t = c_t . h_t + d x_t and
//   g_t = c_t ds_t + exp(delta_(t+1) a) g_(t+1)
// per channel and state:
//   db_t = sum over channels g delta x,  dc_t = sum over channels ds h,
//   into = g . b,  dx = d ds + delta into,  q = g exp(delta a) h_(t-1),
//   ddelta = a . q + x into,  da = sum over rows q delta,  dz = dy s silu'(z).
//
// The rows are taken in chunks.  First every chunk's own states from zero,
// before every tile of kTileRows rows (tb_scan.cu), and its own part of the
// carried exp(delta a) g (k_scan_carry), then their joining along the grids,
// forward and backward (tb_scan_join.cu); then all chunks at once, each with
// what enters it from both sides, tile by tile from its last one.  The states
// before a tile are its own part and what the chunk started from, decayed by
// the sum of delta between.  Sums over channels go through shared memory over a
// block's four warps, and over blocks through parts that a last kernel adds in
// a fixed order.
//
// A row of 32 channels takes some 360 instructions here; the registers leave
// two blocks of four warps a multiprocessor, whose waits for one another's
// results leave the issue slots 40% busy.  16 grids of 124807 rows, 1024
// channels of 16 states in bf16: 3.8 ms for all of it, of which this kernel 2.8,
// the chunks' states 0.47 and what they carry 0.43.  More than 16 states are
// taken in blocks of 16, all rows for each: forward and gradient of 16384 rows,
// 1024 channels 0.73 ms with 16, 3.30 with 64.
#include "tb_scan.cuh"

namespace tb {
namespace {

constexpr int kWarps = 4;

// ------------------------------------------------- what the chunks carry back

template <class T, int NN>
struct alignas(16) CarryShared {
  T raw[2][3][kTileRows][kScanChannels];  // dt, dy, z of two tiles
  float delta[kTileRows][kScanChannels], ds[kTileRows][kScanChannels];
  float c[kTileRows][2 * NN];
};

// One block of states a warp (blockIdx.y), as the walks are short.  It needs
// nothing of the chunks' own states and runs beside their kernel, whose end it
// waits for at its own: the joining needs both.
template <class T, int NN>
__global__ void __launch_bounds__(32 * kWarps) k_scan_carry(ScanBackwardLaunch g) {
  extern __shared__ __align__(16) char s_raw[];
  constexpr int CH = kScanChannels;
  let_next_kernel_start();
  const ScanLaunch& l = g.f;
  const tb_scan_args& a = l.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  CarryShared<T, NN>& s = reinterpret_cast<CarryShared<T, NN>*>(s_raw)[warp];
  const int blocks_x = (a.groups * l.group_tiles + kWarps - 1) / kWarps;
  const int slot = (int)(blockIdx.x / blocks_x), at = (int)(blockIdx.x % blocks_x) * kWarps + warp;
  const int n0 = blockIdx.y * 2 * NN;
  const ScanTile t = scan_tile<CH>(l, at / l.group_tiles, at % l.group_tiles);
  if (t.group >= a.groups) return;
  const int c4 = lane / 2 * 4, s0 = lane % 2 * NN;
  const f32x2 bias = channel_pair<CH>(a.dt_bias, t);
  float rate[4][NN];  // on their way while the segment is found
  read_dense<NN>(rate, a.a, t, a.states, c4, n0 + s0);
  const LinSegment seg = scan_segment_of(l, slot);
  if (seg.grid < 0 || (seg.index == 0 && !g.g.dstate)) {  // the first chunk's goes nowhere else
    wait_for_last_kernel();
    return;
  }
  const int64_t row0 = seg.begin + seg.first;
  f32x2 h[4][NN / 2] = {}, a2[4][NN / 2];
  const int tiles = (seg.len + kTileRows - 1) / kTileRows;
  auto fetch = [&](int i) {
    if (i >= 0) {
      const int n = min(kTileRows, seg.len - i * kTileRows);
      const int64_t row = row0 + i * kTileRows;
      auto& raw = s.raw[i & 1];
      scan_fetch<T, CH>(&raw[0][0][0], a.dt, a.dt_row, row, n, t, l.vec);
      scan_fetch<T, CH>(&raw[1][0][0], g.g.dy, g.g.dy_row, row, n, t, l.vec);
      if (a.z) scan_fetch<T, CH>(&raw[2][0][0], a.z, a.z_row, row, n, t, l.vec);
    }
    copies_on_their_way();
  };
  ScanStates<T, 2 * NN> nc(a.c, a.c_row, t.group * a.c_group, row0, a.states, n0);
  auto load_states = [&](int i) { nc.load(i * kTileRows, i < 0 ? 0 : min(kTileRows, seg.len - i * kTileRows)); };
  fetch(tiles - 1);
  load_states(tiles - 1);
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int m = 0; m < NN / 2; ++m) a2[j][m] = pair(scan_rate(rate[j][2 * m]), scan_rate(rate[j][2 * m + 1]));
  for (int i = tiles - 1; i >= 0; --i) {
    const int n = min(kTileRows, seg.len - i * kTileRows);
    fetch(i - 1);
    wait_for_copies<1>();
    auto& raw = s.raw[i & 1];
#pragma unroll
    for (int r = 0; r < kTileRows; ++r) {
      f32x2 ds = row_pair<T, CH>(raw[1][r]);
      if (a.z) ds = mul2(ds, scan_gate(row_pair<T, CH>(raw[2][r])));
      f32x2 delta = scan_step_of(row_pair<T, CH>(raw[0][r]), bias, a.softplus);
      if (r >= n) delta = ds = 0;
      pair_of<CH>(s.delta[r]) = delta;
      pair_of<CH>(s.ds[r]) = ds;
    }
    nc.store(s.c);
    __syncwarp();
    load_states(i - 1);
#pragma unroll
    for (int r = kTileRows - 1; r >= 0; --r) {
      float d[4], ds[4];
      f32x2 c[NN / 2];
      read_numbers<4>(d, &s.delta[r][c4]);
      read_numbers<4>(ds, &s.ds[r][c4]);
      read_pairs<NN / 2>(c, &s.c[r][s0]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 dd = both(d[j]), dsj = both(ds[j]);
#pragma unroll
        for (int m = 0; m < NN / 2; ++m) h[j][m] = mul2(scan_decay(dd, a2[j][m]), fma2(c[m], dsj, h[j][m]));
      }
    }
    __syncwarp();
  }
  wait_for_copies<0>();
  float* to = g.seg_back + ((int64_t)slot * l.wide + t.place + c4) * l.pad + n0 + s0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int m = 0; m < NN / 2; m += 2) write_pairs(to + j * l.pad + 2 * m, h[j][m], h[j][m + 1]);
  wait_for_last_kernel();
}

// ------------------------------------------------------------ all of a chunk

constexpr int CH = 32;  // channels of a warp

template <class T, int NN>
struct alignas(16) BackShared {
  float own[2][4][32 * NN], start[4][32 * NN];  // the states before two tiles, from zero, and before the chunk: by lanes
  float before[2][CH];                          // the sums of delta before the tiles
  float delta[kTileRows][CH], dx[kTileRows][CH], ds[kTileRows][CH];
  f32x2 b[kTileRows][4 * NN], c[kTileRows][4 * NN];
  float sums[2][3][4][CH];  // of two rows: a lane's c . h, g . b, a . q
  float bc[2][2][36 * NN];  // of two rows: a lane's channels of db, dc; on different banks
  T raw[2][4][kTileRows][CH];  // x, dt, z, dy of two tiles
};

// 4 NN bytes of the workspace.
template <int NN>
__device__ __forceinline__ void copy_states(float* dst, const float* src) {
  if constexpr (NN == 4) copy_row(dst, src, 16);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src) : "memory");
}

template <class T, int NN, bool kMany>
__global__ void __launch_bounds__(32 * kWarps, 2) k_scan_backward(ScanBackwardLaunch g) {
  extern __shared__ __align__(16) char s_raw[];
  typedef BackShared<T, NN> Shared;
  constexpr int kStates = 4 * NN;
  let_next_kernel_start();
  const ScanLaunch& l = g.f;
  const tb_scan_args& a = l.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, o = lane_row<CH>(), p = lane_pair<CH>();
  Shared& s = reinterpret_cast<Shared*>(s_raw)[warp];
  f32x2(*s_bc)[kTileRows][kStates] = reinterpret_cast<f32x2(*)[kTileRows][kStates]>(s_raw + kWarps * sizeof(Shared));
  const int per_run = a.groups * g.quads, run = (int)(blockIdx.x / per_run), at = (int)(blockIdx.x % per_run);
  const int group = at / g.quads, quad = at % g.quads;
  ScanTile t = scan_tile<CH>(l, group, quad * kWarps + warp);
  const bool placed = (quad * kWarps + warp) * CH < l.group_pad;  // in the workspace; past it the warp adds zeros
  if (!placed) t.place = (int64_t)group * l.group_pad, t.count = 0;
  const int c4 = lane / 4 * 4, s4 = lane % 4 * NN;
  const int64_t mine = (t.place + c4) * l.pad + s4;  // the lane's place in a slot of the workspace
  const f32x2 bias = channel_pair<CH>(a.dt_bias, t), skip = channel_pair<CH>(a.d, t);
  f32x2 sum_d = 0, sum_bias = 0;
  const int blocks = kMany ? l.pad / kStates : 1;
  for (int k = 0; k < blocks; ++k) {
    const int n0 = k * kStates;
    const bool last = k + 1 == blocks;
    f32x2 a2[2][NN], da[2][NN] = {};
    auto as_pairs = [&](f32x2(&h)[2][NN], const float(&f)[4][NN]) {
#pragma unroll
      for (int n = 0; n < NN; ++n) h[0][n] = pair(f[0][n], f[1][n]), h[1][n] = pair(f[2][n], f[3][n]);
    };
    auto nothing = [&](f32x2(&h)[2][NN]) {
#pragma unroll
      for (int n = 0; n < NN; ++n) h[0][n] = h[1][n] = 0;
    };
    {
      float f[4][NN];
      read_dense<NN>(f, a.a, t, a.states, c4, n0 + s4);
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int n = 0; n < NN; ++n) f[j][n] = scan_rate(f[j][n]);
      as_pairs(a2, f);
    }
    if (k == 0) wait_for_last_kernel();
    for (int slot = run * g.per_run; slot < min((run + 1) * g.per_run, l.segments); ++slot) {
      if (k == 0) {
        scan_zero_share<T, CH>(l, g.g.dx, g.g.dx_row, slot, t);
        scan_zero_share<T, CH>(l, g.g.ddt, g.g.ddt_row, slot, t);
        if (a.z) scan_zero_share<T, CH>(l, g.g.dz, g.g.dz_row, slot, t);
      }
      const LinSegment seg = scan_segment_of(l, slot);
      if (seg.grid < 0 || seg.len == 0) continue;
      const int64_t row0 = seg.begin + seg.first;
      const int tiles = (seg.len + kTileRows - 1) / kTileRows;
      const PairOut<T, CH> out_x(g.g.dx, g.g.dx_row, row0, t), out_dt(g.g.ddt, g.g.ddt_row, row0, t), out_z(g.g.dz, g.g.dz_row, row0, t);
      ScanStates<T, kStates> nb(a.b, a.b_row, t.group * a.b_group, row0, a.states, n0),
          nc(a.c, a.c_row, t.group * a.c_group, row0, a.states, n0);
      auto fetch = [&](int i) {
        if (i >= 0) {
          const int64_t row = row0 + i * kTileRows;
          const int n = min(kTileRows, seg.len - i * kTileRows);
          auto& raw = s.raw[i & 1];
          scan_fetch<T, CH>(&raw[0][0][0], a.x, a.x_row, row, n, t, l.vec);
          scan_fetch<T, CH>(&raw[1][0][0], a.dt, a.dt_row, row, n, t, l.vec);
          if (a.z) scan_fetch<T, CH>(&raw[2][0][0], a.z, a.z_row, row, n, t, l.vec);
          scan_fetch<T, CH>(&raw[3][0][0], g.g.dy, g.g.dy_row, row, n, t, l.vec);
          if (i) {
            const int64_t tile = scan_tile_place(row0, i);
            const float* from = l.tile + tile * l.wide * l.pad + mine + n0;
#pragma unroll
            for (int j = 0; j < 4; ++j) copy_states<NN>(&s.own[i & 1][j][lane * NN], from + j * l.pad);
            if (lane < CH / 4) copy_row(&s.before[i & 1][lane * 4], l.tile_sum + tile * l.wide + t.place + lane * 4, 16);
          }
        }
        copies_on_their_way();
      };
      auto load_states = [&](int i) {
        const int n = i < 0 ? 0 : min(kTileRows, seg.len - i * kTileRows);
        nb.load(i * kTileRows, n);
        nc.load(i * kTileRows, n);
      };
      f32x2 carry[2][NN], h[2][NN];
      {
        const int64_t at_slot = (int64_t)slot * l.wide * l.pad + mine + n0;
#pragma unroll
        for (int j = 0; j < 4; ++j) copy_states<NN>(&s.start[j][lane * NN], l.seg + at_slot + j * l.pad);
        fetch(tiles - 1);
        load_states(tiles - 1);
        float f[4][NN];
#pragma unroll
        for (int j = 0; j < 4; ++j) read_numbers<NN>(f[j], g.seg_back + at_slot + j * l.pad);
        as_pairs(carry, f);
        if (!placed) nothing(carry);
      }
      auto forward = [&](int r) {
        f32x2 d[2], x[2], b[NN];
        read_pairs<2>(d, &s.delta[r][c4]);
        read_pairs<2>(x, &s.dx[r][c4]);
        read_pairs<NN>(b, &s.b[r][s4]);
#pragma unroll
        for (int n = 0; n < NN; ++n)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            h[j][n] = fma2(scan_decay(d[j], a2[j][n]), h[j][n], mul2(x[j], b[n]));
          }
      };
      for (int i = tiles - 1; i >= 0; --i) {
        const int rows = min(kTileRows, seg.len - i * kTileRows);
        auto& raw = s.raw[i & 1];
        nb.store(s.b);
        nc.store(s.c);
        fetch(i - 1);
        load_states(i - 1);
        wait_for_copies<1>();
#pragma unroll
        for (int m = 0; m < kTileRows / 2; ++m) {
          const int r = 2 * m + o;
          f32x2 delta = scan_step_of(row_pair<T, CH>(raw[1][r]), bias, a.softplus), ds = row_pair<T, CH>(raw[3][r]);
          if (a.z) ds = mul2(ds, scan_gate(row_pair<T, CH>(raw[2][r])));
          if (r >= rows) delta = ds = 0;
          pair_of<CH>(s.delta[r]) = delta;
          pair_of<CH>(s.dx[r]) = mul2(delta, row_pair<T, CH>(raw[0][r]));
          pair_of<CH>(s.ds[r]) = ds;
        }
        // the states before the tile
        {
          float f[4][NN];
#pragma unroll
          for (int j = 0; j < 4; ++j) read_numbers<NN>(f[j], &s.start[j][lane * NN]);
          as_pairs(h, f);
          if (i) {
            f32x2 d[2], own[2][NN];
            read_pairs<2>(d, &s.before[i & 1][c4]);
#pragma unroll
            for (int j = 0; j < 4; ++j) read_numbers<NN>(f[j], &s.own[i & 1][j][lane * NN]);
            as_pairs(own, f);
            float most = 0.f;  // one question for all of them
#pragma unroll
            for (int n = 0; n < NN; ++n)
#pragma unroll
              for (int j = 0; j < 2; ++j) most = fmaxf(most, scan_exponent(d[j], a2[j][n]));
            if (most > kMostExponent) {
#pragma unroll
              for (int n = 0; n < NN; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) h[j][n] = scan_carried(d[j], a2[j][n], h[j][n], own[j][n]);
            } else {
#pragma unroll
              for (int n = 0; n < NN; ++n)
#pragma unroll
                for (int j = 0; j < 2; ++j) h[j][n] = fma2(scan_decay(d[j], a2[j][n]), h[j][n], own[j][n]);
            }
          }
        }
        if (!placed) nothing(h);
        f32x2 first[2][NN];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int n = 0; n < NN; ++n) first[j][n] = h[j][n];
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 4; ++r) forward(r);
#pragma unroll
        for (int half = 1; half >= 0; --half) {
          if (!half)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int n = 0; n < NN; ++n) h[j][n] = first[j][n];
          // the states before four rows and after each; their decays are made again on the way back (held in registers
          // too, they cost spills: 3.05 ms of the training step below, 2.8 so)
          f32x2 hs[5][2][NN];
#pragma unroll
          for (int r = 0; r <= 4; ++r) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int n = 0; n < NN; ++n) hs[r][j][n] = h[j][n];
            if (r < 4) forward(4 * half + r);
          }
#pragma unroll
          for (int r = 3; r >= 0; --r) {
            const int at_row = 4 * half + r;
            f32x2 d[2], x[2], ds[2], b[NN], c[NN], y[2] = {}, into[2] = {}, qa[2] = {};
            float db[NN], dc[NN];
            read_pairs<2>(d, &s.delta[at_row][c4]);
            read_pairs<2>(x, &s.dx[at_row][c4]);
            read_pairs<2>(ds, &s.ds[at_row][c4]);
            read_pairs<NN>(b, &s.b[at_row][s4]);
            read_pairs<NN>(c, &s.c[at_row][s4]);
#pragma unroll
            for (int n = 0; n < NN; ++n) {
              f32x2 sum_b = 0, sum_c = 0;
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const f32x2 grad = fma2(c[n], ds[j], carry[j][n]);
                y[j] = n ? fma2(c[n], hs[r + 1][j][n], y[j]) : mul2(c[n], hs[r + 1][j][n]);
                sum_c = j ? fma2(ds[j], hs[r + 1][j][n], sum_c) : mul2(ds[j], hs[r + 1][j][n]);
                sum_b = j ? fma2(grad, x[j], sum_b) : mul2(grad, x[j]);
                into[j] = n ? fma2(grad, b[n], into[j]) : mul2(grad, b[n]);
                carry[j][n] = mul2(grad, scan_decay(d[j], a2[j][n]));
                const f32x2 q = mul2(carry[j][n], hs[r][j][n]);
                qa[j] = n ? fma2(q, a2[j][n], qa[j]) : mul2(q, a2[j][n]);
                da[j][n] = fma2(q, d[j], da[j][n]);
              }
              const float2 fb = halves(sum_b), fc = halves(sum_c);
              db[n] = fb.x + fb.y;
              dc[n] = fc.x + fc.y;
            }
            write_pairs(&s.sums[r & 1][0][lane % 4][c4], y[0], y[1]);
            write_pairs(&s.sums[r & 1][1][lane % 4][c4], into[0], into[1]);
            write_pairs(&s.sums[r & 1][2][lane % 4][c4], qa[0], qa[1]);
#pragma unroll
            for (int n = 0; n < NN; n += 2) {
              const int to = lane / 4 * kStates + s4 + n;
              *reinterpret_cast<float2*>(&s.bc[r & 1][0][to]) = make_float2(db[n], db[n + 1]);
              *reinterpret_cast<float2*>(&s.bc[r & 1][1][to]) = make_float2(dc[n], dc[n + 1]);
            }
            if (r & 1) continue;
            __syncwarp();
            // the sums of two rows, one each half of the warp: by channels, then by states of db and dc
            const int rr = at_row + o;
            f32x2 sum[3];
#pragma unroll
            for (int v = 0; v < 3; ++v)
              sum[v] = add2(add2(pair_of<CH>(s.sums[o][v][0]), pair_of<CH>(s.sums[o][v][1])),
                            add2(pair_of<CH>(s.sums[o][v][2]), pair_of<CH>(s.sums[o][v][3])));
            const int to = i * kTileRows + rr;
            if (kMany && rr < rows) {
              float* acc = g.acc + ((row0 + to) * a.channels + t.first + 2 * p) * 3;
#pragma unroll
              for (int m = 0; m < 2; ++m)
                if (2 * p + m < t.count)
#pragma unroll
                  for (int v = 0; v < 3; ++v) {
                    float2 f = halves(sum[v]);
                    float& mine = m ? f.y : f.x;
                    if (k) mine += acc[3 * m + v];
                    if (!last) acc[3 * m + v] = mine;
                    sum[v] = pair(f.x, f.y);
                  }
            }
            if (rr < rows && last) {
              const f32x2 xf = row_pair<T, CH>(raw[0][rr]), dsf = pair_of<CH>(s.ds[rr]);
              const f32x2 inner = fma2(skip, xf, sum[0]);
              f32x2 ddt = fma2(xf, sum[1], mul2(sum[2], both(kLn2)));
              if (a.softplus) ddt = mul2(ddt, scan_sigmoid(add2(row_pair<T, CH>(raw[1][rr]), bias)));
              out_x.put(to, fma2(skip, dsf, mul2(pair_of<CH>(s.delta[rr]), sum[1])));
              out_dt.put(to, ddt);
              if (a.z) {
                const f32x2 z = row_pair<T, CH>(raw[2][rr]), sg = scan_sigmoid(z);
                const f32x2 slope = mul2(sg, fma2(z, fma2(sg, both(-1.f), both(1.f)), both(1.f)));
                out_z.put(to, mul2(mul2(row_pair<T, CH>(raw[3][rr]), inner), slope));
              }
              sum_d = fma2(dsf, xf, sum_d);
              sum_bias = add2(sum_bias, ddt);
            }
            if (p < kStates) {
              const f32x2* from = reinterpret_cast<const f32x2*>(&s.bc[o][p / (2 * NN)][0]) + p % (2 * NN);
              f32x2 f = from[0];
#pragma unroll
              for (int m = 1; m < 8; ++m) f = add2(f, from[m * 2 * NN]);
              s_bc[warp][rr][p] = f;
            }
            __syncwarp();
          }
        }
        __syncthreads();
        if (threadIdx.x < kTileRows * kStates) {
          const int r = threadIdx.x / kStates, v = threadIdx.x % kStates;
          if (r < rows) {
            const f32x2 f = add2(add2(s_bc[0][r][v], s_bc[1][r][v]), add2(s_bc[2][r][v], s_bc[3][r][v]));
            const int64_t row = ((int64_t)quad * l.tokens + row0 + i * kTileRows + r) * a.groups + group;
            *reinterpret_cast<f32x2*>(&g.bc[(row * 2 + v / (2 * NN)) * l.pad + n0 + v % (2 * NN) * 2]) = f;
          }
        }
        __syncthreads();
      }
    }
    if (placed) {
      float* to = g.part_a + (int64_t)run * l.wide * l.pad + mine + n0;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float f[2][NN];
#pragma unroll
        for (int n = 0; n < NN; ++n) {
          const float2 v = halves(da[j][n]);
          f[0][n] = v.x, f[1][n] = v.y;
        }
        write_numbers<NN>(to + 2 * j * l.pad, f[0]);
        write_numbers<NN>(to + (2 * j + 1) * l.pad, f[1]);
      }
    }
  }
  wait_for_copies<0>();
  sum_d = add2(sum_d, __shfl_xor_sync(0xffffffffu, sum_d, 16));
  sum_bias = add2(sum_bias, __shfl_xor_sync(0xffffffffu, sum_bias, 16));
  if (o == 0 && placed) {
    float* to = g.part_d + (int64_t)run * 2 * l.wide + t.place + 2 * p;
    *reinterpret_cast<f32x2*>(to) = sum_d;
    *reinterpret_cast<f32x2*>(to + l.wide) = sum_bias;
  }
}

// db and dc = the quads' parts summed, and da, dd, ddt_bias the runs', in fixed orders.
template <class T>
__global__ void __launch_bounds__(512) k_scan_sums(ScanBackwardLaunch g) {
  __shared__ float s[16][33];
  const ScanLaunch& l = g.f;
  const tb_scan_args& a = l.a;
  const int64_t elements = l.tokens * a.groups * 2 * a.states, rows_blocks = (elements + 511) / 512;
  wait_for_last_kernel();
  if (blockIdx.x < rows_blocks) {
    const int64_t i = (int64_t)blockIdx.x * 512 + threadIdx.x;
    if (i >= elements) return;
    const int n = (int)(i % a.states), which = (int)(i / a.states % 2);
    const int64_t rg = i / (2 * a.states), row = rg / a.groups;
    const LinCover cover = lin_cover(l);
    float sum = 0.f;
    if (row >= cover.begin && row < cover.end)
      for (int q = 0; q < g.quads; ++q) sum += g.bc[(((int64_t)q * l.tokens * a.groups + rg) * 2 + which) * l.pad + n];
    ((T*)(which ? g.g.dc : g.g.db))[rg * a.states + n] = RowType<T>::from(sum);
    return;
  }
  const int64_t per_a = (int64_t)l.wide * l.pad, width = per_a + 2 * (int64_t)l.wide;
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t o = (blockIdx.x - rows_blocks) * 32 + x;
  float sum = 0.f;
  if (o < width) {
    const float* part = o < per_a ? g.part_a + o : g.part_d + (o - per_a);
    const int64_t stride = o < per_a ? per_a : 2 * (int64_t)l.wide;
    for (int r = y; r < g.runs; r += 16) sum += part[r * stride];
  }
  s[y][x] = sum;
  __syncthreads();
  if (y || o >= width) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) sum += s[i][x];
  const int64_t place = o < per_a ? o / l.pad : (o - per_a) % l.wide;
  const int per = a.channels / a.groups, in = (int)(place % l.group_pad);
  if (in >= per) return;
  const int64_t c = place / l.group_pad * per + in;
  if (o < per_a) {
    const int n = (int)(o % l.pad);
    if (n < a.states) g.g.da[c * a.states + n] = sum;
  } else if (o - per_a < l.wide) {
    if (g.g.dd) g.g.dd[c] = sum;
  } else if (g.g.ddt_bias) {
    g.g.ddt_bias[c] = sum;
  }
}

template <class T, int NN>
cudaError_t go_carry(const ScanBackwardLaunch& g, cudaStream_t s) {
  static std::atomic<bool> ready[kMaxDevices];
  const int bytes = kWarps * sizeof(CarryShared<T, NN>);
  const cudaError_t e = allow_shared(k_scan_carry<T, NN>, bytes, ready);
  if (e != cudaSuccess) return e;
  const int64_t blocks_x = ((int64_t)g.f.a.groups * g.f.group_tiles + kWarps - 1) / kWarps;
  const dim3 grid((unsigned)(g.f.segments * blocks_x), g.f.pad / (2 * NN));
  return launch_early(k_scan_carry<T, NN>, grid, 32 * kWarps, bytes, s, true, g);
}
template <class T, int NN, bool kMany>
cudaError_t go_back(const ScanBackwardLaunch& g, cudaStream_t s) {
  static std::atomic<bool> ready[kMaxDevices];
  const int bytes = kWarps * (sizeof(BackShared<T, NN>) + kTileRows * 8 * NN * sizeof(float));
  const cudaError_t e = allow_shared(k_scan_backward<T, NN, kMany>, bytes, ready);
  if (e != cudaSuccess) return e;
  return launch_early(k_scan_backward<T, NN, kMany>, (unsigned)((int64_t)g.runs * g.f.a.groups * g.quads), 32 * kWarps, bytes, s,
                      true, g);
}
template <class T>
cudaError_t back(const ScanBackwardLaunch& g, cudaStream_t s) {
  if (g.f.pass == 8) return go_back<T, 2, false>(g, s);
  return g.f.pad == 16 ? go_back<T, 4, false>(g, s) : go_back<T, 4, true>(g, s);
}
template <class T>
cudaError_t carry(const ScanBackwardLaunch& g, cudaStream_t s) {
  return g.f.pass == 8 ? go_carry<T, 4>(g, s) : go_carry<T, 8>(g, s);
}

}  // namespace

cudaError_t launch_scan_carry(const void* args, cudaStream_t s) {
  const ScanBackwardLaunch& g = *(const ScanBackwardLaunch*)args;
  switch (g.f.a.type) {
    case TB_TYPE_F32: return carry<float>(g, s);
    case TB_TYPE_F16: return carry<__half>(g, s);
    default: return carry<__nv_bfloat16>(g, s);
  }
}
cudaError_t launch_scan_backward(const void* args, cudaStream_t s) {
  const ScanBackwardLaunch& g = *(const ScanBackwardLaunch*)args;
  switch (g.f.a.type) {
    case TB_TYPE_F32: return back<float>(g, s);
    case TB_TYPE_F16: return back<__half>(g, s);
    default: return back<__nv_bfloat16>(g, s);
  }
}
cudaError_t launch_scan_sums(const void* args, cudaStream_t s) {
  const ScanBackwardLaunch& g = *(const ScanBackwardLaunch*)args;
  const tb_scan_args& a = g.f.a;
  const int64_t rows = (g.f.tokens * a.groups * 2 * a.states + 511) / 512;
  const int64_t columns = ((int64_t)g.f.wide * (g.f.pad + 2) + 31) / 32;
  auto go = [&](auto kernel) { return launch_early(kernel, (unsigned)(rows + columns), 512, 0, s, g.runs > 0, g); };
  switch (a.type) {
    case TB_TYPE_F32: return go(k_scan_sums<float>);
    case TB_TYPE_F16: return go(k_scan_sums<__half>);
    default: return go(k_scan_sums<__nv_bfloat16>);
  }
}

}  // namespace tb
