// Linear attention with a decay for each head on the tensor cores for rows in
// 32 or 16 bits of any type, stride and head size up to 128: the chunks of
// tb_linattn_chunk.cu with every operand split into kTerms bfloat16 terms.
//
// A float is the sum of three bfloat16 terms (24 bits), a half of two (11
// bits).  Three terms: the six products of terms whose ranks add up to two or
// less leave 2^-24 of a product out, so sums keep 32-bit accuracy; two terms:
// three products, 2^-16, for 16-bit outputs.  Scores, W = decayed values and
// the state are split the same way as they become operands.  Six products in
// place of one still are a third of what the recurrence costs in packed
// 32-bit multiply-adds (64 rows of 128 keys and values: 7200 clocks of the
// tensor cores, 24600 of the FP32 pipes).
//
// A block walks one segment of one head.  Three warps read rows, split them
// and lay them out as tiles; one thread issues the products; 8 warps hold the
// state and make W, straight from memory (a lane is a value); 4 warps take the
// scores (lanes 64 to 127) and then the output, which lies in the columns that
// the scores leave.
//
// A chunk takes 3 to 4 us, which the row warps bound: their loads, conversions
// and stores of the terms (the tensor pipe is busy 30% of the time).  Measured:
// 32 grids of 512 rows and 8 heads of 64 in fp32 87 us; 10 of 5000 rows 361 us.
#include "tb_linattn_tc.cuh"

namespace tb {
namespace {

constexpr int kThreads = 512;
// 8 warps of the state and W, 3 of the rows, the products, 4 of the scores and the output
constexpr int kWarpLoad = 8, kLoadWarps = 3, kWarpMma = 11;

__device__ unsigned int g_gave_up;

enum Bars {
  kFull = 0, kEmpty = kFull + 2, kSReady = kEmpty + 2, kSFull, kWFull, kWFree, kKvReady, kKvFree, kStFull, kStFree,
  kOReady, kOFree, kDrain, kBars
};

struct Shared {
  uint64_t bar[kBars];
  uint32_t tmem;
  volatile uint32_t gave_up;
  volatile uint32_t bad[2];  // chunk + 1 whose values are not all finite, by the chunk's parity
  LinSegment seg;
  float w[2 * kC];           // fold decay^(31-m), reverse: fold decay^(m-32); 0 past the 64th
  float o[2 * kC];           // mul decay^(m-31), reverse: mul decay^(32-m)
};

// Elements of E: floats, or 16 bits that are halves or bfloat16 numbers by
// `half` (the loads are the same, and what differs is outside their loops).
template <class E>
__device__ __forceinline__ float value(E x, bool half) {
  if constexpr (sizeof(E) == 4) return x;
  else return half ? __half2float(__ushort_as_half(x)) : __uint_as_float((uint32_t)x << 16);
}
template <class E>
__device__ __forceinline__ float load1(const void* x, int64_t at, bool half) {
  return value<E>(((const E*)x)[at], half);
}
template <class E>
__device__ __forceinline__ void store1(void* x, int64_t at, bool half, float f) {
  if constexpr (sizeof(E) == 4) ((E*)x)[at] = f;
  else ((E*)x)[at] = half ? __half_as_ushort(__float2half_rn(f)) : (E)(bf16x2(f, f) & 0xffffu);
}
// Eight elements: one 16-byte vector or two.
template <class E>
struct Eight {
  uint4 w[sizeof(E) / 2];
};
template <class E>
__device__ __forceinline__ void load8(Eight<E>& r, const E* x, bool vec, int left) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(E) / 2; ++i) r.w[i] = __ldg(reinterpret_cast<const uint4*>(x) + i);
  } else {
    auto bits = [&](int i) -> uint32_t {
      if (i >= left) return 0u;
      if constexpr (sizeof(E) == 4) return __float_as_uint(x[i]);
      else return x[i];
    };
    auto word = [&](int i) { return sizeof(E) == 4 ? bits(i) : bits(2 * i) | bits(2 * i + 1) << 16; };
#pragma unroll
    for (int i = 0; i < (int)sizeof(E) / 2; ++i)
      r.w[i] = make_uint4(word(4 * i), word(4 * i + 1), word(4 * i + 2), word(4 * i + 3));
  }
}
template <class E>
__device__ __forceinline__ void values8(const Eight<E>& r, bool half, f32x2 (&f)[4]) {
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      f[2 * i] = pair(__uint_as_float(r.w[i].x), __uint_as_float(r.w[i].y));
      f[2 * i + 1] = pair(__uint_as_float(r.w[i].z), __uint_as_float(r.w[i].w));
    }
  } else {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = half ? halves_of(w[i], __half()) : halves_of(w[i], __nv_bfloat16());
      f[i] = pair(y.x, y.y);
    }
  }
}

// The next term of a pair of floats, taken off them.
__device__ __forceinline__ uint32_t take_term(f32x2& e) {
  const uint32_t x = bf16x2(halves(e).x, halves(e).y);
  e = fma2(pair(low(x), high(x)), pair(-1.f, -1.f), e);
  return x;
}

__device__ __forceinline__ void tmem_st8(uint32_t t, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(t), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Rows j whose value is not finite, which W has zeros for: their scores times
// the value join the rows i that see them, in the output as this thread wrote it.
template <class E>
__device__ __noinline__ void add_not_finite_split(const LinProblem& p, bool is_half, int64_t row0, int h, int v, int n,
                                                  uint32_t scores, int terms) {
  const float sign = sign_of(p.mul) * sign_of(p.fold);
#pragma unroll 1
  for (int j = 0; j < n; ++j) {
    const float c = load1<E>(p.c, (row0 + j) * p.c_row + h * p.c_head + v, is_half);
    if (!not_finite(c)) continue;
#pragma unroll 1
    for (int i = p.reverse ? 0 : j; i <= (p.reverse ? j : n - 1); ++i) {
      float s = 0.f;
      for (int t = 0; t < terms; ++t) s += shared_bf16(tile_at(scores + t * kTile, i, j));
      const int64_t at = (row0 + i) * p.o_row + h * p.o_head + v;
      store1<E>(p.out, at, is_half, fmaf(s * sign, c, load1<E>(p.out, at, is_half)));
    }
  }
}
// And b_j c_j the state's update.
template <class E>
__device__ __noinline__ void add_not_finite_state_split(const LinProblem& p, bool is_half, int64_t row0, int h, int v, int n,
                                                        uint32_t columns, int key, int keys) {
  const float sign = sign_of(p.fold);
#pragma unroll 1
  for (int k0 = 0; k0 < keys; k0 += 16) {
    uint32_t y[16];
    tmem_ld16(columns + k0, y);
    tmem_wait_ld();
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      const float c = v < p.V ? load1<E>(p.c, (row0 + j) * p.c_row + h * p.c_head + v, is_half) : 0.f;
      if (!not_finite(c)) continue;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int k = key + k0 + i;
        if (k < p.K)
          y[i] = __float_as_uint(
              fmaf(load1<E>(p.b, (row0 + j) * p.b_row + h * p.b_head + k, is_half) * sign, c, __uint_as_float(y[i])));
      }
    }
    __syncwarp();
    tmem_st16(columns + k0, y);
  }
  tmem_wait_st();
}

template <class T>
__device__ __noinline__ void walk_rows(const LinLaunch& l, const LinProblem& p, const LinSegment& seg, int h,
                                       float* s_rows) {
  scan_walk<T, 32>(l, p, seg, h, s_rows, 256);
}

// kStates: the states of segments alone, without outputs.
template <class E, int kTerms, bool kStates>
__global__ void __launch_bounds__(kThreads, 1) k_split(const __grid_constant__ LinLaunch l) {
  constexpr uint32_t kColS = 0, kColKv = 64, kColW = 192, kColZ = kColW + 32 * kTerms;
  static_assert(kColZ + 64 * kTerms <= 512, "tensor memory");
  constexpr int kStageBytes = 2 * kTerms * 2 * kTile;  // A, B: terms of two 64-key blocks
  constexpr int kProducts = kTerms == 3 ? 6 : 3;

  if (kStates) let_next_kernel_start();
  extern __shared__ char s_raw[];
  __shared__ Shared s;
  // score tiles of each term, then the stages (the product A B^T reads the 8 KB before A too)
  const uint32_t tiles = (smem_addr(s_raw) + 1023) & ~1023u;
  const uint32_t stage0 = tiles + kTerms * kTile;

  const int slot0 = blockIdx.x / (l.heads * l.n), walk = blockIdx.x % (l.heads * l.n);
  const LinProblem& p = l.p[walk / l.heads];
  const int h = walk % l.heads;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  auto bar = [&](int i) { return smem_addr(&s.bar[i]); };
  const bool reverse = p.reverse;
  const float decay = l.decay[h];
  const bool steep = !(decay >= kSteep && decay <= 1.f / kSteep);
  const bool is_half = l.type == TB_TYPE_F16;

  if (warp == 0) {
    const LinSegment seg = lin_segment(l, l.sorted ? lin_grid_of_rank(l, slot0) : slot0);
    if (lane == 0) s.seg = seg;
  } else if (warp == 1) {
    if (lane == 0) {
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(kFull + i), kLoadWarps);
        mbar_init(bar(kEmpty + i), 1);
      }
      mbar_init(bar(kSReady), 1);
      mbar_init(bar(kSFull), 2);
      mbar_init(bar(kWFull), 8);
      mbar_init(bar(kWFree), 1);
      mbar_init(bar(kKvReady), 1);
      mbar_init(bar(kKvFree), 8);
      mbar_init(bar(kStFull), 8);
      mbar_init(bar(kStFree), 1);
      mbar_init(bar(kOReady), 1);
      mbar_init(bar(kOFree), 4);
      mbar_init(bar(kDrain), 1);
      s.gave_up = 0;
      s.bad[0] = s.bad[1] = 0;
      fence_mbar_init();
    }
  } else if (warp == kWarpMma) {
    tmem_alloc(smem_addr(&s.tmem), 512);
  } else if (warp >= 4 && warp < 8 && !steep) {
    const int m = threadIdx.x - 128;
    const float log = log2f(decay), x = reverse ? (float)(m - 32) : (float)(31 - m);
    s.w[m] = m < kC ? p.fold * exp2f(x * log) : 0.f;
    s.o[m] = m < kC ? p.mul * exp2f(-x * log) : 0.f;
  } else if (!kStates && warp > kWarpMma) {
    constexpr int first = (kWarpMma + 1) * 32;
    lin_zero_share<typename LinBits<sizeof(E)>::type>(l, p, slot0, h, 1, threadIdx.x - first, kThreads - first);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const LinSegment seg = s.seg;
  const uint32_t tmem = s.tmem;
  // a slot without a segment, or a segment whose state nobody reads
  const bool idle = seg.grid < 0 || (kStates && seg.index + 1 == seg.count && !p.last);
  const int chunks = idle || steep ? 0 : (seg.len + kC - 1) / kC;
  auto rows_of = [&](int t) { return min(kC, seg.len - t * kC); };
  auto row_of = [&](int t) {
    return reverse ? seg.end - seg.first - (int64_t)t * kC - rows_of(t) : seg.begin + seg.first + (int64_t)t * kC;
  };
  auto wait = [&](int i, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait(bar(i), parity & 1, &s.gave_up));
  };
  auto arrive = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(i));
  };
  const int keys = p.K > 64 ? 128 : 64;  // of the tiles
  const int quarter = warp & 3, v = quarter * 32 + lane;
  const bool live = quarter * 32 < p.V;  // warp-uniform
  const uint32_t lanes = tmem + ((uint32_t)quarter << 21);
  // the tiles of a stage: term x of A, of B
  auto tile_a = [&](uint32_t at, int x) { return at + x * 2 * kTile; };
  auto tile_b = [&](uint32_t at, int x) { return at + (kTerms + x) * 2 * kTile; };

  if (warp >= kWarpLoad && warp < kWarpLoad + kLoadWarps) {
    // ---------------------------------------------------------------- rows
    // A thread takes the same 8 elements of every kRowStep-th row of B, then of A; a batch of rows is loaded while
    // the one before it is split.
    const int shift = keys > 64 ? 4 : 3, me = threadIdx.x - kWarpLoad * 32;
    const int k = (me & ((1 << shift) - 1)) * 8, r0 = me >> shift, step = kLoadWarps * 32 >> shift;
    const int sweeps = (kC + step - 1) / step, total = (kStates ? 1 : 2) * sweeps;
    const uint32_t to0 = (k >> 6) * kTile + r0 * 128;
    constexpr int kBatch = 4;
    Eight<E> next[kBatch];
    auto load = [&](int t, int q0) {
      const int n = rows_of(t);
      const int64_t row0 = row_of(t);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int q = q0 + b;
        const bool is_b = q < sweeps;
        const int r = r0 + (is_b ? q : q - sweeps) * step;
#pragma unroll
        for (int i = 0; i < (int)sizeof(E) / 2; ++i) next[b].w[i] = make_uint4(0u, 0u, 0u, 0u);
        if (q < total && r < n && k < p.K)
          load8<E>(next[b],
                   (const E*)(is_b ? p.b : p.a) + (row0 + r) * (is_b ? p.b_row : p.a_row) +
                       h * (is_b ? p.b_head : p.a_head) + k,
                   p.vec & (is_b ? 2 : 1), p.K - k);
      }
    };
    if (chunks) load(0, 0);
#pragma unroll 1
    for (int t = 0; t < chunks; ++t) {
      if (t >= 2 && !wait(kEmpty + (t & 1), t / 2 - 1)) break;
      const uint32_t at = stage0 + (t & 1) * kStageBytes;
#pragma unroll 1
      for (int q0 = 0; q0 < total; q0 += kBatch) {
        Eight<E> now[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) now[b] = next[b];
        if (q0 + kBatch < total) load(t, q0 + kBatch);
        else if (t + 1 < chunks) load(t + 1, 0);
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int q = q0 + b;
          const bool is_b = q < sweeps;
          const int move = (is_b ? q : q - sweeps) * step, r = r0 + move;
          if (q >= total || r >= kC) continue;
          const uint32_t to = (is_b ? tile_b(at, 0) : tile_a(at, 0)) + to0 + move * 128 + ((((k >> 3) & 7) ^ (r & 7)) << 4);
          f32x2 e[4];
          values8<E>(now[b], is_half, e);
#pragma unroll
          for (int x = 0; x < kTerms; ++x) {
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = take_term(e[j]);
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + x * 2 * kTile), "r"(y[0]), "r"(y[1]),
                         "r"(y[2]), "r"(y[3])
                         : "memory");
          }
        }
      }
      fence_async_smem();
      arrive(kFull + (t & 1));
    }
  } else if (warp == kWarpMma) {
    if (chunks && elect_one()) {
      const uint32_t kv_desc = mma_desc(128, 64, true) + (keys > 64 ? (uint32_t)(64 / 8) << 17 : 0u);
      constexpr uint32_t kRowDesc = mma_desc(128, kC, false);
      auto one = [&](int i, uint32_t parity) { return mbar_wait(bar(i), parity & 1, &s.gave_up); };
      // the products of terms x and y of the left and the right operand, the largest last: a sum is then rounded at
      // its full size only as often as it has steps of 16
      constexpr int kLeft[6] = {kTerms == 3 ? 2 : 1, 0, kTerms == 3 ? 1 : 0, 1, 0, 0};
      constexpr int kRight[6] = {0, kTerms == 3 ? 2 : 1, kTerms == 3 ? 1 : 0, 0, 1, 0};
      constexpr uint32_t kTermStep = 2 * kTile >> 4;  // of a descriptor, from a term's tiles to the next term's
      const int steps = keys / 16;
      bool ok = true;
#pragma unroll 1
      for (int t = 0; ok && t < chunks; ++t) {
        const uint32_t at = stage0 + (t & 1) * kStageBytes;
        ok = one(kFull + (t & 1), t >> 1);
        if (!kStates) {
          // A B^T, rows i in lanes 64 to 127
          ok = ok && (t == 0 || one(kOFree, t - 1));
          if (!ok) break;
          tc_fence_after();
          const uint64_t left = smem_desc(tile_a(at, 0) - kTile, 16), right = smem_desc(tile_b(at, 0), 16);
#pragma unroll
          for (int i = 0; i < kProducts; ++i)
#pragma unroll 1
            for (int k = 0; k < steps; k += 4) {
              const uint32_t off = (k >> 2) * kTile >> 4;
#pragma unroll
              for (int q = 0; q < 4; ++q)
                mma_ss(tmem + kColS, left + off + kLeft[i] * kTermStep + 2 * q, right + off + kRight[i] * kTermStep + 2 * q,
                       kRowDesc, i > 0 || k > 0 || q > 0);
            }
          mma_commit(bar(kSReady));
        }
        // W^T B
        ok = ok && one(kWFull, t) && (t == 0 || one(kKvFree, t - 1));
        if (!ok) break;
        tc_fence_after();
        {
          const uint64_t right = smem_desc(tile_b(at, 0), kTile);
#pragma unroll
          for (int i = 0; i < kProducts; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_ts(tmem + kColKv, tmem + kColW + kLeft[i] * 32 + j * 8, right + kRight[i] * kTermStep + j * (2048 >> 4),
                     kv_desc, i > 0 || j > 0);
        }
        mma_commit(bar(kKvReady));
        if (!kStates) {
          // Z^T A^T, where the scores were
          ok = one(kStFull, t) && one(kSFull, t);
          if (!ok) break;
          tc_fence_after();
          const uint64_t rows = smem_desc(tile_a(at, 0), 16), weights = smem_desc(tiles, 16);
#pragma unroll
          for (int i = 0; i < kProducts; ++i)
#pragma unroll 1
            for (int k = 0; k < steps; k += 4) {
              const uint32_t off = (k >> 2) * kTile >> 4;
#pragma unroll
              for (int q = 0; q < 4; ++q)
                mma_ts(tmem + kColS, tmem + kColZ + kLeft[i] * 64 + k * 8 + q * 8, rows + off + kRight[i] * kTermStep + 2 * q,
                       kRowDesc, i > 0 || k > 0 || q > 0);
            }
          mma_commit(bar(kStFree));
          // W^T scores^T
#pragma unroll
          for (int i = 0; i < kProducts; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
              mma_ts(tmem + kColS, tmem + kColW + kLeft[i] * 32 + j * 8, weights + (kRight[i] * kTile >> 4) + j * 2, kRowDesc,
                     true);
          mma_commit(bar(kOReady));
        }
        mma_commit(bar(kWFree));
        mma_commit(bar(kEmpty + (t & 1)));
      }
      if (!ok) {  // products in flight finish before tensor memory is given back
        uint32_t flag = 0;
        mma_commit(bar(kDrain));
        mbar_wait(bar(kDrain), 0, &flag);
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ state, W
    const int half = warp >> 2, own = keys / 2;  // keys of a thread
    const int64_t state_at = ((int64_t)seg.grid * l.heads + h) * p.K * p.V;
    float* seg_state = p.seg ? p.seg + ((int64_t)seg.slot * l.heads + h) * p.K * p.V : nullptr;
    const float log = log2f(decay);
    const float enter = chunks ? exp2f((reverse ? 31.f : 32.f) * log) : 1.f, full = exp2f(64.f * log);
    if (l.phase == 2) wait_for_last_kernel();  // the states that enter
    f32x2 u[32];  // Z, by pairs of keys
    {
      const float* from = l.phase == 2 ? seg_state : p.first ? p.first + state_at : nullptr;
      const int64_t step = l.phase == 2 ? p.V : p.first_k;
      const int left = kStates || idle || steep || !from || v >= p.V ? 0 : min(own, p.K - half * own);
      if (from) from += half * own * step + v * (l.phase == 2 ? 1 : p.first_v);
#pragma unroll
      for (int i = 0; i < 64; i += 2, from += 2 * step)
        u[i / 2] = pair(i < left ? from[0] * enter : 0.f, i + 1 < left ? from[step] * enter : 0.f);
    }
#pragma unroll 1
    for (int t = -1; t < chunks; ++t) {
      const int x = t + 1;
      const bool more = x < chunks;
      if (more && live) {
        // this chunk's values on their way to L2, a line of 32 for every row (registers that held them would spill)
        const int n = rows_of(x), r = half * 32 + lane;
        if (r < n)
          asm volatile("prefetch.global.L2 [%0];" ::"l"((const E*)p.c + (row_of(x) + r) * p.c_row + h * p.c_head +
                                                         quarter * 32));
      }
      if (t >= 0) {
        // the state after this chunk
        const int n = rows_of(t);
        if (!wait(kKvReady, t)) break;
        tc_fence_after();
        const float d = t + 1 < chunks ? full : exp2f((float)(n - (reverse ? 31 : 32)) * log);
        if (live) {
          const uint32_t columns = lanes + kColKv + half * own;
          if (s.bad[t & 1] == (uint32_t)t + 1)
            add_not_finite_state_split<E>(p, is_half, row_of(t), h, v, n, columns, half * own, own);
          const f32x2 d2 = pair(d, d);
#pragma unroll
          for (int k0 = 0; k0 < 64; k0 += 16) {
            if (k0 >= own) break;
            uint32_t z[16];
            tmem_ld16(columns + k0, z);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; i += 2)
              u[(k0 + i) / 2] = mul2(add2(u[(k0 + i) / 2], pair(__uint_as_float(z[i]), __uint_as_float(z[i + 1]))), d2);
          }
        }
        tc_fence_before();
        arrive(kKvFree);
      }
      if (!kStates && more) {
        // Z^T as the next chunk's operand
        if (x > 0 && !wait(kStFree, x - 1)) break;
        tc_fence_after();
        if (live) {
#pragma unroll
          for (int k0 = 0; k0 < 64; k0 += 16) {
            if (k0 >= own) break;
            f32x2 e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = u[k0 / 2 + i];
#pragma unroll
            for (int y = 0; y < kTerms; ++y) {
              uint32_t z[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) z[i] = take_term(e[i]);
              tmem_st8(lanes + kColZ + y * 64 + (half * own + k0) / 2, z);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        arrive(kStFull);
      }
      if (more) {
        // W^T, in its one buffer once the last chunk's products are done with it
        if (x > 0 && !wait(kWFree, x - 1)) break;
        tc_fence_after();
        if (live) {
          const int n = rows_of(x);
          const float* w = s.w + (reverse ? kC - n : 0) + half * 32;
          const E* from = (const E*)p.c + (row_of(x) + half * 32) * p.c_row + h * p.c_head + v;
#pragma unroll 1
          for (int r0 = 0; r0 < 32; r0 += 16) {
            E raw[16];
#pragma unroll
            for (int i = 0; i < 16; ++i, from += p.c_row)
              raw[i] = half * 32 + r0 + i < n && v < p.V ? __ldg(from) : E(0);
            float c[16], finite = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              c[i] = value<E>(raw[i], is_half);
              finite = fmaf(c[i], 0.f, finite);
            }
            if (finite != finite) {
              // 0 x infinity of a later row is no part of an earlier row's sum: the products take zeros, and the
              // warps of the output and of the state add these values to what sees them
#pragma unroll
              for (int i = 0; i < 16; ++i) c[i] = not_finite(c[i]) ? 0.f : c[i];
              s.bad[x & 1] = x + 1;
            }
            __syncwarp();
            f32x2 e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              e[i] = mul2(pair(c[2 * i], c[2 * i + 1]), pair(w[r0 + 2 * i], w[r0 + 2 * i + 1]));
#pragma unroll
            for (int y = 0; y < kTerms; ++y) {
              uint32_t z[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) z[i] = take_term(e[i]);
              tmem_st8(lanes + kColW + y * 32 + half * 16 + r0 / 2, z);
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        arrive(kWFull);
      }
    }
    float* dst = kStates ? seg_state : l.phase == 0 && p.last ? p.last + state_at : nullptr;
    if (!idle && !steep && dst && !s.gave_up && v < p.V) {
      dst += half * own * p.V + v;
      const int left = min(own, p.K - half * own);
#pragma unroll
      for (int i = 0; i < 64; i += 2, dst += 2 * p.V) {
        if (i < left) dst[0] = halves(u[i / 2]).x;
        if (i + 1 < left) dst[p.V] = halves(u[i / 2]).y;
      }
    }
  } else if (!kStates) {
    // ------------------------------------------------------ scores, output
#pragma unroll 1
    for (int t = 0; t < chunks; ++t) {
      const int n = rows_of(t);
      if (quarter >= 2) {
        const int i = (quarter - 2) * 32 + lane;
        if (!wait(kSReady, t)) break;
        tc_fence_after();
#pragma unroll 1
        for (int j0 = 0; j0 < kC; j0 += 16) {
          uint32_t x[16];
          tmem_ld16(lanes + kColS + j0, x);
          tmem_wait_ld();
          f32x2 e[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int k = j0 + 2 * j;
            e[j] = pair((reverse ? k >= i : k <= i) ? __uint_as_float(x[2 * j]) : 0.f,
                        (reverse ? k + 1 >= i : k + 1 <= i) ? __uint_as_float(x[2 * j + 1]) : 0.f);
          }
#pragma unroll
          for (int y = 0; y < kTerms; ++y) {
            uint32_t z[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) z[j] = take_term(e[j]);
#pragma unroll
            for (int q = 0; q < 2; ++q)
              asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                               tiles + y * kTile + i * 128 + (((j0 / 8 + q) ^ (i & 7)) << 4)),
                           "r"(z[4 * q]), "r"(z[4 * q + 1]), "r"(z[4 * q + 2]), "r"(z[4 * q + 3])
                           : "memory");
          }
        }
        fence_async_smem();
        tc_fence_before();
        arrive(kSFull);
      }
      if (!wait(kOReady, t)) break;
      tc_fence_after();
      if (live) {
        uint32_t x[4][16];
#pragma unroll
        for (int i = 0; i < 4; ++i) tmem_ld16(lanes + kColS + 16 * i, x[i]);
        tmem_wait_ld();
        const bool bad = s.bad[t & 1] == (uint32_t)t + 1;
        if (!bad) {
          tc_fence_before();
          arrive(kOFree);
        }
        const int64_t row0 = row_of(t);
        const float* w = s.o + (reverse ? kC - n : 0);
        if (v < p.V) {
          E* out = (E*)p.out + row0 * p.o_row + h * p.o_head + v;
          auto put = [&](int i) {
            store1<E>(out, 0, is_half, __uint_as_float(x[i / 16][i % 16]) * w[i]);
            out += p.o_row;
          };
          if (n == kC) {
#pragma unroll
            for (int i = 0; i < kC; ++i) put(i);
          } else {
#pragma unroll
            for (int i = 0; i < kC; ++i) {
              if (i >= n) break;
              put(i);
            }
          }
          if (bad) add_not_finite_split<E>(p, is_half, row0, h, v, n, tiles, kTerms);
        }
        __syncwarp();
        if (bad) {
          tc_fence_before();
          arrive(kOFree);
        }
      } else {
        tc_fence_before();
        arrive(kOFree);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && s.gave_up) atomicAdd(&g_gave_up, 1u);
  if (warp == kWarpMma) tmem_free(tmem, 512);
  if (!steep || idle || warp >= 8) return;
  if (l.phase == 2) wait_for_last_kernel();
  float* rows = reinterpret_cast<float*>(s_raw + (tiles - smem_addr(s_raw)));
  if constexpr (sizeof(E) == 4) walk_rows<float>(l, p, s.seg, h, rows);
  else if (is_half) walk_rows<__half>(l, p, s.seg, h, rows);
  else walk_rows<__nv_bfloat16>(l, p, s.seg, h, rows);
}

template <class E, int kTerms, bool kStates>
cudaError_t go(const LinLaunch& l, cudaStream_t s) {
  constexpr int bytes = 1024 + kTerms * kTile + 2 * 2 * kTerms * 2 * kTile;
  static_assert(bytes > 116 * 1024 && bytes < 222 * 1024, "one block a multiprocessor: tensor memory is not shared");
  static std::atomic<bool> ready[kMaxDevices];
  const cudaError_t e = allow_shared(k_split<E, kTerms, kStates>, bytes, ready);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (int64_t)l.segments * l.heads * l.n;
  return launch_early(k_split<E, kTerms, kStates>, (unsigned)blocks, kThreads, bytes, s, l.phase == 2, l);
}

__global__ void __launch_bounds__(32) k_wait_selftest(uint32_t polls) {
  __shared__ uint64_t bar;
  __shared__ volatile uint32_t gave_up;
  if (mbar_selftest(&bar, &gave_up, polls) && threadIdx.x == 0) atomicAdd(&g_gave_up, 1u);
}

}  // namespace

cudaError_t launch_linear_split(const void* args, cudaStream_t s) {
  const LinLaunch& l = *(const LinLaunch*)args;
  if (l.type == TB_TYPE_F32) return l.phase == 1 ? go<float, 3, true>(l, s) : go<float, 3, false>(l, s);
  bool exact = false;  // 32-bit states come out
  for (int i = 0; i < l.n; ++i) exact = exact || (l.p[i].last && l.phase != 2);
  if (l.phase == 1) return exact ? go<uint16_t, 3, true>(l, s) : go<uint16_t, 2, true>(l, s);
  return exact ? go<uint16_t, 3, false>(l, s) : go<uint16_t, 2, false>(l, s);
}

cudaError_t linear_split_selftest(const void* args, cudaStream_t s) {
  k_wait_selftest<<<1, 32, 0, s>>>(*(const uint32_t*)args);
  return cudaGetLastError();
}

cudaError_t linear_split_gave_up(cudaStream_t s, unsigned int* count) {
  void* at = nullptr;
  cudaError_t e = cudaGetSymbolAddress(&at, g_gave_up);
  if (e == cudaSuccess) e = cudaMemcpyAsync(count, at, sizeof *count, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  return e;
}

}  // namespace tb
