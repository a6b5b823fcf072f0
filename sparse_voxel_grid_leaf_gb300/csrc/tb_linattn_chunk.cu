// Linear attention with a decay for each head on the tensor cores: bfloat16
// rows, heads of up to 128 keys and values, in chunks of 64 rows.
//
// Over a chunk of rows i, j (in the order of the walk) with entering state X:
//   P_ij   = fold mul decay^(i-j) (a_i . b_j) for j <= i, else 0
//   out_i  = sum_j P_ij c_j + mul decay^(i+e) a_i X       e = 1 forward, 0 reverse
//   X'     = decay^n X + sum_j fold decay^(n-e-j) b_j c_j^T
// Four products a chunk, each with the values (or, for P, the rows i) along
// the 128 lanes of tensor memory:
//   A B^T                   both operands in shared memory      -> P
//   C^T P^T, X^T A^T        left operand in tensor memory       -> out^T
//   (decayed C)^T B         left operand in tensor memory       -> X'^T - decay^n X^T
// so that the state X^T stays in the registers of the threads of its lanes (a
// value each), is multiplied by decay^n there in 32 bits, and goes back to
// tensor memory as bfloat16 only as an operand.
//
// Roundings to 16 bits: P (as any attention's weights), X as an operand, and
// the output; the decayed values are split into two bfloat16 terms (16 bits
// of the product of a value and a power), or three (24 bits) where states are
// an output, so the 32-bit states keep 32-bit accuracy.
//
// A block walks one segment of one head: the copy engine fills a ring of row
// tiles, one thread issues the products, and warps take the steps between
// them -- state and decayed values (8 warps), P (2), output (4) -- each on
// its own chunk, through barriers in shared memory.
#include <cstring>

#include "tb_linattn.cuh"
#include "tb_seq.cuh"
#include "tb_tc.cuh"

namespace tb {
namespace {

constexpr int kC = 64;            // rows of a chunk
constexpr int kTile = 8192;       // 64 rows x 128 bytes
constexpr int kMaxStages = 4;
// Warps: 8 of the state, the copies, the products, 2 of P, 4 of the output.
// Sixteen leave 128 registers a thread, which hold the state of 128 keys
// without spills (eighteen left 96, and the spills cost more than a third).
constexpr int kWarpTma = 8, kWarpMma = 9, kWarpP = 10, kWarpOut = 12;
constexpr int threads_of(bool states) { return (states ? kWarpP : 16) * 32; }

constexpr int stages_of(int KP) { return KP == 64 ? 4 : 3; }

// Set when a wait gave up (a bug, or a GPU that stands still): read and
// cleared by launch_linear_status.
__device__ unsigned int g_gave_up;

enum Bars {
  kFull = 0, kEmpty = kFull + kMaxStages, kPReady = kEmpty + kMaxStages, kPFull = kPReady + 2, kWFull = kPFull + 2, kCFull,
  kCFree = kCFull + 2, kKvReady = kCFree + 2, kKvFree, kStFull, kStFree, kOReady, kOFree, kZeros, kDrain, kBars
};

struct Shared {
  uint64_t bar[kBars];
  uint32_t tmem;
  volatile uint32_t gave_up;
  volatile uint32_t bad[kMaxStages];  // chunk + 1 whose values are not all finite
  LinSegment seg;
  float pow[kC + 1];               // decay^n
  float fold[2 * kC + 1];          // fold mul decay^(n - 64), 0 for n < 64
  __align__(16) float up[kC];      // decay^(m+1), times fold (reverse) or mul (forward)
  __align__(16) float down[4][2 * kC];  // decay^(63-m), 0 past m = 63: copy s starts at m = s
};

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float low(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float high(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

__device__ __forceinline__ float shared_bf16(uint32_t at) {
  uint16_t bits;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(bits) : "r"(at));
  return __uint_as_float((uint32_t)bits << 16);
}
__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7f800000u) == 0x7f800000u; }

// Adds P_ij c_j of the rows j whose value is not finite to the rows i that see
// them, in a warp's staged output (the product had zeros in their place).
__device__ __noinline__ void add_not_finite(uint32_t stage, uint32_t p_tile, uint32_t c_tile, int n, bool reverse) {
  const int lane = threadIdx.x & 31;
  const uint32_t col = (lane & 7) * 2;
  const int warp_chunk = ((threadIdx.x >> 5) & 1) * 4 + (lane >> 3);  // the lane's 8 values within 64
  for (int j = 0; j < n; ++j) {
    const float c = shared_bf16(c_tile + j * 128 + ((warp_chunk ^ (j & 7)) << 4) + col);
    if (!not_finite(c)) continue;
    for (int i = reverse ? 0 : j; i <= (reverse ? j : n - 1); ++i) {
      const uint32_t at = stage + i * 64 + (((lane >> 3) ^ ((i >> 1) & 3)) << 4) + col;
      const float pij = shared_bf16(p_tile + i * 128 + (((j >> 3) ^ (i & 7)) << 4) + (j & 7) * 2);
      const float o = fmaf(pij, c, shared_bf16(at));
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(at), "h"((uint16_t)(bf16x2(o, o) & 0xffffu)) : "memory");
    }
  }
}

// KP: keys of a tile, 64 or 128 (fewer are padded with zeros by the copies).
// kStates: the states of segments alone, without outputs.
template <int KP, int kTerms, bool kStates>
__global__ void __launch_bounds__(threads_of(kStates), 1) k_chunks(const __grid_constant__ ChunkLaunch g) {
  constexpr int kCt = KP == 128 && kTerms == 3 ? 1 : 2;  // buffers of C^T in tensor memory
  constexpr uint32_t kColP = 0, kColOi = 128, kColKv = 192, kColCt = kColKv + KP, kColW = kColCt + 32 * kCt,
                     kColSt = kColW + 32 * kTerms;
  static_assert(kColSt + KP / 2 <= 512, "tensor memory");
  constexpr int kBlocks = KP / 64, kStages = stages_of(KP);
  constexpr int kStageBytes = (2 * kBlocks + 2) * kTile;  // A, B, C

  extern __shared__ char s_raw[];
  __shared__ Shared s;
  // two P tiles, then the stages (the product A B^T reads the 8 KB before A too)
  const uint32_t tiles = (smem_addr(s_raw) + 1023) & ~1023u;
  const uint32_t stage0 = tiles + 2 * kTile;

  const LinLaunch& l = g.l;
  const LinProblem& p = l.p[blockIdx.z];
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int h = blockIdx.y;
  auto bar = [&](int i) { return smem_addr(&s.bar[i]); };
  const bool reverse = p.reverse;

  if (warp == 0) {
    const LinSegment seg = lin_segment(l, blockIdx.x);
    if (lane == 0) s.seg = seg;
  } else if (warp == 1) {
    if (lane == 0) {
      for (int i = 0; i < kStages; ++i) {
        mbar_init(bar(kFull + i), 1);
        mbar_init(bar(kEmpty + i), kStates ? 9 : 13);  // products, state warps, output warps
        s.bad[i] = 0;
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(bar(kPReady + i), 1);
        mbar_init(bar(kPFull + i), 2);
        mbar_init(bar(kCFree + i), 1);
        mbar_init(bar(kCFull + i), 8);
      }
      mbar_init(bar(kWFull), 8);
      mbar_init(bar(kKvReady), 1);
      mbar_init(bar(kKvFree), 8);
      mbar_init(bar(kStFull), 8);
      mbar_init(bar(kStFree), 1);
      mbar_init(bar(kOReady), 1);
      mbar_init(bar(kOFree), 4);
      mbar_init(bar(kZeros), 8);
      mbar_init(bar(kDrain), 1);
      s.gave_up = 0;
      fence_mbar_init();
    }
  } else if (warp == kWarpMma) {
    tmem_alloc(smem_addr(&s.tmem), 512);
  } else if (warp >= 4 && warp < 8) {
    const int i = threadIdx.x - 128;
    const float d = l.decay[h];
    if (i <= kC) {
      const float x = lin_power(d, (float)i);
      s.pow[i] = x;
      s.fold[kC + i] = p.fold * p.mul * x;
      if (i) s.up[i - 1] = x * (reverse ? p.fold : p.mul);
    }
    if (i < kC) s.fold[i] = 0.f;
    for (int c = 0; c < 4; ++c) s.down[c][i] = i + c < kC ? lin_power(d, (float)(kC - 1 - i - c)) : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const LinSegment seg = s.seg;
  const uint32_t tmem = s.tmem;
  // a slot without a segment, or a segment whose state nobody reads
  const bool idle = seg.grid < 0 || (kStates && seg.index + 1 == seg.count && !p.last);
  const int chunks = idle ? 0 : (seg.len + kC - 1) / kC;
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
  const int value_blocks = p.V > 64 ? 2 : 1;

  if (warp == kWarpTma) {
    if (elect_one()) {
      const CUtensorMap* ma = &g.map[g.a[blockIdx.z]];
      const CUtensorMap* mb = &g.map[g.b[blockIdx.z]];
      const CUtensorMap* mc = &g.map[g.c[blockIdx.z]];
      tma_prefetch(ma);
      tma_prefetch(mb);
      tma_prefetch(mc);
      const uint32_t bytes = ((kStates ? 1 : 2) * kBlocks + value_blocks) * kTile;
      int t = 0;
      for (; t < chunks; ++t) {
        const int st = t % kStages;
        if (t >= kStages && !mbar_wait(bar(kEmpty + st), (t / kStages - 1) & 1, &s.gave_up)) break;
        const uint32_t at = stage0 + st * kStageBytes;
        const int row = (int)row_of(t);
        mbar_expect(bar(kFull + st), bytes);
        for (int i = 0; i < kBlocks; ++i) tma_load_3d(at + (kBlocks + i) * kTile, mb, 64 * i, h, row, bar(kFull + st));
        for (int i = 0; i < value_blocks; ++i)
          tma_load_3d(at + (2 * kBlocks + i) * kTile, mc, 64 * i, h, row, bar(kFull + st));
        if (!kStates)
          for (int i = 0; i < kBlocks; ++i) tma_load_3d(at + i * kTile, ma, 64 * i, h, row, bar(kFull + st));
      }
      if (s.gave_up) {  // copies in flight land before the block ends
        for (int i = t > kStages ? t - kStages : 0; i < t; ++i) {
          uint32_t flag = 0;
          mbar_wait(bar(kFull + i % kStages), (i / kStages) & 1, &flag);
        }
      }
    }
  } else if (warp == kWarpMma) {
    if (chunks && elect_one()) {
      constexpr uint32_t kPDesc = mma_desc(128, kC, false);
      constexpr uint32_t kKvDesc = mma_desc(128, KP, true);
      auto scores = [&](int t) {  // A B^T, rows i in lanes 64 to 127
        const uint32_t at = stage0 + t % kStages * kStageBytes;
#pragma unroll
        for (int k = 0; k < KP / 16; ++k) {
          const uint32_t off = (k >> 2) * kTile + (k & 3) * 32;
          mma_ss(tmem + kColP + (t & 1) * 64, smem_desc(at - kTile + off, 16),
                 smem_desc(at + kBlocks * kTile + off, 16), kPDesc, k > 0);
        }
        mma_commit(bar(kPReady + (t & 1)));
      };
      auto one = [&](int i, uint32_t parity) {
        const bool ok = mbar_wait(bar(i), parity & 1, &s.gave_up);
        tc_fence_after();
        return ok;
      };
      bool ok = one(kFull, 0);
      if (ok && !kStates) scores(0);
      for (int t = 0; ok && t < chunks; ++t) {
        const uint32_t at = stage0 + t % kStages * kStageBytes;
        if (!kStates && t + 1 < chunks) {
          ok = one(kFull + (t + 1) % kStages, (t + 1) / kStages) && (t == 0 || one(kOFree, t - 1));
          if (!ok) break;
          scores(t + 1);
        }
        // (decayed C)^T B
        ok = one(kFull + t % kStages, t / kStages) && one(kWFull, t) && (t == 0 || one(kKvFree, t - 1));
        if (!ok) break;
#pragma unroll
        for (int term = 0; term < kTerms; ++term)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_ts(tmem + kColKv, tmem + kColW + term * 32 + j * 8, smem_desc(at + kBlocks * kTile + j * 2048, kTile),
                   kKvDesc, term > 0 || j > 0);
        mma_commit(bar(kKvReady));
        if (!kStates) {
          // X^T A^T
          ok = one(kStFull, t) && (t == 0 || one(kOFree, t - 1));
          if (!ok) break;
#pragma unroll
          for (int k = 0; k < KP / 16; ++k)
            mma_ts(tmem + kColOi, tmem + kColSt + k * 8, smem_desc(at + (k >> 2) * kTile + (k & 3) * 32, 16), kPDesc,
                   k > 0);
          mma_commit(bar(kStFree));
          // C^T P^T
          ok = one(kCFull + t % kCt, t / kCt) && one(kPFull + (t & 1), t >> 1);
          if (!ok) break;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            mma_ts(tmem + kColP + (t & 1) * 64, tmem + kColCt + t % kCt * 32 + j * 8,
                   smem_desc(tiles + (t & 1) * kTile + j * 32, 16), kPDesc, j > 0);
          mma_commit(bar(kOReady));
          mma_commit(bar(kCFree + t % kCt));
        }
        mma_commit(bar(kEmpty + t % kStages));
      }
      if (!ok) {  // products in flight finish before tensor memory is given back
        uint32_t flag = 0;
        mma_commit(bar(kDrain));
        mbar_wait(bar(kDrain), 0, &flag);
      }
    }
  } else if (warp < 8) {
    // ------------------------------------------ state, decayed values, C^T
    constexpr int NK = KP / 2;  // keys of a thread
    const int half = warp >> 2, v = (warp & 3) * 32 + lane;
    const bool live = (warp & 3) * 32 < p.V;  // warp-uniform
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    const int64_t state_at = ((int64_t)seg.grid * l.heads + h) * p.K * p.V;
    float* seg_state = p.seg ? p.seg + ((int64_t)blockIdx.x * l.heads + h) * p.K * p.V : nullptr;
    float u[NK];
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const int k = half * NK + i;
      u[i] = 0.f;
      if (!kStates && !idle && k < p.K && v < p.V) {
        if (l.phase == 2) u[i] = seg_state[(int64_t)k * p.V + v];
        else if (p.first) u[i] = p.first[state_at + k * p.first_k + v * p.first_v];
      }
    }
    for (int t = 0; t < chunks; ++t) {
      const int st = t % kStages, n = rows_of(t);
      const uint32_t at = stage0 + st * kStageBytes;
      if (!wait(kFull + st, t / kStages)) break;
      if (n < kC) {
        // rows past the segment belong to others: no NaN of theirs may meet the zeros that their weights are
        for (int i = threadIdx.x; i < (kBlocks + value_blocks) * (kC - n) * 8; i += 256) {
          const int blk = i / ((kC - n) * 8), r = i % ((kC - n) * 8);
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(
                           at + (kBlocks + blk) * kTile + n * 128 + r * 16),
                       "r"(0)
                       : "memory");
        }
        fence_async_smem();
        arrive(kZeros);  // once: only the last chunk is short
        if (!wait(kZeros, 0)) break;
      }
      if (!kStates && t >= kCt && !wait(kCFree + t % kCt, t / kCt - 1)) break;
      if (live) {
        // this warp's 32 values x its half of the rows, as 8 x 8 blocks read across: a register is two rows of a value
        const float* w = (reverse ? s.up : s.down[(kC - n) & 3] + ((kC - n) & ~3)) + half * 32 + 2 * (lane & 3);
        float2 wv[4];
#pragma unroll
        for (int m = 0; m < 4; ++m) wv[m] = *reinterpret_cast<const float2*>(w + 8 * m);
        const int r = half * 32 + (lane >> 4) * 8 + (lane & 7);
        const uint32_t rows = at + (2 * kBlocks + ((warp & 3) >> 1)) * kTile + r * 128;
#pragma unroll
        for (int g16 = 0; g16 < 2; ++g16) {
          uint32_t ct[8], x[kTerms][8];
          const uint32_t from = rows + ((((warp & 1) * 4 + g16 * 2 + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
          ldmatrix_trans4(from, ct[0], ct[1], ct[2], ct[3]);
          ldmatrix_trans4(from + 16 * 128, ct[4], ct[5], ct[6], ct[7]);
          uint32_t finite = 0;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(finite) : "r"(ct[i]), "r"(0));
            float e0 = low(ct[i]) * wv[i / 2].x, e1 = high(ct[i]) * wv[i / 2].y;
#pragma unroll
            for (int term = 0; term < kTerms; ++term) {
              x[term][i] = bf16x2(e0, e1);
              e0 -= low(x[term][i]);
              e1 -= high(x[term][i]);
            }
          }
          const bool bad = not_finite(low(finite)) || not_finite(high(finite));
          if (__any_sync(0xffffffffu, bad)) {
            // 0 x infinity of a later row is no part of an earlier row's sum: the product takes zeros, and the
            // output warps add these values to the rows that see them
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (not_finite(low(ct[i]))) ct[i] &= 0xffff0000u;
              if (not_finite(high(ct[i]))) ct[i] &= 0xffffu;
            }
            s.bad[st] = t + 1;
          }
          const uint32_t to = lanes + ((uint32_t)g16 << 20) + half * 16;
#pragma unroll
          for (int term = 0; term < kTerms; ++term) tmem_st_16x16(to + kColW + term * 32, x[term]);
          if (!kStates) tmem_st_16x16(to + kColCt + t % kCt * 32, ct);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      arrive(kWFull);
      if (!kStates) arrive(kCFull + t % kCt);
      arrive(kEmpty + st);
      if (!kStates) {
        // X^T, as an operand, for this chunk
        if (t > 0 && !wait(kStFree, t - 1)) break;
        if (live) {
#pragma unroll
          for (int k0 = 0; k0 < NK; k0 += 32) {
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = bf16x2(u[k0 + 2 * i], u[k0 + 2 * i + 1]);
            tmem_st16(lanes + kColSt + (half * NK + k0) / 2, x);
          }
          tmem_wait_st();
        }
        tc_fence_before();
        arrive(kStFull);
      }
      if (!wait(kKvReady, t)) break;
      tc_fence_after();
      const float d = s.pow[n];
      if (live) {
#pragma unroll
        for (int k0 = 0; k0 < NK; k0 += 16) {
          uint32_t x[16];
          tmem_ld16(lanes + kColKv + half * NK + k0, x);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) u[k0 + i] = fmaf(u[k0 + i], d, __uint_as_float(x[i]));
        }
      }
      tc_fence_before();
      arrive(kKvFree);
    }
    float* dst = kStates ? seg_state : l.phase == 0 && p.last ? p.last + state_at : nullptr;
    if (!idle && dst && !s.gave_up && v < p.V) {
#pragma unroll
      for (int i = 0; i < NK; ++i) {
        const int k = half * NK + i;
        if (k < p.K) dst[(int64_t)k * p.V + v] = u[i];
      }
    }
  } else if (!kStates && warp < kWarpOut) {
    // ------------------------------------------------------------------- P
    const int half = warp & 1, i = half * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    for (int t = 0; t < chunks; ++t) {
      const int n = rows_of(t);
      if (!wait(kPReady + (t & 1), t >> 1)) break;
      tc_fence_after();
      const uint32_t row = tiles + (t & 1) * kTile + i * 128;
#pragma unroll
      for (int b = 0; b < 2; ++b) {  // columns 32 b to 32 b + 31
        uint32_t x[32];
        if (reverse ? b >= half : b <= half) {
          tmem_ld32(lanes + kColP + (t & 1) * 64 + 32 * b, x);
          tmem_wait_ld();
          // fold[|i - j|]; on the diagonal block and past the rows the index may be negative, and P is 0
          if (reverse) {
            const float* w = s.fold + kC + 32 * b - i;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float f = __uint_as_float(x[j]) * w[j];
              x[j] = 32 * b + j >= i && 32 * b + j < n ? __float_as_uint(f) : 0u;
            }
          } else {
            const float* w = s.fold + kC + i - 32 * b;
#pragma unroll
            for (int j = 0; j < 32; ++j) {
              const float f = __uint_as_float(x[j]) * w[-j];
              x[j] = b < half || j <= lane ? __float_as_uint(f) : 0u;
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = 0u;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row + (((b * 4 + q) ^ (i & 7)) << 4)),
                       "r"(bf16x2(__uint_as_float(x[8 * q]), __uint_as_float(x[8 * q + 1]))),
                       "r"(bf16x2(__uint_as_float(x[8 * q + 2]), __uint_as_float(x[8 * q + 3]))),
                       "r"(bf16x2(__uint_as_float(x[8 * q + 4]), __uint_as_float(x[8 * q + 5]))),
                       "r"(bf16x2(__uint_as_float(x[8 * q + 6]), __uint_as_float(x[8 * q + 7])))
                       : "memory");
      }
      fence_async_smem();
      tc_fence_before();
      arrive(kPFull + (t & 1));
    }
  } else if (!kStates) {
    // -------------------------------------------------------------- output
    const bool live = (warp & 3) * 32 < p.V;
    const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
    const uint32_t out0 = stage0 + kStages * kStageBytes + (warp & 3) * 2 * 4096;  // two buffers of 64 rows x 64 bytes
    const CUtensorMap* map = &g.map[kLinMaxRows + blockIdx.z];
    for (int t = 0; t < chunks; ++t) {
      const int st = t % kStages, n = rows_of(t);
      if (!wait(kOReady, t)) break;
      tc_fence_after();
      if (live) {
        const float* w = (reverse ? s.down[(kC - n) & 3] + ((kC - n) & ~3) : s.up) + 2 * (lane & 3);
        const bool bad = s.bad[st] == (uint32_t)t + 1;
        const uint32_t buf = out0 + (t & 1) * 4096;
        if (lane == 0) tma_store_wait<1>();
        __syncwarp();
        const int row = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
        for (int g16 = 0; g16 < 2; ++g16) {
          uint32_t x[32], y[32];
          tmem_ld_16x64(lanes + ((uint32_t)g16 << 20) + kColP + (t & 1) * 64, x);
          tmem_ld_16x64(lanes + ((uint32_t)g16 << 20) + kColOi, y);
          tmem_wait_ld();
          if (g16 == 1 && !bad) {
            tc_fence_before();
            arrive(kOFree);
          }
          const uint32_t to = buf + row * 64 + (((g16 * 2 + ((lane >> 3) & 1)) ^ ((row >> 1) & 3)) << 4);
          uint32_t o[16];
#pragma unroll
          for (int m = 0; m < 8; ++m) {
            const float2 wv = *reinterpret_cast<const float2*>(w + 8 * m);
            auto both = [&](int i) {
              return bf16x2(fmaf(__uint_as_float(y[i]), wv.x, __uint_as_float(x[i])),
                            fmaf(__uint_as_float(y[i + 1]), wv.y, __uint_as_float(x[i + 1])));
            };
            o[2 * m] = both(4 * m);
            o[2 * m + 1] = both(4 * m + 2);
          }
#pragma unroll
          for (int m = 0; m < 4; ++m)
            stmatrix_trans4(to + m * 16 * 64, o[4 * m], o[4 * m + 1], o[4 * m + 2], o[4 * m + 3]);
        }
        __syncwarp();
        if (bad) {
          add_not_finite(buf, tiles + (t & 1) * kTile, stage0 + st * kStageBytes + (2 * kBlocks + ((warp & 3) >> 1)) * kTile,
                         n, reverse);
          tc_fence_before();
          arrive(kOFree);
        }
        const int64_t row0 = row_of(t);
        if (n == kC) {
          fence_async_smem();
          __syncwarp();
          if (lane == 0) tma_store_3d(map, (warp & 3) * 32, h, (int)row0, buf);
        } else {
          // the rows that follow are not this segment's: plain stores
          for (int i = lane; i < n * 4; i += 32) {
            const int rr = i >> 2, v = (warp & 3) * 32 + (i & 3) * 8;
            uint4 o;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(o.x), "=r"(o.y), "=r"(o.z), "=r"(o.w)
                         : "r"(buf + rr * 64 + (((i & 3) ^ ((rr >> 1) & 3)) << 4)));
            if (v < p.V) *reinterpret_cast<uint4*>((__nv_bfloat16*)p.out + (row0 + rr) * p.o_row + h * p.o_head + v) = o;
          }
        }
      } else {
        tc_fence_before();
        arrive(kOFree);
      }
      arrive(kEmpty + st);
    }
    if (lane == 0) tma_store_wait<0>();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && s.gave_up) atomicOr(&g_gave_up, 1u);
  if (warp == kWarpMma) tmem_free(tmem, 512);
}

template <int KP, int kTerms, bool kStates>
cudaError_t go(const ChunkLaunch& g, cudaStream_t s) {
  constexpr int bytes = 1024 + 2 * kTile + stages_of(KP) * (2 * (KP / 64) + 2) * kTile + (kStates ? 0 : 4 * 2 * 4096);
  static_assert(bytes > 116 * 1024 && bytes < 224 * 1024, "one block a multiprocessor: tensor memory is not shared");
  static bool ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(k_chunks<KP, kTerms, kStates>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) ready[dev] = true;
  }
  const dim3 grid(g.l.segments, g.l.heads, g.l.n);
  k_chunks<KP, kTerms, kStates><<<grid, threads_of(kStates), bytes, s>>>(g);
  return cudaGetLastError();
}

typedef CUresult (*Encode)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                           const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                           CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
  static const Encode fn = [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      f = nullptr;
    }
    return (Encode)f;
  }();
  return fn;
}

// Rows [tokens, heads, size] as the copy engine takes them, a box of 64 rows of
// one head: 64 elements of it read, or 32 written.  False where it cannot.
bool row_map(CUtensorMap* m, const void* at, int size, int heads, int64_t tokens, int64_t row, int64_t head, int box_size) {
  if (!encoder() || ((uintptr_t)at & 15)) return false;
  // a stride that nothing is reached by still has to be one the encoding takes
  if (heads == 1) head = size;
  if (tokens == 1) row = (int64_t)heads * size;
  if (head <= 0 || row <= 0 || head % 8 || row % 8 || head >= 1ll << 38 || row >= 1ll << 38) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)size, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)head * 2, (cuuint64_t)row * 2};
  const cuuint32_t box[3] = {(cuuint32_t)box_size, 1, kC}, step[3] = {1, 1, 1};
  return encoder()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(at), dims, strides, box, step,
                   CU_TENSOR_MAP_INTERLEAVE_NONE, box_size == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

bool linear_chunk_plan(ChunkLaunch& g) {
  const LinLaunch& l = g.l;
  struct Rows {
    const void* at;
    int size;
    int64_t row, head;
  } known[kLinMaxRows];
  int n = 0;
  auto find = [&](const Rows& x, uint8_t* to) {
    for (int i = 0; i < n; ++i)
      if (known[i].at == x.at && known[i].size == x.size && known[i].row == x.row && known[i].head == x.head) {
        *to = (uint8_t)i;
        return true;
      }
    if (n == kLinMaxRows || !row_map(&g.map[n], x.at, x.size, l.heads, l.tokens, x.row, x.head, 64)) return false;
    known[n] = x;
    *to = (uint8_t)n++;
    return true;
  };
  if (l.type != TB_TYPE_BF16) return false;
  for (int i = 0; i < l.n; ++i) {
    const LinProblem& p = l.p[i];
    if (p.K % 8 || p.V % 8 || p.reverse != p.late || (p.reverse ? p.mul : p.fold) != 1.f) return false;
    if (!find({p.a, p.K, p.a_row, p.a_head}, &g.a[i]) || !find({p.b, p.K, p.b_row, p.b_head}, &g.b[i]) ||
        !find({p.c, p.V, p.c_row, p.c_head}, &g.c[i]) ||
        !row_map(&g.map[kLinMaxRows + i], p.out, p.V, l.heads, l.tokens, p.o_row, p.o_head, 32))
      return false;
  }
  return true;
}

cudaError_t launch_linear_chunks(const void* args, cudaStream_t s) {
  const ChunkLaunch& g = *(const ChunkLaunch*)args;
  bool wide = false, exact = false;
  for (int i = 0; i < g.l.n; ++i) {
    wide = wide || g.l.p[i].K > 64;
    exact = exact || g.l.p[i].last;
  }
  if (g.l.phase == 1) {
    if (wide) return exact ? go<128, 3, true>(g, s) : go<128, 2, true>(g, s);
    return exact ? go<64, 3, true>(g, s) : go<64, 2, true>(g, s);
  }
  if (g.l.phase == 2) exact = false;  // the states that leave come from phase 1
  if (wide) return exact ? go<128, 3, false>(g, s) : go<128, 2, false>(g, s);
  return exact ? go<64, 3, false>(g, s) : go<64, 2, false>(g, s);
}

cudaError_t linear_gave_up(cudaStream_t s, bool* gave_up) {
  void* at = nullptr;
  unsigned int got = 0;
  cudaError_t e = cudaGetSymbolAddress(&at, g_gave_up);
  if (e == cudaSuccess) e = cudaMemcpyAsync(&got, at, sizeof got, cudaMemcpyDeviceToHost, s);
  if (e == cudaSuccess) e = cudaMemsetAsync(at, 0, sizeof got, s);
  if (e == cudaSuccess) e = cudaStreamSynchronize(s);
  *gave_up = got != 0;
  return e;
}

}  // namespace tb
