// Host-side launchers of the sequence operators' kernels (internal to libtb.so).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/tb.h"

namespace tb {

// Kernel kinds of tb_profile_read, continued by the sequence operators.
enum SeqKernel {
  kSeqRotary, kSeqNorm, kSeqNormBackward, kSeqNormWeight, kSeqStep, kSeqScan,
  kSeqChunks, kSeqChunkStates, kSeqSplit, kSeqSplitStates, kSeqCombine, kSeqSelftest, kSeqNumKernels
};

// Every launch of a sequence operator is counted, and timed when profiling is
// enabled on the calling thread (defined next to the pass kernels' own).
typedef cudaError_t (*SeqLaunch)(const void* args, cudaStream_t s);
cudaError_t seq_launch(SeqKernel kind, cudaStream_t s, SeqLaunch f, const void* args);
tb_status seq_fail(tb_status st, const char* fmt, ...);
// Multiprocessors of the current device (0: no device).
int seq_sms();

// ------------------------------------------------------------------- rotary
struct RotaryLaunch {
  tb_rotary_args a;
  int vec;        // elements of the vectors that rows are moved by
  int per_block;  // tokens of one block
};
cudaError_t launch_rotary(const void* args, cudaStream_t s);

// --------------------------------------------------------------------- norm
struct NormLaunch {
  tb_norm_args a;
  int vec, per_row, nv, rows;  // threads of a row, vectors of a thread, rows of a block
  int groups;                  // through shared memory by groups of `rows` rows, nv buffers deep, per_row threads a block; 0: not
  int blocks;
};
// Bytes of a buffer for a group of rows, which starts anywhere in a vector.
constexpr size_t norm_buffer_bytes(int width, int size, int rows) {
  return ((size_t)rows * width * size + ((size_t)rows * width * size % 16 ? 15 + 16 : 0)) / 16 * 16;
}
// Shared memory of the kernels that move groups of rows: `fixed` bytes an
// element of a row (a multiple of 16 in all), then the buffers.
inline size_t norm_group_bytes(int width, int size, int tensors, int rows, int stages, int fixed) {
  const size_t head = fixed == 8 ? 2 * (((size_t)width + 3) / 4 * 16) : ((size_t)width * size + 15) / 16 * 16;
  return head + stages * tensors * norm_buffer_bytes(width, size, rows);
}
constexpr int kNormGroupBytes = 200 * 1024;  // at most
cudaError_t launch_norm(const void* args, cudaStream_t s);
struct NormBackwardLaunch {
  tb_norm_backward_args a;
  int vec, per_row, nv, rows;
  int groups;
  int blocks;
};
cudaError_t launch_norm_backward(const void* args, cudaStream_t s);
cudaError_t launch_norm_weight(const void* args, cudaStream_t s);

// --------------------------------------------------------- linear attention
struct StepLaunch {
  tb_linear_step_args a;
};
cudaError_t launch_linear_step(const void* args, cudaStream_t s);

// One sum over the earlier rows of every grid, in the order of `reverse`:
//   U_t = d U_{t-1} + fold * b_t c_t^T,   out_t = mul * a_t U_t
// over rows a, b [T, H, K] and c, out [T, H, V].  The forward pass and the
// three gradients are this sum over different rows:
//   o  = sum(q, k, v)             forward,  state S,   mul = scale
//   dq = sum(do, v, k)            forward,  state S^T, mul = scale
//   dv = sum(k, q, do)            reverse,  state U,   fold = scale
//   dk = sum(v, do, q)            reverse,  state U^T, fold = scale
// The carried state X of the forward order is S after a token (decayed as the
// next one enters, late = 0); that of the reverse order is decayed as a token
// leaves (late = 1), so that the gradient of a grid's last state enters its
// last token undecayed and the gradient of its first state comes out decayed.
struct LinProblem {
  const void *a, *b, *c;
  void* out;                  // NULL: the states alone
  int64_t a_row, a_head, b_row, b_head, c_row, c_head, o_row, o_head;
  int32_t K, V;
  const float* first;         // [B, H] states a grid starts from, or NULL: zero
  int64_t first_k, first_v;   // element strides of one state (transposed reads)
  float* last;                // [B, H, K, V] states that come out, or NULL
  float* seg;                 // [segments, H, K, V]: states of the segments of a split call
  float mul, fold;
  int32_t reverse, late;
  int32_t vec;                // rows of a (1) and b (2) that 16-byte vectors of 8 elements can read
};
constexpr int kLinMaxProblems = 3;
struct LinLaunch {
  LinProblem p[kLinMaxProblems];
  int32_t n;
  int32_t type;
  int32_t heads;
  int32_t grids;
  int64_t tokens;
  const int64_t* offsets;     // NULL: one grid of all tokens
  const float* decay;
  int32_t segment;            // tokens of one segment; 0: a grid is one segment
  int32_t segments;           // segment slots: the grid's x extent
  int32_t phase;              // 0: whole grids; 1: states of segments; 2: outputs of segments
  int32_t sorted;             // chunk kernel, whole grids: the longest ones first
};
constexpr int kLinMaxSorted = 64;  // grids that a warp sorts
// Whether a block of the chunk kernel takes two heads (one head alone goes the
// same way: 27 grids of 1570 rows with states, the gradient 77 us, 105 as a
// single head; 300 of 64 rows 16.4 and 14.5).
inline bool linear_pairs(int K, int V) { return K <= 64 && V <= 64; }
// The chunk kernel's call (tb_linattn_chunk.cu): the walk and the row tensors
// as the copy engine reads them.
constexpr int kLinMaxRows = 4;
struct ChunkLaunch {
  LinLaunch l;
  CUtensorMap map[kLinMaxRows + kLinMaxProblems];  // rows that are read, then the problems' outputs
  uint8_t a[kLinMaxProblems], b[kLinMaxProblems], c[kLinMaxProblems];  // the maps of a problem's rows
};
// Completes g for its g.l; false where the chunk kernel does not take the rows.
bool linear_chunk_plan(ChunkLaunch& g);
cudaError_t launch_linear_chunks(const void* args, cudaStream_t s);
// The same chunks for any rows, as sums of bfloat16 terms (tb_linattn_split.cu).
cudaError_t launch_linear_split(const void* args, cudaStream_t s);
// Blocks of a chunk kernel in which a bounded wait gave up so far.  Waits for the stream.
cudaError_t linear_split_gave_up(cudaStream_t s, unsigned int* count);
cudaError_t linear_gave_up(cudaStream_t s, unsigned int* count);
// A wait of the given polls (uint32_t) that gives up.
cudaError_t linear_selftest(const void* args, cudaStream_t s);
cudaError_t linear_split_selftest(const void* args, cudaStream_t s);
cudaError_t launch_linear_scan(const void* args, cudaStream_t s);
cudaError_t launch_linear_combine(const void* args, cudaStream_t s);

}  // namespace tb
