// The states of beams follow their parents, in place: sequence s of a group of
// W takes over the first len[p] tokens of sequence p = parent[s] of its group,
// in every array [n_seqs, heads, cap, bytes] (packed codes, norms, windows,
// token histories).
//
// In place without a second copy: a thread owns the same few bytes (a column)
// of all W sequences.  It reads the columns that somebody takes over, all of
// them before it writes the first, and no other thread touches them.  So swaps,
// cycles and several children of one parent need no order between threads.  What
// does not move is neither read nor written.
//
// Columns are 16 bytes wide; where many sequences of a group move and follow each
// other, 8 above 16 sequences and 4 above 32, so that a thread holds 64 registers of
// data in flight; arrays whose rows do not start on such a boundary take the widest
// column that they allow.  The last
// column of a sequence that ends inside it is written byte by byte: what lies
// behind a sequence's tokens is left as it was.
//
// Bound: HBM; a byte that moves is read once and written once.  Rows of 512 KB in
// 8 heads, 32 of 64 sequences moved, in groups of 8, 16 and 64: 39 us, 5.4 to 5.8
// TB/s of the 6.8 of a copy; all of a group of 8 in a cycle 6.2, of 64 (4-byte
// columns) 2.9.  Four moves with four columns each in flight against all of a
// group of 8 with two: 31.0 against 34.6 us for 64 sequences in 17 arrays.
#include <cuda_runtime.h>

#include "tq_launch.cuh"

namespace tq {

int sm_count();

namespace {

constexpr int kThreads = 128;
constexpr int kMaxGroup = 64;
constexpr int kMaxArrays = 96;   // of one launch (the kernel's parameters stay below 4 KB)

struct StateArrays {
  uint8_t* data[kMaxArrays];
  const int32_t* len[kMaxArrays];   // NULL: cap
  int64_t cap[kMaxArrays];          // slots
  int32_t bytes[kMaxArrays];        // of a slot
  int32_t unit0[kMaxArrays];        // (group, head) units before this array
  int32_t heads[kMaxArrays];
  int32_t n, units, groups, W, split;
  const int32_t* parent;            // [groups W]
};

// A sequence that takes over the first `end` bytes of sequence `from`.
struct Move {
  int to, from;
  int64_t end;
};

// Columns of up to M moves, C of a thread in flight: all of them are read before
// the first is written.
template <class T, int M, int C>
__device__ __forceinline__ void move_columns(uint8_t* base, int64_t stride, const Move* moves, int n, int64_t at, int64_t step) {
  constexpr int64_t kCol = sizeof(T);
  T v[C][M];
#pragma unroll
  for (int k = 0; k < M; ++k) {
    if (k >= n) break;
    const Move m = moves[k];
    const uint8_t* from = base + m.from * stride + at;
#pragma unroll
    for (int c = 0; c < C; ++c)
      if (at + c * step < m.end) v[c][k] = *reinterpret_cast<const T*>(from + c * step);
  }
#pragma unroll
  for (int k = 0; k < M; ++k) {
    if (k >= n) break;
    const Move m = moves[k];
    uint8_t* to = base + m.to * stride + at;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int64_t left = m.end - (at + c * step);
      if (left >= kCol) {
        *reinterpret_cast<T*>(to + c * step) = v[c][k];
      } else if (left > 0) {
        for (int b = 0; b < left; ++b) {   // words, not an array whose address is taken
          uint32_t w;
          if constexpr (kCol == 16) w = b < 4 ? v[c][k].x : b < 8 ? v[c][k].y : b < 12 ? v[c][k].z : v[c][k].w;
          else if constexpr (kCol == 8) w = b < 4 ? v[c][k].x : v[c][k].y;
          else w = (uint32_t)v[c][k];
          to[c * step + b] = (uint8_t)(w >> (8 * (b & 3)));
        }
      }
    }
  }
}

// W: sequences of a group at most.  Up to kFew moves, or any number where no
// sequence that moves is another's parent (survivors that stay in their place),
// go kFew at a time, columns T wide and kFewColumns of a thread in flight.  Else
// all of a group's go together, columns TB wide and C of a thread in flight.
constexpr int kFew = 4, kFewColumns = 4;
template <class T, class TB, int W, int C>
__global__ void __launch_bounds__(kThreads) states_kernel(const __grid_constant__ StateArrays a) {
  __shared__ Move s_move[W];
  __shared__ int64_t s_most;
  __shared__ int s_moves, s_chained;
  const int unit = blockIdx.x / a.split, part = blockIdx.x - unit * a.split;
  int i = 0;
  {
    int hi = a.n;
    while (hi - i > 1) {
      const int mid = (i + hi) >> 1;
      if (a.unit0[mid] <= unit) i = mid; else hi = mid;
    }
  }
  const int u = unit - a.unit0[i], heads = a.heads[i], g = u / heads, h = u - g * heads;
  const int64_t row = a.cap[i] * a.bytes[i], stride = row * heads;
  uint8_t* base = a.data[i] + ((int64_t)g * a.W * heads + h) * row;
  if (threadIdx.x < 32) {   // the group's moves, in order, by one warp
    const int lane = threadIdx.x;
    int n = 0;
    int64_t most = 0;
    uint64_t moved = 0, parents = 0;
#pragma unroll
    for (int k0 = 0; k0 < W; k0 += 32) {
      const int k = k0 + lane;
      Move m{k, k, 0};
      if (k < a.W) {
        const int64_t p = (int64_t)a.parent[(int64_t)g * a.W + k] - (int64_t)g * a.W;
        if (p >= 0 && p < a.W && p != k) {   // a parent outside the group: the sequence stays as it is
          m.from = (int)p;
          int64_t len = a.cap[i];
          if (a.len[i]) {
            const int64_t tokens = a.len[i][(int64_t)g * a.W + p];
            len = tokens < 0 ? 0 : imin64(tokens, len);
          }
          m.end = len * a.bytes[i];
        }
      }
      const uint32_t found = __ballot_sync(kFull, m.end > 0);
      if (m.end > 0) s_move[n + __popc(found & ((1u << lane) - 1))] = m;
      n += __popc(found);
      moved |= (uint64_t)found << k0;
      parents |= m.end > 0 ? 1ull << m.from : 0ull;
      most = m.end > most ? m.end : most;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const int64_t other = __shfl_xor_sync(kFull, most, o);
      most = other > most ? other : most;
      parents |= __shfl_xor_sync(kFull, parents, o);
    }
    if (lane == 0) {
      s_moves = n;
      s_most = most;
      s_chained = (moved & parents) != 0;
    }
  }
  __syncthreads();
  const int64_t most = s_most;
  const int n = s_moves;
  if (n <= kFew || !s_chained) {
    constexpr int64_t kCol = sizeof(T), step = kThreads * kCol;
    for (int64_t c0 = (int64_t)part * kFewColumns * step; c0 < most; c0 += (int64_t)a.split * kFewColumns * step)
      for (int k = 0; k < n; k += kFew)
        move_columns<T, kFew, kFewColumns>(base, stride, s_move + k, n - k, c0 + threadIdx.x * kCol, step);
  } else {
    constexpr int64_t kCol = sizeof(TB), step = kThreads * kCol;
    for (int64_t c0 = (int64_t)part * C * step; c0 < most; c0 += (int64_t)a.split * C * step)
      move_columns<TB, W, C>(base, stride, s_move, n, c0 + threadIdx.x * kCol, step);
  }
}

// Bytes of the widest column: what the array's address and rows are multiples of.
int column_of(const tq_state_array& s) {
  const uint64_t m = reinterpret_cast<uintptr_t>(s.data) | (uint64_t)(s.cap * s.bytes);
  return m % 16 == 0 ? 16 : m % 8 == 0 ? 8 : m % 4 == 0 ? 4 : m % 2 == 0 ? 2 : 1;
}

template <class T, class TB, int W, int C>
bool launch_states(StateArrays& a, cudaStream_t st) {
  // blocks of a unit: enough for the whole GPU, none without a column in the longest sequence
  int64_t longest = 0;
  for (int i = 0; i < a.n; ++i) {
    const int64_t row = a.cap[i] * a.bytes[i];
    longest = row > longest ? row : longest;
  }
  const int64_t piece = (int64_t)kThreads * kFewColumns * sizeof(T), pieces = (longest + piece - 1) / piece;
  int64_t split = (8 * (int64_t)sm_count() + a.units - 1) / a.units;
  split = split > pieces ? pieces : split;
  a.split = (int)(split < 1 ? 1 : split);
  return launch(states_kernel<T, TB, W, C>, (int64_t)a.units * a.split, kThreads, false, st, a);
}

// Arrays of one column width and group size.
bool launch_class(StateArrays& a, int col, cudaStream_t st) {
  if (col == 16) {
    if (a.W <= 4) return launch_states<uint4, uint4, 4, kFewColumns>(a, st);
    if (a.W <= 8) return launch_states<uint4, uint4, 8, 2>(a, st);
    if (a.W <= 16) return launch_states<uint4, uint4, 16, 1>(a, st);
    if (a.W <= 32) return launch_states<uint4, uint2, 32, 1>(a, st);
    return launch_states<uint4, uint32_t, 64, 1>(a, st);
  }
  if (col == 8) return launch_states<uint2, uint32_t, 64, 1>(a, st);
  if (col == 4) return launch_states<uint32_t, uint32_t, 64, 1>(a, st);
  if (col == 2) return launch_states<uint16_t, uint16_t, 64, 1>(a, st);
  return launch_states<uint8_t, uint8_t, 64, 1>(a, st);
}

}  // namespace
}  // namespace tq

extern "C" int tq_states_reorder(const tq_state_array* states, int n_states, int n_seqs, int W, const int32_t* parent,
                                 void* stream) {
  if (n_states < 0 || n_seqs < 0 || W <= 0 || (n_states && !states)) return TQ_ERR_ARG;
  if (n_seqs % W) return TQ_ERR_ARG;
  if (W > tq::kMaxGroup) return TQ_ERR_UNSUPPORTED;
  const int groups = n_seqs / W;
  for (int i = 0; i < n_states; ++i) {
    const tq_state_array& s = states[i];
    if (s.cap < 0 || s.heads <= 0 || s.bytes <= 0) return TQ_ERR_ARG;
    if (s.cap > 0 && n_seqs > 0 && !s.data) return TQ_ERR_ARG;
    if (s.cap > 0x7fffffff || (int64_t)groups * s.heads > 1 << 20) return TQ_ERR_UNSUPPORTED;
    if ((reinterpret_cast<uintptr_t>(s.len) & 3u) != 0) return TQ_ERR_ALIGN;
  }
  if (n_states == 0 || n_seqs == 0) return TQ_OK;
  if (!parent) return TQ_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(parent) & 3u) != 0) return TQ_ERR_ALIGN;
  if (W == 1) return TQ_OK;   // nobody has another parent
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  bool ok = true;
  for (int col = 16; col && ok; col >>= 1) {
    tq::StateArrays a{};
    a.groups = groups;
    a.W = W;
    a.parent = parent;
    auto flush = [&]() {
      if (a.n) ok = ok && tq::launch_class(a, col, st);
      a.n = a.units = 0;
    };
    for (int i = 0; i < n_states && ok; ++i) {
      const tq_state_array& s = states[i];
      if (s.cap == 0 || tq::column_of(s) != col) continue;
      const int units = groups * s.heads;
      if (a.n == tq::kMaxArrays || a.units + units > 1 << 20) flush();
      a.data[a.n] = static_cast<uint8_t*>(s.data);
      a.len[a.n] = s.len;
      a.cap[a.n] = s.cap;
      a.bytes[a.n] = s.bytes;
      a.heads[a.n] = s.heads;
      a.unit0[a.n] = a.units;
      a.units += units;
      ++a.n;
    }
    flush();
  }
  return ok && cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
