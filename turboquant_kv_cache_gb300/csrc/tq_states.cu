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
// Columns are 16 bytes wide up to 16 sequences, 8 up to 32 and 4 up to 64, so
// that a thread holds 64 registers of data in flight; arrays whose rows do not
// start on such a boundary take the widest column that they allow.  The last
// column of a sequence that ends inside it is written byte by byte: what lies
// behind a sequence's tokens is left as it was.
//
// Bound: HBM; a byte that moves is read once and written once.
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

// T: a column.  W: sequences of a group at most.  C: columns in flight.
template <class T, int W, int C>
__global__ void __launch_bounds__(kThreads) states_kernel(const __grid_constant__ StateArrays a) {
  constexpr int64_t kCol = sizeof(T);
  __shared__ int s_from[W];
  __shared__ int64_t s_end[W];   // bytes that the sequence takes over
  __shared__ int64_t s_most;
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
  if (threadIdx.x < W) {
    const int k = threadIdx.x;
    int from = k;
    int64_t end = 0;
    if (k < a.W) {
      const int64_t p = (int64_t)a.parent[(int64_t)g * a.W + k] - (int64_t)g * a.W;
      if (p >= 0 && p < a.W && p != k) {   // a parent outside the group: the sequence stays as it is
        from = (int)p;
        int64_t len = a.cap[i];
        if (a.len[i]) {
          const int64_t n = a.len[i][(int64_t)g * a.W + p];
          len = n < 0 ? 0 : imin64(n, len);
        }
        end = len * a.bytes[i];
      }
    }
    s_from[k] = from;
    s_end[k] = end;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int64_t most = 0;
    for (int k = 0; k < W; ++k) most = s_end[k] > most ? s_end[k] : most;
    s_most = most;
  }
  __syncthreads();
  const int64_t most = s_most, step = kThreads * kCol;
  for (int64_t c0 = (int64_t)part * C * step; c0 < most; c0 += (int64_t)a.split * C * step) {
    T v[C][W];
    const int64_t at = c0 + threadIdx.x * kCol;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const int64_t end = s_end[k];
      const uint8_t* from = base + s_from[k] * stride + at;
#pragma unroll
      for (int c = 0; c < C; ++c)
        if (at + c * step < end) v[c][k] = *reinterpret_cast<const T*>(from + c * step);
    }
#pragma unroll
    for (int k = 0; k < W; ++k) {
      const int64_t end = s_end[k];
      uint8_t* to = base + k * stride + at;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int64_t left = end - (at + c * step);
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
}

// Bytes of the widest column: what the array's address and rows are multiples of.
int column_of(const tq_state_array& s) {
  const uint64_t m = reinterpret_cast<uintptr_t>(s.data) | (uint64_t)(s.cap * s.bytes);
  return m % 16 == 0 ? 16 : m % 8 == 0 ? 8 : m % 4 == 0 ? 4 : m % 2 == 0 ? 2 : 1;
}

template <class T, int W, int C>
bool launch_states(StateArrays& a, cudaStream_t st) {
  // blocks of a unit: enough for the whole GPU, none without a column in the longest sequence
  int64_t longest = 0;
  for (int i = 0; i < a.n; ++i) {
    const int64_t row = a.cap[i] * a.bytes[i];
    longest = row > longest ? row : longest;
  }
  const int64_t pieces = (longest + kThreads * C * (int64_t)sizeof(T) - 1) / (kThreads * C * (int64_t)sizeof(T));
  int64_t split = (8 * (int64_t)sm_count() + a.units - 1) / a.units;
  split = split > pieces ? pieces : split;
  a.split = (int)(split < 1 ? 1 : split);
  return launch(states_kernel<T, W, C>, (int64_t)a.units * a.split, kThreads, false, st, a);
}

// Arrays of one column width and group size.
bool launch_class(StateArrays& a, int col, cudaStream_t st) {
  if (col >= 16 && a.W <= 4) return launch_states<uint4, 4, 4>(a, st);
  if (col >= 16 && a.W <= 8) return launch_states<uint4, 8, 2>(a, st);
  if (col >= 16 && a.W <= 16) return launch_states<uint4, 16, 1>(a, st);
  if (col >= 8 && a.W <= 32) return launch_states<uint2, 32, 1>(a, st);
  if (col >= 4) return launch_states<uint32_t, 64, 1>(a, st);
  if (col >= 2) return launch_states<uint16_t, 64, 1>(a, st);
  return launch_states<uint8_t, 64, 1>(a, st);
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
