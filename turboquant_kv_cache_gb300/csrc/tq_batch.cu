// Where the rows of a ragged batch go: requests of different lengths packed
// row behind row.  Sequence b has rows [start_b, start_b + new_len[b]) with
// start the exclusive prefix sum of new_len; its row j is at position
// kv_len[b] + j of the sequence, in the cache slot that the page table (or the
// contiguous layout) gives for that position.
//
// A block sums up the lengths and searches the sums for the sequence of each
// of its rows, so no block waits for another.  Up to kOneLaunch sequences every
// block does the sums for itself, in shared memory; beyond that a block writes
// them first and a second launch searches them in the L2.  A warp looks for the
// sequences of its first and last row, a thread between those two.  Graph
// replays, one launch against two:
//   sequences x rows    256 x 2000    4.0   6.1 us
//                       2048 x 16000  5.0   8.5
//                       4096 x 32000  9.2   9.8
//                       2048 x 1000003  9.0   11.3
//                       4096 x 1000003  22.2  13.3
//
// Bound: a launch and the latency of the sums for small batches (8 sequences and
// 96 rows with a table row each 4.4 us; 16000 rows of 2048 sequences 5.0).  Large
// ones have that too, before a block's first row: 1000003 rows of 2048 sequences take
// 9.2 us, their 20 MB 3 us at a copy's rate.  140 instructions a row keep 44% of the
// issue slots busy, and the rows are 1.6 rounds of the grid: latency and instructions
// about alike (13 us with a search of all sequences by each thread, 11 with
// lengths loaded 4 bytes at a time; 11 with six blocks an SM, 9.5 with two).
#include <cuda_runtime.h>

#include "tq_launch.cuh"

namespace tq {

int sm_count();

namespace {

constexpr int kThreads = 256;
constexpr int kSumThreads = 1024;
constexpr int kOneLaunch = 2048;   // sequences whose sums every block does for itself
constexpr int kRowsPerThread = 4;
constexpr int kAhead = 4;          // table pieces a warp has in flight
constexpr int kMostSeqs = 1 << 20;

struct SlotArgs {
  const int32_t* new_len;
  const int32_t* kv_len;       // NULL: 0
  const int32_t* page_table;   // NULL: contiguous
  int64_t S_cap;
  int32_t page_size, pages_per_seq, B, n_rows;
  FastDiv by_page;             // division by page_size
  int32_t* row_start;          // [B + 1]
  int32_t* seq;                // [n_rows] or NULL
  int32_t* pos;                // [n_rows]
  int64_t* slot;               // [n_rows]
  int32_t* row_len;            // [n_rows] or NULL
  int32_t* row_table;          // [n_rows][row_pages] or NULL
  int32_t row_pages;
  int32_t* result;             // [4] or NULL
};

// Sum over the block's threads before this one of their v, modulo 2^32 (which
// is what counts where all rows fit), and *total, the sum of all in 64 bits.
// Every thread calls it; s_part holds a value for each warp and direction.
__device__ __forceinline__ uint32_t scan_rows(int64_t v, uint32_t (*s_part)[3], int64_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  uint32_t x = (uint32_t)v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  // the sum of a thread in pieces of 22 bits
  const uint32_t lo = __reduce_add_sync(kFull, (uint32_t)v & 0x3fffffu), hi = __reduce_add_sync(kFull, (uint32_t)(v >> 22));
  __syncthreads();   // the parts of an earlier call have been read
  if (lane == 31) {
    s_part[w][0] = x;
    s_part[w][1] = lo;
    s_part[w][2] = hi;
  }
  __syncthreads();
  const bool mine = lane < nw;
  const uint32_t before = __reduce_add_sync(kFull, mine && lane < w ? s_part[lane][0] : 0u);
  *total = (int64_t)__reduce_add_sync(kFull, mine ? s_part[lane][1] : 0u);
  // (1024 threads of 2^41 rows at most, see kMostSeqs: the pieces add up in 32 bits)
  *total += (int64_t)__reduce_add_sync(kFull, mine ? s_part[lane][2] : 0u) << 22;
  return before + x - (uint32_t)v;
}

__device__ __forceinline__ bool length_ok(const SlotArgs& a, int len, int have) {
  return (len | have) >= 0 && (uint32_t)len + (uint32_t)have <= (uint32_t)a.S_cap;   // S_cap is below 2^31
}

// {status, rows, 0, 0} of the whole batch; rows that are not laid out are none.
__device__ __forceinline__ int64_t report(const SlotArgs& a, bool bad, int64_t total, bool write) {
  const bool ok = !bad && total <= a.n_rows;
  if (write && a.result) {
    const int64_t missing = total - a.n_rows;
    a.result[0] = bad ? -1 : ok ? 0 : (int)imin64(missing, 0x7fffffff);
    a.result[1] = ok ? (int)total : 0;
    a.result[2] = a.result[3] = 0;
  }
  return ok ? total : 0;
}

// The sequence of row r, one of [lo, hi]: the first whose rows end behind it
// (end[b] > r).
__device__ __forceinline__ int find_seq(const int32_t* end, int lo, int hi, int r) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > r) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Rows and table rows of this block, given the ends of the sequences' rows,
// shift(b), what a row of sequence b lacks of its position, and the rows in all.
template <class Shift>
__device__ __forceinline__ void write_rows(const SlotArgs& a, const int32_t* end, Shift shift, int total) {
  constexpr int R = kRowsPerThread;
  const uint32_t tid = blockIdx.x * kThreads + threadIdx.x, threads = gridDim.x * kThreads;
  // (whole warps: they look for their sequences together)
  for (uint32_t r0 = tid * R; r0 - (threadIdx.x & 31) * R < (uint32_t)a.n_rows; r0 += threads * R) {
    int seq[R], pos[R], len[R], page[R];
    int64_t slot[R];
    // the sequences of the warp's rows: lane 0 looks for the first, lane 1 for the last
    const uint32_t w0 = r0 - (threadIdx.x & 31) * R, w1 = min(w0 + 32 * R, (uint32_t)total);
    int lo = 0, hi = 0;
    if (w0 < w1) {
      const int found = find_seq(end, 0, a.B - 1, (int)((threadIdx.x & 31) == 0 ? w0 : w1 - 1));
      lo = __shfl_sync(kFull, found, 0);
      hi = __shfl_sync(kFull, found, 1);
    }
    int b = -1, last = 0;   // b has rows up to last
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int r = (int)r0 + k;
      seq[k] = pos[k] = -1;
      len[k] = 0;
      if (r0 + k < (uint32_t)total) {
        if (b < 0 || r >= last) {
          b = find_seq(end, b < 0 ? lo : b + 1, hi, r);
          last = end[b];
        }
        seq[k] = b;
        pos[k] = r + shift(b);
        len[k] = pos[k] + 1;
      }
    }
    // the rows' pages, loaded together
#pragma unroll
    for (int k = 0; k < R; ++k) {
      page[k] = -1;
      slot[k] = -1;
      if (a.page_table && seq[k] >= 0) {
        const uint32_t pg = fast_div((uint32_t)pos[k], a.by_page);
        page[k] = a.page_table[(int64_t)seq[k] * a.pages_per_seq + pg];
        slot[k] = pos[k] - (int)pg * a.page_size;
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      if (a.page_table) slot[k] = page[k] < 0 ? -1 : (int64_t)page[k] * a.page_size + slot[k];
      else if (seq[k] >= 0) slot[k] = seq[k] * a.S_cap + pos[k];
    }
    if (r0 + R <= (uint32_t)a.n_rows) {
      if (a.seq) *reinterpret_cast<int4*>(a.seq + r0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      *reinterpret_cast<int4*>(a.pos + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (a.row_len) *reinterpret_cast<int4*>(a.row_len + r0) = make_int4(len[0], len[1], len[2], len[3]);
      *reinterpret_cast<longlong2*>(a.slot + r0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2*>(a.slot + r0 + 2) = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (r0 + k >= (uint32_t)a.n_rows) break;
        if (a.seq) a.seq[r0 + k] = seq[k];
        a.pos[r0 + k] = pos[k];
        if (a.row_len) a.row_len[r0 + k] = len[k];
        a.slot[r0 + k] = slot[k];
      }
    }
  }
  if (!a.row_table) return;
  // table rows in pieces of 32 entries, a warp each, kAhead of them in flight
  const int lane = threadIdx.x & 31;
  const uint32_t pieces = (a.row_pages + 31) / 32;
  const int64_t items = (int64_t)a.n_rows * pieces, warps = threads / 32;
  for (int64_t it0 = tid / 32; it0 < items; it0 += warps * kAhead) {
    int v[kAhead];
    int64_t to[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t it = it0 + u * warps;
      const int64_t r = div_small(it, pieces);
      const int j = (int)(it - r * pieces) * 32 + lane;
      v[u] = 0;
      to[u] = it < items && j < a.row_pages ? r * a.row_pages + j : -1;
      if (to[u] >= 0 && r < total) v[u] = a.page_table[(int64_t)find_seq(end, 0, a.B - 1, (int)r) * a.pages_per_seq + j];
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u)
      if (to[u] >= 0) a.row_table[to[u]] = v[u];
  }
}

// A thread's run of `per` sequences: their rows in all, and whether one's
// lengths are not valid.
__device__ __forceinline__ int64_t run_sum(const SlotArgs& a, int b0, int b1, bool* bad) {
  int64_t sum = 0;
  for (int b = b0; b < b1; ++b) {
    const int len = a.new_len[b], have = a.kv_len ? a.kv_len[b] : 0;
    if (length_ok(a, len, have)) sum += len; else *bad = true;
  }
  return sum;
}

template <int MOST>   // sequences of a thread
__global__ void __launch_bounds__(kThreads) batch_slots_kernel(const SlotArgs a) {
  extern __shared__ int32_t s_end[];   // [B], then what a row of each lacks of its position
  int32_t* s_shift = s_end + a.B;
  __shared__ uint32_t s_part[kThreads / 32][3];
  const int b0 = min((int)threadIdx.x * MOST, a.B), n = min(MOST, a.B - b0);
  int len[MOST], have[MOST];
  // all of a thread's loads in flight, 16 bytes at a time where its run is whole
  const bool wide = MOST % 4 == 0 && n == MOST &&
                    ((reinterpret_cast<uintptr_t>(a.new_len) | reinterpret_cast<uintptr_t>(a.kv_len)) & 15u) == 0;
  if (wide) {
    if constexpr (MOST % 4 == 0) {
#pragma unroll
      for (int k = 0; k < MOST; k += 4) {
        const int4 l = *reinterpret_cast<const int4*>(a.new_len + b0 + k);
        const int4 h = a.kv_len ? *reinterpret_cast<const int4*>(a.kv_len + b0 + k) : make_int4(0, 0, 0, 0);
        len[k] = l.x, len[k + 1] = l.y, len[k + 2] = l.z, len[k + 3] = l.w;
        have[k] = h.x, have[k + 1] = h.y, have[k + 2] = h.z, have[k + 3] = h.w;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < MOST; ++k) {
      len[k] = k < n ? a.new_len[b0 + k] : 0;
      have[k] = k < n && a.kv_len ? a.kv_len[b0 + k] : 0;
    }
  }
  bool bad = false;
  int64_t sum = 0;
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    if (length_ok(a, len[k], have[k])) sum += len[k]; else bad = true;
  }
  int64_t all;
  uint32_t at = scan_rows(sum, s_part, &all);
  const bool any_bad = __syncthreads_or(bad);
  const bool first = blockIdx.x == 0;
  const int total = (int)report(a, any_bad, all, first && threadIdx.x == 0);
  if (first && threadIdx.x == 0) a.row_start[0] = 0;
#pragma unroll
  for (int k = 0; k < MOST; ++k) {
    if (k >= n) break;
    const int start = (int)at;
    if (total) at += len[k];
    const int end = total ? (int)at : 0;
    s_end[b0 + k] = end;
    s_shift[b0 + k] = have[k] - start;
    if (first) a.row_start[b0 + k + 1] = end;
  }
  __syncthreads();
  write_rows(a, s_end, [&](int b) { return s_shift[b]; }, total);
}

// Many sequences: the sums by one block.
__global__ void __launch_bounds__(kSumThreads) batch_sums_kernel(const SlotArgs a) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");   // first of its call: nothing to wait for
  __shared__ uint32_t s_part[kSumThreads / 32][3];
  const int64_t per64 = (a.B + kSumThreads - 1) / kSumThreads;
  const int b0 = (int)imin64(threadIdx.x * per64, a.B), b1 = (int)imin64(b0 + per64, a.B);
  bool bad = false;
  const int64_t sum = run_sum(a, b0, b1, &bad);
  int64_t all;
  uint32_t at = scan_rows(sum, s_part, &all);
  const bool any_bad = __syncthreads_or(bad);
  const int64_t total = report(a, any_bad, all, threadIdx.x == 0);
  if (threadIdx.x == 0) a.row_start[0] = 0;
  for (int b = b0; b < b1; ++b) {
    if (total) at += a.new_len[b];
    a.row_start[b + 1] = total ? (int)at : 0;
  }
}

__global__ void __launch_bounds__(kThreads) batch_rows_kernel(const SlotArgs a) {
  chain_begin();
  write_rows(a, a.row_start + 1, [&](int b) { return (a.kv_len ? a.kv_len[b] : 0) - a.row_start[b]; }, a.row_start[a.B]);
}

}  // namespace
}  // namespace tq

extern "C" int tq_batch_slots(const int32_t* new_len, const int32_t* kv_len, int B, int64_t S_cap,
                              const int32_t* page_table, int page_size, int pages_per_seq, int n_rows,
                              int32_t* row_start, int32_t* seq, int32_t* pos, int64_t* slot, int32_t* row_len,
                              int32_t* row_table, int row_pages, int32_t* result, void* stream) {
  if (B <= 0 || n_rows < 0 || S_cap <= 0 || row_pages < 0 || !new_len || !row_start) return TQ_ERR_ARG;
  if (n_rows && (!pos || !slot)) return TQ_ERR_ARG;
  if (page_table && (page_size <= 0 || page_size % 32 || pages_per_seq <= 0 ||
                     (int64_t)page_size * pages_per_seq < S_cap))
    return TQ_ERR_ARG;
  if (row_table && (!page_table || row_pages < 1 || row_pages > pages_per_seq)) return TQ_ERR_ARG;
  // positions are 32-bit, and a thread adds up 2^10 sequences at most
  if (S_cap > 0x7fffffff - 64 || B > tq::kMostSeqs) return TQ_ERR_UNSUPPORTED;
  if (!tq::aligned16(seq) || !tq::aligned16(pos) || !tq::aligned16(slot) || !tq::aligned16(row_len)) return TQ_ERR_ALIGN;
  for (const void* p : {(const void*)new_len, (const void*)kv_len, (const void*)page_table, (const void*)row_start,
                        (const void*)row_table, (const void*)result})
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return TQ_ERR_ALIGN;
  const tq::SlotArgs a{new_len, kv_len, page_table, S_cap, page_size, pages_per_seq, B, n_rows,
                       tq::make_div(page_table ? page_size : 1), row_start, seq, pos,
                       slot, row_len, row_table, row_table ? row_pages : 0, result};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // a thread's four rows, and where table rows are written four pieces a warp
  const int64_t by_rows = (n_rows + tq::kThreads * tq::kRowsPerThread - 1) / (tq::kThreads * tq::kRowsPerThread);
  const int64_t pieces = (int64_t)n_rows * ((a.row_pages + 31) / 32);
  const int64_t by_table = (pieces + tq::kAhead * tq::kThreads / 32 - 1) / (tq::kAhead * tq::kThreads / 32);
  const int64_t want = by_rows > by_table ? by_rows : by_table, most = 4 * tq::sm_count();
  const int64_t grid = want < 1 ? 1 : want > most ? most : want;
  bool ok;
  if (B <= tq::kOneLaunch) {
    constexpr int T = tq::kThreads;
    const auto kern = B <= T ? tq::batch_slots_kernel<1> : B <= 4 * T ? tq::batch_slots_kernel<4>
                                                                     : tq::batch_slots_kernel<tq::kOneLaunch / T>;
    kern<<<(unsigned)grid, tq::kThreads, 8 * (size_t)B, st>>>(a);
    ok = true;
  } else {
    ok = tq::launch(tq::batch_sums_kernel, 1, tq::kSumThreads, false, st, a) &&
         (!n_rows || tq::launch(tq::batch_rows_kernel, grid, tq::kThreads, true, st, a));
  }
  return ok && cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
