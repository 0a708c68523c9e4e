// Where the rows of a ragged batch go: requests of different lengths packed
// row behind row.  Sequence b has rows [start_b, start_b + new_len[b]) with
// start the exclusive prefix sum of new_len; its row j is at position
// kv_len[b] + j of the sequence, in the cache slot that the page table (or the
// contiguous layout) gives for that position.
//
// A block sums up the lengths and searches the sums for the sequence of each
// of its rows, so no block waits for another.  Up to kOneLaunch sequences every
// block does the sums for itself, in shared memory; beyond that a block writes
// them first and a second launch searches them in the L2.
//
// Bound: a launch and the latency of the sums for small batches; the writes,
// 20 bytes a row, for large ones.
#include <cuda_runtime.h>

#include "tq_launch.cuh"

namespace tq {

int sm_count();

namespace {

constexpr int kThreads = 256;
constexpr int kSumThreads = 1024;
constexpr int kOneLaunch = 4096;   // sequences whose sums every block does for itself
constexpr int kRowsPerThread = 4;
constexpr int kAhead = 4;          // table pieces a warp has in flight

struct SlotArgs {
  const int32_t* new_len;
  const int32_t* kv_len;       // NULL: 0
  const int32_t* page_table;   // NULL: contiguous
  int64_t S_cap;
  int32_t page_size, pages_per_seq, B, n_rows;
  int32_t* row_start;          // [B + 1]
  int32_t* seq;                // [n_rows] or NULL
  int32_t* pos;                // [n_rows]
  int64_t* slot;               // [n_rows]
  int32_t* row_len;            // [n_rows] or NULL
  int32_t* row_table;          // [n_rows][row_pages] or NULL
  int32_t row_pages;
  int32_t* result;             // [4] or NULL
};

// Sum of v over the block's threads before this one; *total over all.  Every
// thread calls it; s_part holds blockDim.x / 32 values.
__device__ __forceinline__ int64_t scan64(int64_t v, int64_t* s_part, int64_t* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // the parts of an earlier call have been read
  if (lane == 31) s_part[w] = x;
  __syncthreads();
  int64_t before = 0, all = 0;
  for (int i = 0; i < nw; ++i) {
    const int64_t p = s_part[i];
    if (i < w) before += p;
    all += p;
  }
  *total = all;
  return before + x - v;
}

__device__ __forceinline__ bool length_ok(const SlotArgs& a, int len, int have) {
  return len >= 0 && have >= 0 && (int64_t)len + have <= a.S_cap;
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

// The sequence of row r: the first whose rows end behind it (end[b] > r).
__device__ __forceinline__ int find_seq(const int32_t* end, int B, int r) {
  int lo = 0, hi = B - 1;   // a live row has one
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > r) hi = mid; else lo = mid + 1;
  }
  return lo;
}

// Rows and table rows of this block, given the ends of the sequences' rows and
// their number of rows in all.
__device__ __forceinline__ void write_rows(const SlotArgs& a, const int32_t* end, int total) {
  constexpr int R = kRowsPerThread;
  const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x, threads = (int64_t)gridDim.x * kThreads;
  for (int64_t r0 = tid * R; r0 < a.n_rows; r0 += threads * R) {
    int seq[R], pos[R], len[R];
    int64_t slot[R];
    int b = -1, last = 0, shift = 0;   // b has rows up to last; position = row + shift
#pragma unroll
    for (int k = 0; k < R; ++k) {
      const int r = (int)r0 + k;
      seq[k] = pos[k] = -1;
      len[k] = 0;
      slot[k] = -1;
      if (r0 + k < total) {
        if (b < 0 || r >= last) {
          b = find_seq(end, a.B, r);
          last = end[b];
          shift = (a.kv_len ? a.kv_len[b] : 0) - (b ? end[b - 1] : 0);
        }
        const int p = r + shift;
        seq[k] = b;
        pos[k] = p;
        len[k] = p + 1;
        if (a.page_table) {
          const int pg = p / a.page_size;
          const int page = a.page_table[(int64_t)b * a.pages_per_seq + pg];
          slot[k] = page < 0 ? -1 : (int64_t)page * a.page_size + (p - pg * a.page_size);
        } else {
          slot[k] = b * a.S_cap + p;
        }
      }
    }
    if (r0 + R <= a.n_rows) {
      if (a.seq) *reinterpret_cast<int4*>(a.seq + r0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      *reinterpret_cast<int4*>(a.pos + r0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (a.row_len) *reinterpret_cast<int4*>(a.row_len + r0) = make_int4(len[0], len[1], len[2], len[3]);
      *reinterpret_cast<longlong2*>(a.slot + r0) = make_longlong2(slot[0], slot[1]);
      *reinterpret_cast<longlong2*>(a.slot + r0 + 2) = make_longlong2(slot[2], slot[3]);
    } else {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (r0 + k >= a.n_rows) break;
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
  const int pieces = (a.row_pages + 31) / 32;
  const int64_t items = (int64_t)a.n_rows * pieces, warps = threads / 32;
  for (int64_t it0 = tid / 32; it0 < items; it0 += warps * kAhead) {
    int v[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t it = it0 + u * warps;
      const int64_t r = it / pieces;
      const int j = (int)(it - r * pieces) * 32 + lane;
      v[u] = it < items && r < total && j < a.row_pages
                 ? a.page_table[(int64_t)find_seq(end, a.B, (int)r) * a.pages_per_seq + j]
                 : 0;
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int64_t it = it0 + u * warps;
      const int64_t r = it / pieces;
      const int j = (int)(it - r * pieces) * 32 + lane;
      if (it < items && j < a.row_pages) a.row_table[r * a.row_pages + j] = v[u];
    }
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

__global__ void __launch_bounds__(kThreads) batch_slots_kernel(const SlotArgs a) {
  __shared__ int32_t s_end[kOneLaunch];
  __shared__ int64_t s_part[kThreads / 32];
  const int per = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
  bool bad = false;
  const int64_t sum = run_sum(a, b0, b1, &bad);
  int64_t all;
  int64_t at = scan64(sum, s_part, &all);
  const bool any_bad = __syncthreads_or(bad);
  const bool first = blockIdx.x == 0;
  const int total = (int)report(a, any_bad, all, first && threadIdx.x == 0);
  if (first && threadIdx.x == 0) a.row_start[0] = 0;
  for (int b = b0; b < b1; ++b) {
    if (total) at += a.new_len[b];
    const int end = total ? (int)at : 0;
    s_end[b] = end;
    if (first) a.row_start[b + 1] = end;
  }
  __syncthreads();
  write_rows(a, s_end, total);
}

// Many sequences: the sums by one block.
__global__ void __launch_bounds__(kSumThreads) batch_sums_kernel(const SlotArgs a) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");   // first of its call: nothing to wait for
  __shared__ int64_t s_part[kSumThreads / 32];
  const int64_t per64 = (a.B + kSumThreads - 1) / kSumThreads;
  const int b0 = (int)imin64(threadIdx.x * per64, a.B), b1 = (int)imin64(b0 + per64, a.B);
  bool bad = false;
  const int64_t sum = run_sum(a, b0, b1, &bad);
  int64_t all;
  int64_t at = scan64(sum, s_part, &all);
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
  write_rows(a, a.row_start + 1, a.row_start[a.B]);
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
  if (S_cap > 0x7fffffff - 64) return TQ_ERR_UNSUPPORTED;   // positions are 32-bit
  if (!tq::aligned16(seq) || !tq::aligned16(pos) || !tq::aligned16(slot) || !tq::aligned16(row_len)) return TQ_ERR_ALIGN;
  for (const void* p : {(const void*)new_len, (const void*)kv_len, (const void*)page_table, (const void*)row_start,
                        (const void*)row_table, (const void*)result})
    if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return TQ_ERR_ALIGN;
  const tq::SlotArgs a{new_len, kv_len, page_table, S_cap, page_size, pages_per_seq, B, n_rows, row_start, seq, pos,
                       slot, row_len, row_table, row_table ? row_pages : 0, result};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  // a thread's four rows, and where table rows are written four pieces a warp
  const int64_t by_rows = (n_rows + tq::kThreads * tq::kRowsPerThread - 1) / (tq::kThreads * tq::kRowsPerThread);
  const int64_t pieces = (int64_t)n_rows * ((a.row_pages + 31) / 32);
  const int64_t by_table = (pieces + tq::kAhead * tq::kThreads / 32 - 1) / (tq::kAhead * tq::kThreads / 32);
  const int64_t want = by_rows > by_table ? by_rows : by_table, most = 8 * tq::sm_count();
  const int64_t grid = want < 1 ? 1 : want > most ? most : want;
  bool ok;
  if (B <= tq::kOneLaunch) {
    ok = tq::launch(tq::batch_slots_kernel, grid, tq::kThreads, false, st, a);
  } else {
    ok = tq::launch(tq::batch_sums_kernel, 1, tq::kSumThreads, false, st, a) &&
         (!n_rows || tq::launch(tq::batch_rows_kernel, grid, tq::kThreads, true, st, a));
  }
  return ok && cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
