// The page table's life on the device: sequences fork (sharing full pages by
// reference, copying the part-filled one), grow, give up their pages, and the
// pool is compacted.  Nothing is read back by the host: the number of pages
// taken or moved is decided by kernels and the copies run over lists that
// earlier kernels of the call wrote to the workspace.
//
// Order.  Fresh pages are the free pages in ascending order, dealt to the
// entries in order; the k-th hole takes the k-th live page behind the live
// count.  Both are ranks from prefix sums over the reference counts, so the
// result does not depend on the order in which blocks run.  Reference counts
// change by atomic adds, which commute.
//
// Steps, each a launch that the next one's set-up overlaps:
//   count   free pages of every chunk of kChunk pages
//   plan    one block: prefix sum over the chunks; for a fork also the checks
//           of every entry, the pages it needs and their prefix sum
//   assign  chunks deal their free pages by rank (fork), or list holes and
//           pages to move by rank (compact)
//   rename  tables and counts follow (compact)
//   move    a block per entry shares the parent's pages (fork); page contents
// A small pool's call is bound by its launches (2 us each on the GPU, 3 on the
// host), so there one block does everything but the move, two launches instead
// of four or five.  What bounds that block are the counts it reads, up to eight
// a thread, and for a compaction the rows, a warp each.  Graph replays without
// caches, one block against several:
//   fork, children sharing whole rows    entries x pages a row   us
//     pool of 2000                       8 x 1023        7.6     11.5
//                                        190 x 127       9.5     14.1
//     pool of 8192                       8 x 255        10.0     11.7
//                                        250 x 63       12.7     13.8
//                                        1000 x 31      16.5     16.9
//     pool of 16384                      8 x 4095       15.9     14.9
//                                        128 x 255      19.8     13.4
//   compaction                           sequences x pages a row
//     pool of 2000                       8 x 1023        5.5     10.3
//                                        64 x 127        6.1      7.5
//                                        160 x 127       9.3      7.7
//                                        256 x 31        9.4      8.1
//     pool of 4096                       64 x 127        6.4      7.9
//     pool of 8192                       8 x 255         8.5      8.6
//                                        64 x 127       10.6      7.8
// so the limits are 8192 pages and 1024 entries, 4096 pages and 128 sequences.
//
// Bound: launches, and for large pools the copies, which read and write every
// moved byte once.  Measured in graph replays, with the call that frees pages
// and a reset of the books before each: 3 freed, 4 forked and 4 grown over 512
// pages of 28 KB 11.1 us; 60, 150 and 40 over 2000 pages in 64 arrays (134 MB
// moved, 20 us at a copy's rate) 31.6 us; 512 pages compacted 9.1 us, 2500 in
// 64 arrays (557 MB, 83 us) 107.3 us.
#include <cuda_runtime.h>

#include "tq_device.cuh"

namespace tq {

int sm_count();

namespace {

constexpr int kChunk = 1024;          // pages per block of count and assign
constexpr int kThreads = 256;
constexpr int kPlanThreads = 1024;
// what one block takes: pages of the pool (8 or 4 a thread), entries of a fork, sequences of a compacted pool
constexpr int kForkPages = 8192, kForkEntries = 1024;
constexpr int kPackPages = 4096, kPackSeqs = 128;
constexpr int kAhead = 8;             // table entries whose loads a thread has in flight
constexpr int kMaxArrays = 128;       // cache arrays one move launch takes
constexpr int kPiece = 16384;         // bytes one block copies at a time: four 16-byte loads in flight a thread
constexpr int kMaxPerSeq = 1 << 20;   // pages of a sequence: kPlanThreads of them sum below 2^31
constexpr int kMaxPages = 1 << 28;    // pages of a pool
constexpr int kManyPages = 1 << 29;   // more than any pool has

// Workspace header, then the arrays of Work.
struct Head {
  int32_t ok;        // 0: the plan was refused, nothing changes
  int32_t need;      // fresh pages the entries take together
  int32_t n_live;    // compact: pages in use
  int32_t moves;     // page copies
};

struct Work {
  Head* head;
  int32_t* chunk;    // [chunks] free pages of each chunk, then before each
  int32_t* mark;     // [n_seqs] 1: a child of this call
  int32_t* off;      // [n + 1] fresh pages before entry i
  int32_t* first;    // [n] first table index a fresh page goes to, behind the shared ones replaced
  int32_t* cow;      // [n] shared pages that fresh ones replace
  int32_t* src;      // [n] or [num_pages]: page copied
  int32_t* dst;      // [n] or [num_pages]: page it is copied to
  int32_t* rank;     // [num_pages] compact: rank of a page that moves.  fork: for a fresh page, by rank, that
                     // replaces a shared one the table index, then (from deal on) the page replaced
};

size_t carve(void* ws, int n_seqs, int num_pages, int n, Work* w) {
  uint8_t* p = static_cast<uint8_t*>(ws);
  size_t at = 0;
  auto take = [&](size_t count) {
    int32_t* r = reinterpret_cast<int32_t*>(p + at);
    at += (count * 4 + 255) / 256 * 256;
    return r;
  };
  const int chunks = (num_pages + kChunk - 1) / kChunk;
  const size_t lists = n > num_pages ? n : num_pages;
  Work t;
  t.head = reinterpret_cast<Head*>(take(sizeof(Head) / 4));
  t.chunk = take(chunks + 1);
  t.mark = take(n_seqs);
  t.off = take((size_t)n + 1);
  t.first = take(n);
  t.cow = take(n);
  t.src = take(lists);
  t.dst = take(lists);
  t.rank = take(num_pages);
  if (w) *w = t;
  return at;
}

// Sum of v over the block, and the sum of the threads before this one.
// Every thread calls it; s_part holds blockDim.x / 32 + 1 values.
__device__ __forceinline__ int block_scan(int v, int* s_part, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();   // the part sums of an earlier call have been read
  if (lane == 31) s_part[w] = x;
  __syncthreads();
  if (w == 0) {
    int p = lane < nw ? s_part[lane] : 0;
    const int own = p;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kFull, p, o);
      if (lane >= o) p += y;
    }
    if (lane < nw) s_part[lane] = p - own;
    if (lane == 31) s_part[32] = p;
  }
  __syncthreads();
  *total = s_part[32];
  return s_part[w] + x - v;
}

// Kernels of one call in a row: a kernel may start when the one before it
// has, and waits here until that one has ended and its writes are visible.
__device__ __forceinline__ void chain_begin() {
  asm volatile("griddepcontrol.launch_dependents;\ngriddepcontrol.wait;\n" ::: "memory");
}

__device__ __forceinline__ int free_at(const int32_t* ref, int p, int n) { return p < n && ref[p] == 0 ? 1 : 0; }

__global__ void __launch_bounds__(kThreads) pages_count_kernel(const int32_t* __restrict__ ref, int num_pages, Work w) {
  chain_begin();
  __shared__ int s_part[33];
  int c = 0;
  for (int i = threadIdx.x; i < kChunk; i += kThreads) c += free_at(ref, blockIdx.x * kChunk + i, num_pages);
  int total;
  block_scan(c, s_part, &total);
  if (threadIdx.x == 0) w.chunk[blockIdx.x] = total;
}

// Exclusive prefix sum of w.chunk in place; returns the total.
__device__ int scan_chunks(Work w, int chunks, int* s_part) {
  int base = 0;
  for (int c0 = 0; c0 < chunks; c0 += kPlanThreads) {
    const int c = c0 + threadIdx.x;
    const int v = c < chunks ? w.chunk[c] : 0;
    int total;
    const int before = block_scan(v, s_part, &total);
    if (c < chunks) w.chunk[c] = base + before;
    base += total;
  }
  return base;
}

struct ForkArgs {
  tq_page_pool pool;
  const int32_t* parent;
  const int32_t* child;
  const int32_t* share_len;
  const int32_t* new_len;
  int32_t* result;
  int n;
  Work w;
};

// What entry i of a fork takes, but for the shared pages in [at, last) of its
// own row that it replaces.  ok: the entry can be done.
struct Entry {
  int parent, child, at, last, first, fresh, total, src;
  bool ok;
};

__device__ __forceinline__ bool held_by_others(const tq_page_pool& p, int page) {
  return page >= 0 && page < p.num_pages && p.ref[page] > 1;
}

__device__ Entry read_entry(const ForkArgs& a, int i) {
  Entry e{};
  const tq_page_pool& p = a.pool;
  e.parent = a.parent[i];
  e.child = a.child[i];
  e.src = -1;
  const int share = a.share_len[i], len = a.new_len[i];
  e.ok = e.child >= 0 && e.child < p.n_seqs && e.parent >= -1 && e.parent < p.n_seqs && share >= 0 && len >= share;
  if (!e.ok) return e;
  const bool grow = e.parent == e.child;
  const int held = e.parent >= 0 ? p.n_pages[e.parent] : 0;
  const int64_t total = ((int64_t)len + p.page_size - 1) / p.page_size;
  e.ok = held >= 0 && held <= p.pages_per_seq && total <= p.pages_per_seq && (int64_t)held * p.page_size >= share &&
         (grow || p.n_pages[e.child] == 0);
  if (!e.ok) return e;
  e.total = (int)total;
  e.at = share / p.page_size;          // the page that is written next
  const int part = share % p.page_size;
  const int32_t* row = e.parent >= 0 ? p.page_table + (int64_t)e.parent * p.pages_per_seq : nullptr;
  if (grow) {
    e.first = held;
    e.fresh = e.total > held ? e.total - held : 0;
    // the held pages that tokens [share, len) go to: shared ones would be written
    e.last = min(held, max(e.total, e.at + 1));
    if (part && e.at < held && held_by_others(p, row[e.at])) e.src = row[e.at];
    if (e.total < held) e.total = held;
  } else {
    e.first = e.at;
    e.fresh = e.total - e.at;
    if (part) e.src = row[e.at];
  }
  if (!grow && part && (e.src < 0 || e.src >= p.num_pages)) e.ok = false;   // a table entry that is no page
  return e;
}

// How many of the pages [j0, j1) of sequence s others hold too; with `list`
// their table indexes, ascending, go there.  Every lane asks for its own
// (nothing where j0 >= j1), one range after the other by the whole warp.
__device__ __forceinline__ int shared_pages(const tq_page_pool& p, int s, int j0, int j1, int32_t* list) {
  const int lane = threadIdx.x & 31;
  int n = 0;
  for (uint32_t todo = __ballot_sync(kFull, j0 < j1); todo; todo &= todo - 1) {
    const int l = __ffs(todo) - 1;
    const int32_t* row = p.page_table + (int64_t)__shfl_sync(kFull, s, l) * p.pages_per_seq;
    const int a = __shfl_sync(kFull, j0, l), b = __shfl_sync(kFull, j1, l);
    int32_t* to = reinterpret_cast<int32_t*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(list), l));
    int c = 0;
    for (int k = a; k < b; k += 32) {
      const bool found = k + lane < b && held_by_others(p, row[k + lane]);
      const uint32_t m = __ballot_sync(kFull, found);
      if (found && to) to[c + __popc(m & ((1u << lane) - 1))] = k + lane;
      c += __popc(m);
    }
    if (lane == l) n = c;
  }
  return n;
}

// Checks every entry and sums up what they need, given the free pages; takes
// the sequences' new page counts over when all is well (and returns that).
// One block of kPlanThreads.
__device__ bool plan_entries(const ForkArgs& a, int n_free, int* s_part) {
  const Work& w = a.w;
  const tq_page_pool& p = a.pool;
  for (int i = threadIdx.x; i < p.n_seqs; i += kPlanThreads) w.mark[i] = 0;
  __syncthreads();
  int bad = 0;
  for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
    const int c = a.child[i];
    if (c >= 0 && c < p.n_seqs && atomicExch(&w.mark[c], 1)) bad = 1;   // the same child twice
  }
  __syncthreads();
  int base = 0, copies = 0;
  for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
    const int i = i0 + threadIdx.x;
    Entry e{};
    e.ok = true;
    if (i < a.n) {
      e = read_entry(a, i);
      // a parent that changes in this call
      if (e.ok && e.parent >= 0 && e.parent != e.child && w.mark[e.parent]) e.ok = false;
      if (!e.ok) {
        bad = 1;
        e.fresh = 0;
      }
    }
    // most ranges are one page, which its own thread looks at
    int cow = e.ok && e.last == e.at + 1 && held_by_others(p, p.page_table[(int64_t)e.child * p.pages_per_seq + e.at]);
    const int many = shared_pages(p, e.child, e.at, e.ok && e.last > e.at + 1 ? e.last : e.at, nullptr);
    cow += many;
    int total;
    // an entry takes at most kMaxPerSeq pages, so a block's sum fits; the
    // running sum saturates above any pool, whose size is checked against it
    const int before = block_scan(e.fresh + cow, s_part, &total);
    if (i < a.n) {
      w.off[i] = min(base + before, kManyPages);
      w.first[i] = e.first;
      w.cow[i] = cow;
      w.src[i] = e.src;
      w.dst[i] = -1;
    }
    base = min(base + total, kManyPages);
    copies += i < a.n && e.ok && e.src >= 0 ? 1 : 0;
  }
  const int any_bad = __syncthreads_or(bad);
  int n_copies;
  block_scan(copies, s_part, &n_copies);
  const bool ok = !any_bad && base <= n_free;
  if (ok) {   // every count has been read: the sequences hold their new pages from here on
    for (int i0 = 0; i0 < a.n; i0 += kPlanThreads) {
      const int i = i0 + threadIdx.x;
      int c = 0, at = 0, last = 0;
      int32_t* list = nullptr;
      if (i < a.n) {
        c = a.child[i];
        const int held = p.n_pages[c];   // a sequence is one entry's child: this thread's to read and change
        const int total = (int)(((int64_t)a.new_len[i] + p.page_size - 1) / p.page_size);
        if (w.cow[i]) {
          at = a.share_len[i] / p.page_size;
          last = min(held, max(total, at + 1));
          list = w.rank + w.off[i];
        }
        if (a.parent[i] != c || total > held) p.n_pages[c] = total;
      }
      shared_pages(p, c, at, last, list);
    }
  }
  if (threadIdx.x == 0) {
    w.off[a.n] = base;
    w.head->ok = ok;
    w.head->need = base;
    w.head->moves = ok ? a.n : 0;
    if (a.result) {
      a.result[0] = any_bad ? -1 : (ok ? 0 : base - n_free);
      a.result[1] = ok ? base : 0;
      a.result[2] = ok ? n_copies : 0;
      a.result[3] = 0;
    }
  }
  __syncthreads();
  return ok;
}

// The r-th fresh page, `page`, goes to the entry whose pages hold rank r.
__device__ void deal(const ForkArgs& a, int r, int page) {
  const Work& w = a.w;
  int lo = 0, hi = a.n;   // the last entry with off <= r
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (w.off[mid] <= r) lo = mid; else hi = mid;
  }
  const int t = r - w.off[lo], cow = w.cow[lo];
  int32_t* row = a.pool.page_table + (int64_t)a.child[lo] * a.pool.pages_per_seq;
  if (t < cow) {   // in a shared page's place, whose count falls once no count is read any more
    const int idx = w.rank[r];
    w.rank[r] = row[idx];
    row[idx] = page;
  } else {
    row[w.first[lo] + t - cow] = page;
  }
  a.pool.ref[page] = 1;
  if (t == 0) w.dst[lo] = page;   // the copy of a part-filled page goes to the first fresh page
}

// Entry i shares its parent's full pages (its first, which no entry of the
// call changes), and the shared pages that it replaced lose it as a holder;
// by one block.
__device__ void share(const ForkArgs& a, int i) {
  const tq_page_pool& p = a.pool;
  const int parent = a.parent[i], child = a.child[i], cow = a.w.cow[i];
  for (int t = threadIdx.x; t < cow; t += kThreads) atomicSub(&p.ref[a.w.rank[a.w.off[i] + t]], 1);
  if (parent < 0 || parent == child) return;
  const int full = a.w.first[i];
  const int32_t* from = p.page_table + (int64_t)parent * p.pages_per_seq;
  int32_t* to = p.page_table + (int64_t)child * p.pages_per_seq;
  for (int k = threadIdx.x; k < full; k += kAhead * kThreads) {
    int page[kAhead];
#pragma unroll
    for (int u = 0; u < kAhead; ++u) page[u] = k + u * kThreads < full ? from[k + u * kThreads] : 0;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (k + u * kThreads >= full) break;
      to[k + u * kThreads] = page[u];
      if (page[u] >= 0 && page[u] < p.num_pages) atomicAdd(&p.ref[page[u]], 1);
    }
  }
}

__global__ void __launch_bounds__(kPlanThreads) pages_fork_plan_kernel(const ForkArgs a, int chunks) {
  chain_begin();
  __shared__ int s_part[33];
  plan_entries(a, scan_chunks(a.w, chunks, s_part), s_part);
}

// A small pool's fork: count, plan and assign in one block, a thread taking
// `per` consecutive pages.
__global__ void __launch_bounds__(kPlanThreads) pages_fork_small_kernel(const ForkArgs a, int per) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");   // first of its call: nothing to wait for
  __shared__ int s_part[33];
  const int p0 = threadIdx.x * per, p1 = min(p0 + per, a.pool.num_pages);
  int c = 0, n_free;
  uint32_t free_bits = 0;   // per <= 8
  for (int p = p0; p < p1; ++p) {
    const int f = a.pool.ref[p] == 0 ? 1 : 0;
    c += f;
    free_bits |= (uint32_t)f << (p - p0);
  }
  int r = block_scan(c, s_part, &n_free);
  if (!plan_entries(a, n_free, s_part)) return;
  const int need = a.w.off[a.n];
  for (; free_bits && r < need; ++r, free_bits &= free_bits - 1) deal(a, r, p0 + __ffs(free_bits) - 1);
}

// A block deals a chunk's free pages.
__global__ void __launch_bounds__(kThreads) pages_fork_assign_kernel(const ForkArgs a) {
  chain_begin();
  __shared__ int s_part[33];
  const Work w = a.w;
  const tq_page_pool& p = a.pool;
  if (!w.head->ok) return;
  const int need = w.head->need;
  const int base = w.chunk[blockIdx.x];
  if (base >= need) return;
  constexpr int PER = kChunk / kThreads;
  const int p0 = blockIdx.x * kChunk + threadIdx.x * PER;
  int f[PER], c = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) c += f[k] = free_at(p.ref, p0 + k, p.num_pages);
  int total;
  int r = base + block_scan(c, s_part, &total);
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    if (!f[k]) continue;
    if (r >= need) break;
    deal(a, r++, p0 + k);
  }
}

// The caches' arrays as runs of bytes per page.
struct Arrays {
  uint8_t* base[kMaxArrays];
  int32_t bytes[kMaxArrays];    // per page
  int32_t piece0[kMaxArrays];   // pieces of a page before this array
  int32_t n, pieces;            // arrays, pieces of a whole page
};

// Copies w.moves pages src[r] -> dst[r] (an entry of a fork without a copy
// has src -1), one piece of one array per block and step.  Before that the
// blocks do what is left of a fork's f.n entries (0: nothing), whose pages have
// all been dealt: the counts that tell the free ones are not read any more.
__global__ void __launch_bounds__(kThreads) pages_move_kernel(const ForkArgs f, const __grid_constant__ Arrays a) {
  chain_begin();
  const Work& w = f.w;
  const int moves = w.head->moves, num_pages = f.pool.num_pages;
  if (moves)
    for (int i = blockIdx.x; i < f.n; i += gridDim.x) share(f, i);
  const int64_t items = (int64_t)moves * a.pieces;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int r = (int)(it / a.pieces), pc = (int)(it - (int64_t)r * a.pieces);
    const int src = w.src[r];
    if (src < 0) continue;
    const int dst = w.dst[r];
    if (src >= num_pages || dst < 0 || dst >= num_pages) continue;
    int lo = 0, hi = a.n;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.piece0[mid] <= pc) lo = mid; else hi = mid;
    }
    const int64_t bytes = a.bytes[lo];
    const int64_t at = (int64_t)(pc - a.piece0[lo]) * kPiece;
    const int n16 = (int)(imin64(kPiece, bytes - at) / 16);
    const uint4* s = reinterpret_cast<const uint4*>(a.base[lo] + src * bytes + at);
    uint4* d = reinterpret_cast<uint4*>(a.base[lo] + dst * bytes + at);
    constexpr int U = kPiece / 16 / kThreads;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (threadIdx.x + u * kThreads < n16) v[u] = __ldcs(s + threadIdx.x + u * kThreads);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (threadIdx.x + u * kThreads < n16) d[threadIdx.x + u * kThreads] = v[u];
  }
}

struct CompactArgs {
  tq_page_pool pool;
  int32_t* result;
  Work w;
};

__global__ void __launch_bounds__(kPlanThreads) pages_compact_plan_kernel(const CompactArgs a, int chunks) {
  chain_begin();
  __shared__ int s_part[33];
  const int n_free = scan_chunks(a.w, chunks, s_part);
  const int n_live = a.pool.num_pages - n_free;
  __syncthreads();
  // holes: free pages before n_live
  const int c = n_live / kChunk;
  int part = 0;
  for (int i = threadIdx.x; i < n_live - c * kChunk; i += kPlanThreads) part += a.pool.ref[c * kChunk + i] == 0 ? 1 : 0;
  int holes;
  block_scan(part, s_part, &holes);
  if (threadIdx.x == 0) {
    holes += c < chunks ? a.w.chunk[c] : n_free;
    a.w.head->ok = 1;
    a.w.head->n_live = n_live;
    a.w.head->moves = holes;
    if (a.result) {
      a.result[0] = 0;
      a.result[1] = n_live;
      a.result[2] = holes;
      a.result[3] = 0;
    }
  }
}

// Tables and counts after the lists are there: `lanes` threads (a warp per
// sequence) rename the pages, and the counts move with the pages.
__device__ void rename(const CompactArgs& a, int n_live, int moves, int64_t tid, int64_t step) {
  const Work& w = a.w;
  const tq_page_pool& p = a.pool;
  for (int64_t r = tid; r < moves; r += step) {
    p.ref[w.dst[r]] = p.ref[w.src[r]];
    p.ref[w.src[r]] = 0;
  }
  const int lane = threadIdx.x & 31;
  for (int64_t s = tid / 32; s < p.n_seqs; s += step / 32) {
    int32_t* row = p.page_table + s * p.pages_per_seq;
    const int held = min(p.n_pages[s], p.pages_per_seq);
    for (int j = lane; j < held; j += kAhead * 32) {
      int x[kAhead];   // the entry's page, its rank (-1: none, or a free page, which no table should name), its new page
#pragma unroll
      for (int u = 0; u < kAhead; ++u) x[u] = j + u * 32 < held ? row[j + u * 32] : -1;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) x[u] = x[u] >= n_live && x[u] < p.num_pages ? w.rank[x[u]] : -1;
#pragma unroll
      for (int u = 0; u < kAhead; ++u) x[u] = x[u] >= 0 ? w.dst[x[u]] : -1;
#pragma unroll
      for (int u = 0; u < kAhead; ++u)
        if (x[u] >= 0) row[j + u * 32] = x[u];
    }
  }
}

// Page `page` in the lists of holes before n_live and of pages to move, by
// rank; `before`: the free pages before it.
__device__ void list_page(const Work& w, int page, bool is_free, int before, int n_live, int moves) {
  if (is_free) {
    if (page >= n_live) w.rank[page] = -1;
    else if (before < moves) w.dst[before] = page;
  } else if (page >= n_live) {
    const int r = page - before - (n_live - moves);   // live pages before it, less those before n_live
    if (r >= 0 && r < moves) {
      w.src[r] = page;
      w.rank[page] = r;
    }
  }
}

// A small pool's compaction but for the copies, in one block.
__global__ void __launch_bounds__(kPlanThreads) pages_compact_small_kernel(const CompactArgs a, int per) {
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");   // first of its call: nothing to wait for
  __shared__ int s_part[33];
  const int n = a.pool.num_pages, p0 = min(threadIdx.x * per, n), p1 = min(p0 + per, n);
  int c = 0, n_free, moves;
  uint32_t free_bits = 0;   // per <= 8
  for (int p = p0; p < p1; ++p) {
    const int f = a.pool.ref[p] == 0 ? 1 : 0;
    c += f;
    free_bits |= (uint32_t)f << (p - p0);
  }
  int before = block_scan(c, s_part, &n_free);
  const int n_live = n - n_free, in = min(max(n_live - p0, 0), 31);
  block_scan(__popc(free_bits & ((1u << in) - 1)), s_part, &moves);   // holes
  for (int p = p0; p < p1; ++p) {
    const bool f = (free_bits >> (p - p0)) & 1u;
    list_page(a.w, p, f, before, n_live, moves);
    before += f;
  }
  if (threadIdx.x == 0) {
    a.w.head->ok = 1;
    a.w.head->n_live = n_live;
    a.w.head->moves = moves;
    if (a.result) {
      a.result[0] = 0;
      a.result[1] = n_live;
      a.result[2] = moves;
      a.result[3] = 0;
    }
  }
  __syncthreads();
  if (moves) rename(a, n_live, moves, threadIdx.x, kPlanThreads);
}

// Lists the holes before n_live and the live pages behind it, by rank.
__global__ void __launch_bounds__(kThreads) pages_compact_list_kernel(const CompactArgs a) {
  chain_begin();
  __shared__ int s_part[33];
  const Work w = a.w;
  const int n_live = w.head->n_live, moves = w.head->moves;
  if (!moves) return;
  constexpr int PER = kChunk / kThreads;
  const int p0 = blockIdx.x * kChunk + threadIdx.x * PER;
  int f[PER], c = 0;
#pragma unroll
  for (int k = 0; k < PER; ++k) c += f[k] = free_at(a.pool.ref, p0 + k, a.pool.num_pages);
  int total;
  int before = w.chunk[blockIdx.x] + block_scan(c, s_part, &total);   // free pages before p0
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    if (p0 + k >= a.pool.num_pages) break;
    list_page(w, p0 + k, f[k] != 0, before, n_live, moves);
    before += f[k];
  }
}

__global__ void __launch_bounds__(kThreads) pages_compact_rename_kernel(const CompactArgs a) {
  chain_begin();
  const int moves = a.w.head->moves;
  if (moves)
    rename(a, a.w.head->n_live, moves, (int64_t)blockIdx.x * kThreads + threadIdx.x, (int64_t)gridDim.x * kThreads);
}

// A block per sequence named.
__global__ void __launch_bounds__(kThreads) pages_free_kernel(const tq_page_pool p, const int32_t* __restrict__ seqs,
                                                              const int32_t* __restrict__ keep_len) {
  __shared__ int s_old, s_keep;
  const int s = seqs[blockIdx.x];
  if (s < 0 || s >= p.n_seqs) return;
  if (threadIdx.x == 0) {
    const int len = keep_len ? max(keep_len[blockIdx.x], 0) : 0;
    const int keep = (int)imin64(((int64_t)len + p.page_size - 1) / p.page_size, p.pages_per_seq);
    // the smaller of two entries for one sequence counts: each gives up what
    // it finds above its own
    s_old = min(atomicMin(&p.n_pages[s], keep), p.pages_per_seq);
    s_keep = keep;
  }
  __syncthreads();
  const int32_t* row = p.page_table + (int64_t)s * p.pages_per_seq;
  for (int j = s_keep + threadIdx.x; j < s_old; j += kThreads) {
    const int page = row[j];
    if (page >= 0 && page < p.num_pages) atomicSub(&p.ref[page], 1);
  }
}

// Launches a kernel of a call; chained: its set-up overlaps the kernel before
// it, which it waits for itself (chain_begin).
template <class... P, class... A>
bool launch(void (*kern)(P...), int64_t blocks, int threads, bool chained, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = chained ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess;
}

int check_pool(const tq_page_pool* p) {
  if (!p || !p->page_table || !p->n_pages || !p->ref) return TQ_ERR_ARG;
  if (p->n_seqs <= 0 || p->pages_per_seq <= 0 || p->num_pages <= 0) return TQ_ERR_ARG;
  if (p->page_size <= 0 || p->page_size % 32) return TQ_ERR_ARG;
  if (p->pages_per_seq > kMaxPerSeq || p->num_pages > kMaxPages || p->n_seqs > kMaxPages) return TQ_ERR_UNSUPPORTED;
  return TQ_OK;
}

int check_caches(const tq_kv_view* caches, int n_caches, int Hkv, int page_size) {
  if (n_caches < 0 || (n_caches && (!caches || Hkv <= 0))) return TQ_ERR_ARG;
  for (int i = 0; i < n_caches; ++i) {
    const tq_kv_view& c = caches[i];
    const int st = check_layout(&c.layout);
    if (st != TQ_OK) return st;
    if (!c.codes || !c.scales || (c.layout.qjl_m && (!c.qjl_bits || !c.qjl_rnorm))) return TQ_ERR_ARG;
    if (!aligned16(c.codes) || !aligned16(c.scales) ||
        (c.layout.qjl_m && (!aligned16(c.qjl_bits) || !aligned16(c.qjl_rnorm))))
      return TQ_ERR_ALIGN;
    if ((int64_t)Hkv * page_size * c.layout.head_dim > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
  }
  return TQ_OK;
}

// f: a fork's entries, or none (n = 0) with the pool and the lists; at most
// `most` pages are copied.
int launch_moves(const tq_kv_view* caches, int n_caches, int Hkv, ForkArgs f, int64_t most, cudaStream_t st) {
  const tq_page_pool& p = f.pool;
  Arrays a{};
  bool launched = false, ok = true;
  auto flush = [&]() {
    const int64_t items = most * a.pieces > f.n ? most * a.pieces : f.n;
    const int64_t most_blocks = 8 * sm_count(), grid = items < 1 ? 1 : (items > most_blocks ? most_blocks : items);
    ok = ok && launch(pages_move_kernel, grid, kThreads, true, st, f, a);
    launched = true;
    f.n = 0;   // the first launch has done the entries
    a.n = a.pieces = 0;
  };
  auto add = [&](const void* base, int64_t bytes) {
    a.base[a.n] = static_cast<uint8_t*>(const_cast<void*>(base));
    a.bytes[a.n] = (int32_t)bytes;
    a.piece0[a.n] = a.pieces;
    a.pieces += (int32_t)((bytes + kPiece - 1) / kPiece);
    ++a.n;
  };
  for (int i = 0; i < n_caches; ++i) {
    const tq_kv_view& c = caches[i];
    const int64_t rows = (int64_t)Hkv * p.page_size;
    if (a.n + 4 > kMaxArrays) flush();
    add(c.codes, rows * c.layout.head_dim * c.layout.bits / 8);
    add(c.scales, rows * (c.layout.head_dim / c.layout.block) * 2);
    if (c.layout.qjl_m) {
      add(c.qjl_bits, rows * c.layout.qjl_m / 8);
      add(c.qjl_rnorm, rows * 2);
    }
  }
  if (a.n || (!launched && f.n)) flush();
  return ok && cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

}  // namespace
}  // namespace tq

extern "C" int tq_pages_workspace_bytes(int n_seqs, int num_pages, int n, size_t* bytes) {
  if (n_seqs <= 0 || num_pages <= 0 || n < 0 || !bytes) return TQ_ERR_ARG;
  *bytes = tq::carve(nullptr, n_seqs, num_pages, n, nullptr);
  return TQ_OK;
}

extern "C" int tq_pages_fork(const tq_page_pool* pool, const tq_kv_view* caches, int n_caches, int Hkv,
                             const int32_t* parent, const int32_t* child, const int32_t* share_len,
                             const int32_t* new_len, int n, int32_t* result, void* workspace, size_t workspace_bytes,
                             void* stream) {
  int st = tq::check_pool(pool);
  if (st != TQ_OK) return st;
  st = tq::check_caches(caches, n_caches, Hkv, pool->page_size);
  if (st != TQ_OK) return st;
  if (n < 0 || n > pool->n_seqs) return TQ_ERR_ARG;   // more entries than sequences: a child would be named twice
  if (n && (!parent || !child || !share_len || !new_len)) return TQ_ERR_ARG;
  tq::Work w;
  if (!workspace || workspace_bytes < tq::carve(nullptr, pool->n_seqs, pool->num_pages, n, nullptr))
    return TQ_ERR_WORKSPACE;
  if (!tq::aligned16(workspace)) return TQ_ERR_ALIGN;
  tq::carve(workspace, pool->n_seqs, pool->num_pages, n, &w);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const tq::ForkArgs a{*pool, parent, child, share_len, new_len, result, n, w};
  const int chunks = (pool->num_pages + tq::kChunk - 1) / tq::kChunk;
  bool ok;
  if (pool->num_pages <= tq::kForkPages && n <= tq::kForkEntries) {
    const int per = (pool->num_pages + tq::kPlanThreads - 1) / tq::kPlanThreads;
    ok = tq::launch(tq::pages_fork_small_kernel, 1, tq::kPlanThreads, false, s, a, per);
  } else {
    ok = tq::launch(tq::pages_count_kernel, chunks, tq::kThreads, false, s, pool->ref, pool->num_pages, w) &&
         tq::launch(tq::pages_fork_plan_kernel, 1, tq::kPlanThreads, true, s, a, chunks) &&
         (!n || tq::launch(tq::pages_fork_assign_kernel, chunks, tq::kThreads, true, s, a));
  }
  if (!ok) return TQ_ERR_CUDA;
  if (n) return tq::launch_moves(caches, n_caches, Hkv, a, n, s);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

extern "C" int tq_pages_free(const tq_page_pool* pool, const int32_t* seqs, const int32_t* keep_len, int n,
                             void* stream) {
  const int st = tq::check_pool(pool);
  if (st != TQ_OK) return st;
  if (n < 0 || (n && !seqs)) return TQ_ERR_ARG;
  if (!n) return TQ_OK;
  tq::pages_free_kernel<<<n, tq::kThreads, 0, static_cast<cudaStream_t>(stream)>>>(*pool, seqs, keep_len);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

extern "C" int tq_pages_compact(const tq_page_pool* pool, const tq_kv_view* caches, int n_caches, int Hkv,
                                int32_t* result, void* workspace, size_t workspace_bytes, void* stream) {
  int st = tq::check_pool(pool);
  if (st != TQ_OK) return st;
  st = tq::check_caches(caches, n_caches, Hkv, pool->page_size);
  if (st != TQ_OK) return st;
  tq::Work w;
  if (!workspace || workspace_bytes < tq::carve(nullptr, pool->n_seqs, pool->num_pages, 0, nullptr))
    return TQ_ERR_WORKSPACE;
  if (!tq::aligned16(workspace)) return TQ_ERR_ALIGN;
  tq::carve(workspace, pool->n_seqs, pool->num_pages, 0, &w);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const tq::CompactArgs a{*pool, result, w};
  const int chunks = (pool->num_pages + tq::kChunk - 1) / tq::kChunk;
  bool ok;
  if (pool->num_pages <= tq::kPackPages && pool->n_seqs <= tq::kPackSeqs) {
    const int per = (pool->num_pages + tq::kPlanThreads - 1) / tq::kPlanThreads;
    ok = tq::launch(tq::pages_compact_small_kernel, 1, tq::kPlanThreads, false, s, a, per);
  } else {
    const int64_t work = pool->num_pages > (int64_t)pool->n_seqs * 32 ? pool->num_pages : (int64_t)pool->n_seqs * 32;
    const int64_t all = (work + tq::kThreads - 1) / tq::kThreads, most = 8 * tq::sm_count();
    const int64_t blocks = all > most ? most : all;
    ok = tq::launch(tq::pages_count_kernel, chunks, tq::kThreads, false, s, pool->ref, pool->num_pages, w) &&
         tq::launch(tq::pages_compact_plan_kernel, 1, tq::kPlanThreads, true, s, a, chunks) &&
         tq::launch(tq::pages_compact_list_kernel, chunks, tq::kThreads, true, s, a) &&
         tq::launch(tq::pages_compact_rename_kernel, blocks, tq::kThreads, true, s, a);
  }
  if (!ok) return TQ_ERR_CUDA;
  tq::ForkArgs none{};
  none.pool = *pool;
  none.w = w;
  return tq::launch_moves(caches, n_caches, Hkv, none, pool->num_pages / 2 + 1, s);
}
