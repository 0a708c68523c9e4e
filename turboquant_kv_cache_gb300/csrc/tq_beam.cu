// A beam search's step: of every beam's continuations by every token of the
// vocabulary, the n_out best of each request.
//
// Candidate (w, v) of a request has the score  s_w + (x_wv - lse_w),  with
// lse_w = m + log sum_v exp(x_wv - m), m = max_v x_wv.  Within a row the order
// of the scores is the order of the logits, so the rows need not be
// normalised to be cut down:
//   chunk   one CTA per part of a row, whose logits it reads once, into
//           registers: their maximum, the sum of exp(x - maximum), and the
//           part's n_out largest logits;
//   pick    one CTA per request: lse of every row from its parts, and the
//           n_out best of all parts' candidates.
//
// The largest M of many values, without sorting them: the M-th largest T of
// the threads' own maxima is a bound, since M values are at least T; few others
// are.  What is above T goes to a list, of those equal to T the ones that come
// first fill it up, and a candidate's rank is the number of list entries before
// it.  Equal scores go by place (w V + v, see second_key), so the result does
// not depend on the order in which threads reach the list.
//
// Precision: exp and the parts' sums in 32 bits, log and scores in 64, so that
// the order of two candidates of different rows follows from their scores to
// 1e-7 and the order in one row is exact; a score is rounded once.
// Infinities: a NaN logit counts as -inf and +inf as the largest finite
// number, so a row without any finite logit gives scores of -inf and no NaN.
//
// Bound: HBM for large vocabularies and batches (a logit is read once), the
// latency of two launches for small ones.
#include <cuda_runtime.h>
#include <math.h>

#include "tq_launch.cuh"

namespace tq {

int sm_count();

namespace {

constexpr int kMaxBeams = 64;      // beams of a request, and candidates kept
constexpr int kChunkThreads = 128;
constexpr int kPickThreads = 256;
constexpr int kListCap = 1024;     // chunk: entries above the bound, and kSameMost a thread equal to it
constexpr int kPickCap = 2048;     // pick: entries above the bound
constexpr int kSameMost = 8;       // entries equal to the bound a thread lists
constexpr float kMost = 3.402823466e38f;

struct BeamArgs {
  const void* logits;
  int64_t row_stride;
  const float* scores;       // [B][W] or NULL: 0
  const uint8_t* done;       // [B][W] or NULL
  int64_t eos;
  int32_t B, W, V, n_out, S, keep;
  float2* part;              // [B W][S] maximum, sum
  uint64_t* cand;            // [B W][S][n_out] keys, descending; 0: none
  float* out_scores;
  int32_t* out_parent;
  int32_t* out_token;
  uint8_t* out_done;
};

// A key that orders by value, then by the lower index; never 0 for a logit.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);   // -0 is 0
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
__device__ __forceinline__ uint64_t key_of(float x, int index) {
  return ((uint64_t)ordered(x) << 32) | (uint32_t)~index;
}
__device__ __forceinline__ uint64_t ordered64(double x) {
  const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
  return u ^ ((u >> 63) ? ~0ull : 1ull << 63);
}
__device__ __forceinline__ double unordered64(uint64_t u) {
  return __longlong_as_double((long long)(u ^ ((u >> 63) ? 1ull << 63 : ~0ull)));
}

// A beam's score with NaN as -inf and +inf as the largest finite number.
__device__ __forceinline__ float beam_score(const BeamArgs& a, int64_t row) {
  return a.scores ? fminf(fmaxf(a.scores[row], -INFINITY), kMost) : 0.f;
}
__device__ __forceinline__ bool beam_done(const BeamArgs& a, int64_t row) { return a.done && a.done[row]; }

// Vectors of 16 bytes as logits.
template <bool F32>
struct Vec {
  static constexpr int N = F32 ? 4 : 8;
  uint4 raw;
  __device__ __forceinline__ float at(int e) const {
    const uint32_t w = F32 ? (&raw.x)[e] : (&raw.x)[e >> 1];
    float x;
    if (F32) x = __uint_as_float(w);
    else x = h2f((uint16_t)((e & 1) ? w >> 16 : w & 0xffffu));
    return fminf(fmaxf(x, -INFINITY), kMost);
  }
  // The raw words are what is kept: the next pass converts them again, where
  // the compiler would hold the converted ones in twice the registers.
  __device__ __forceinline__ void keep_raw() { asm volatile("" : "+r"(raw.x), "+r"(raw.y), "+r"(raw.z), "+r"(raw.w)); }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Part `s` of a row that is not read: all logits -inf, or of a finished beam 0
// at eos and -inf elsewhere.  Its first indexes fill the list.
template <int PER>
__device__ void synthetic_part(const BeamArgs& a, int64_t list, int s, int lead, bool at_eos) {
  const int lo = max(s * PER - lead, 0), hi = (int)imin64((int64_t)(s + 1) * PER - lead, a.V);
  const bool has = at_eos && a.eos >= lo && a.eos < hi;
  for (int r = threadIdx.x; r < a.n_out; r += blockDim.x) {
    uint64_t key = 0;
    if (has && r == 0) {
      key = key_of(0.f, (int)a.eos);
    } else {
      int i = lo + r - (has ? 1 : 0);
      if (has && i >= a.eos) ++i;
      if (i < hi) key = key_of(-INFINITY, i);
    }
    a.cand[list * a.n_out + r] = key;
  }
}

template <bool F32, int NV>
__global__ void __launch_bounds__(kChunkThreads) beam_chunk_kernel(const BeamArgs a) {
  constexpr int VEC = Vec<F32>::N, PER = kChunkThreads * NV * VEC;   // logits of a part
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");   // first of its call: nothing to wait for
  __shared__ float s_max[kChunkThreads];
  __shared__ float s_red[2][kChunkThreads / 32];
  __shared__ float s_bound;
  __shared__ int s_above, s_equal, s_many;
  __shared__ uint64_t s_key[kListCap + kSameMost * kChunkThreads];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t list = blockIdx.x;
  const int64_t row = list / a.S;
  const int s = (int)(list - row * a.S);
  const int esz = F32 ? 4 : 2;
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + row * a.row_stride * esz;
  // vectors lie on 16-byte boundaries; the first of a row starts `lead` logits before it
  const int lead = (int)((reinterpret_cast<uintptr_t>(base) & 15u) / esz);
  const float score = beam_score(a, row);
  const bool done = beam_done(a, row);
  if (done || score == -INFINITY) {
    if (tid == 0) a.part[list] = make_float2(-INFINITY, 0.f);
    synthetic_part<PER>(a, list, s, lead, done && score != -INFINITY);
    return;
  }
  const int64_t v0 = (int64_t)s * (kChunkThreads * NV) + tid;
  Vec<F32> x[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int64_t i0 = (v0 + j * kChunkThreads) * VEC - lead;
    if (i0 >= 0 && i0 + VEC <= a.V) {
      x[j].raw = __ldcs(reinterpret_cast<const uint4*>(base + i0 * esz));
    } else {   // the row's first or last vector, or none
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = F32 ? 0xff800000u : 0xfc00fc00u;   // -inf
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        if (i0 + e < 0 || i0 + e >= a.V) continue;
        if (F32) {
          w[e] = reinterpret_cast<const uint32_t*>(base)[i0 + e];
        } else {
          const uint32_t h = reinterpret_cast<const uint16_t*>(base)[i0 + e];
          w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | (h << 16) : (w[e >> 1] & 0xffff0000u) | h;
        }
      }
      x[j].raw = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  float mine = -INFINITY;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) mine = fmaxf(mine, x[j].at(e));
  float m = mine;
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  s_max[tid] = mine;
  if (lane == 0) s_red[0][warp] = m;
  if (tid == 0) s_above = s_equal = s_many = 0;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kChunkThreads / 32; ++w) m = fmaxf(m, s_red[0][w]);
  const float mref = m == -INFINITY ? 0.f : m;
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    x[j].keep_raw();
#pragma unroll
    for (int e = 0; e < VEC; ++e) sum += ex2((x[j].at(e) - mref) * kLog2e);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (lane == 0) s_red[1][warp] = sum;
  // this thread's place among the maxima: one thread has M - 1 before it
  int before = 0;
#pragma unroll 8
  for (int u = 0; u < kChunkThreads; u += 4) {
    const float4 o = *reinterpret_cast<const float4*>(s_max + u);
    before += (o.x > mine || (o.x == mine && u < tid)) + (o.y > mine || (o.y == mine && u + 1 < tid)) +
              (o.z > mine || (o.z == mine && u + 2 < tid)) + (o.w > mine || (o.w == mine && u + 3 < tid));
  }
  if (before == a.n_out - 1) s_bound = mine;
  __syncthreads();
  const float bound = s_bound;
  if (mine >= bound && mine != -INFINITY) {
    int same = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j].keep_raw();
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float v = x[j].at(e);
        if (v < bound || v == -INFINITY) continue;   // -inf: also the places outside the row
        const int i = (int)((v0 + j * kChunkThreads) * VEC + e - lead);
        if (v > bound) {
          const int at = atomicAdd(&s_above, 1);
          if (at < kListCap) s_key[at] = key_of(v, i);
        } else if (++same <= kSameMost) {
          s_key[kListCap + atomicAdd(&s_equal, 1)] = key_of(v, i);
        } else {
          s_many = 1;
        }
      }
    }
  }
  __syncthreads();
  const int above = s_above;
  uint64_t* out = a.cand + list * a.n_out;
  if (tid == 0) {
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < kChunkThreads / 32; ++w) l += s_red[1][w];
    a.part[list] = make_float2(m, l);
  }
  if (above > kListCap) {
    // a few threads hold most of the large values: one after the other, each
    // the largest below the last.  There are more than n_out above the bound
    uint64_t last = ~0ull;
    for (int r = 0; r < a.n_out; ++r) {
      uint64_t best = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        x[j].keep_raw();
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float v = x[j].at(e);
          const uint64_t k = key_of(v, (int)((v0 + j * kChunkThreads) * VEC + e - lead));
          if (v > bound && k < last && k > best) best = k;
        }
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const uint64_t k = __shfl_xor_sync(kFull, best, o);
        best = k > best ? k : best;
      }
      __syncthreads();   // the last round's results have been read
      if (lane == 0) s_key[warp] = best;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kChunkThreads / 32; ++w) best = s_key[w] > best ? s_key[w] : best;
      if (tid == 0) out[r] = best;
      last = best;
    }
    return;
  }
  for (int i = tid; i < above; i += kChunkThreads) {
    const uint64_t k = s_key[i];
    int r = 0;
    for (int u = 0; u < above; ++u) r += s_key[u] > k;
    if (r < a.n_out) out[r] = k;
  }
  if (above >= a.n_out) return;
  if (bound != -INFINITY && !s_many) {
    const int equal = s_equal;   // with those above at least n_out
    for (int i = tid; i < equal; i += kChunkThreads) {
      const uint64_t k = s_key[kListCap + i];
      int r = above;
      for (int u = 0; u < equal; ++u) r += s_key[kListCap + u] > k;
      if (r < a.n_out) out[r] = k;
    }
  } else if (warp == 0) {
    // many logits are the bound itself (a mask's value, or -inf): the first of
    // them, which are among the part's first few then
    const int lo = max(s * PER - lead, 0), hi = (int)imin64((int64_t)(s + 1) * PER - lead, a.V);
    int r = above;
    for (int i0 = lo; i0 < hi && r < a.n_out; i0 += 64) {
      float v[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = i0 + 32 * u + lane;
        float f = NAN;
        if (i < hi) {
          f = F32 ? reinterpret_cast<const float*>(base)[i] : h2f(reinterpret_cast<const uint16_t*>(base)[i]);
          f = fminf(fmaxf(f, -INFINITY), kMost);
        }
        v[u] = f;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t found = __ballot_sync(kFull, v[u] == bound);
        const int at = r + __popc(found & ((1u << lane) - 1));
        if (((found >> lane) & 1u) && at < a.n_out) out[at] = key_of(bound, i0 + 32 * u + lane);
        r += __popc(found);
      }
    }
    for (r += lane; r < a.n_out; r += 32) out[r] = 0;   // a part of fewer logits
  }
}

// Exclusive prefix sum of v over the block; every thread calls it.
__device__ __forceinline__ int scan_block(int v, int* s_part, int* total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_part[w] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < kPickThreads / 32; ++i) {
    const int p = s_part[i];
    if (i < w) before += p;
    all += p;
  }
  *total = all;
  return before + x - v;
}

// What orders candidates of equal score: the lower beam, then the higher logit
// (two logits of a row can have one score, where the beam's own is so large
// that 64 bits do not tell them apart), then the lower token.  In 64 bits:
// 63 - beam, the ordered logit, and the token counted down.
constexpr uint64_t kTokenMask = (1ull << 26) - 1;
__device__ __forceinline__ uint64_t second_key(int w, uint32_t logit, uint32_t token) {
  return ((uint64_t)(kMaxBeams - 1 - w) << 58) | ((uint64_t)logit << 26) | (kTokenMask - token);
}
__device__ __forceinline__ int key_beam(uint64_t second) { return kMaxBeams - 1 - (int)(second >> 58); }
__device__ __forceinline__ int key_token(uint64_t second) { return (int)(kTokenMask - (second & kTokenMask)); }

__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(const BeamArgs a) {
  __shared__ double s_lse[kMaxBeams], s_base[kMaxBeams];
  __shared__ uint64_t s_max[kPickThreads];
  __shared__ uint64_t s_score[kPickCap], s_second[kPickCap];
  __shared__ uint64_t s_best[kMaxBeams], s_best2[kMaxBeams];
  __shared__ uint64_t s_bound;
  __shared__ int s_n, s_part[kPickThreads / 32];
  __shared__ uint8_t s_done[kMaxBeams];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x, M = a.n_out, lists = a.W * a.S;
  const int64_t row0 = (int64_t)b * a.W;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  for (int w = warp; w < a.W; w += kPickThreads / 32) {
    const float score = beam_score(a, row0 + w);
    const bool done = beam_done(a, row0 + w);
    double lse = 0.0;   // of a finished beam
    if (!done && score != -INFINITY) {
      const float2* p = a.part + (row0 + w) * a.S;
      float m = -INFINITY;
      for (int i = lane; i < a.S; i += 32) m = fmaxf(m, p[i].x);
#pragma unroll
      for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      double sum = 0.0;
      for (int i = lane; i < a.S; i += 32) {
        const float2 q = p[i];
        if (q.x != -INFINITY) sum += (double)(q.y * ex2((q.x - m) * kLog2e));
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      if (m != -INFINITY) lse = (double)m + log(sum);
    }
    if (lane == 0) {
      s_base[w] = (double)score;
      s_lse[w] = lse;
      s_done[w] = done;
    }
  }
  if (tid == 0) s_n = 0;
  __syncthreads();
  // score of entry r of list h (descending in r), as an ordered key; 0: none
  auto entry = [&](int h, int r, uint64_t* second) -> uint64_t {
    const uint64_t k = a.cand[(row0 * a.S + h) * M + r];
    if (!k) return 0;
    const int w = h / a.S;
    const float x = unordered((uint32_t)(k >> 32));
    *second = second_key(w, (uint32_t)(k >> 32), ~(uint32_t)k);
    const double base = s_base[w];
    return ordered64(x == -INFINITY || base == -INFINITY ? -INFINITY : base + ((double)x - s_lse[w]));
  };
  uint64_t mine = 0;
  uint64_t second;
  for (int h = tid; h < lists; h += kPickThreads) {
    const uint64_t k = entry(h, 0, &second);
    mine = k > mine ? k : mine;
  }
  s_max[tid] = mine;
  __syncthreads();
  int before = 0;
#pragma unroll 8
  for (int u = 0; u < kPickThreads; ++u) {
    const uint64_t o = s_max[u];
    before += o > mine || (o == mine && u < tid);
  }
  if (before == M - 1) s_bound = mine;
  __syncthreads();
  // a bound of 0 is that of a thread without a list: everything is above it
  const uint64_t bound = s_bound, nothing = ordered64(-INFINITY);
  // entries from `least` on to the list; returns how many there are
  auto gather = [&](uint64_t least) {
    if (mine >= least)
      for (int h = tid; h < lists; h += kPickThreads)
        for (int r = 0; r < M; ++r) {
          const uint64_t k = entry(h, r, &second);
          if (k < least) break;
          const int at = atomicAdd(&s_n, 1);
          if (at < kPickCap) {
            s_score[at] = k;
            s_second[at] = second;
          }
        }
    __syncthreads();
    return s_n;
  };
  // with those equal to it, but for -inf, which many may be
  int n = gather(bound > nothing ? bound : bound + 1);
  if (n > kPickCap && bound > nothing) {   // many are equal to the bound
    __syncthreads();
    if (tid == 0) s_n = 0;
    __syncthreads();
    n = gather(bound + 1);
  }
  if (n > kPickCap) {
    // one after the other, each the best behind the last
    uint64_t last = ~0ull, last2 = ~0ull;
    for (int r0 = 0; r0 < M; ++r0) {
      uint64_t best = 0, best2 = 0;
      if (mine > bound)
        for (int h = tid; h < lists; h += kPickThreads)
          for (int r = 0; r < M; ++r) {
            const uint64_t k = entry(h, r, &second);
            if (k <= bound || k < best) break;
            if ((k < last || (k == last && second < last2)) && (k > best || second > best2)) {
              best = k;
              best2 = second;
            }
          }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const uint64_t k = __shfl_xor_sync(kFull, best, o), k2 = __shfl_xor_sync(kFull, best2, o);
        if (k > best || (k == best && k2 > best2)) {
          best = k;
          best2 = k2;
        }
      }
      __syncthreads();
      if (lane == 0) {
        s_score[warp] = best;
        s_second[warp] = best2;
      }
      __syncthreads();
      for (int w = 0; w < kPickThreads / 32; ++w) {
        if (s_score[w] > best || (s_score[w] == best && s_second[w] > best2)) {
          best = s_score[w];
          best2 = s_second[w];
        }
      }
      if (tid == 0) {
        s_best[r0] = best;
        s_best2[r0] = best2;
      }
      last = best;
      last2 = best2;
    }
    n = M;
  } else {
    for (int i = tid; i < n; i += kPickThreads) {
      const uint64_t k = s_score[i], k2 = s_second[i];
      int r = 0;
      for (int u = 0; u < n; ++u) r += s_score[u] > k || (s_score[u] == k && s_second[u] > k2);
      if (r < M) {
        s_best[r] = k;
        s_best2[r] = k2;
      }
    }
  }
  // what is equal to the bound, in order of place, as lists and their equal entries are
  for (int h0 = 0, got = n; got < M && h0 < lists; h0 += kPickThreads) {
    const int h = h0 + tid;
    int first = 0, c = 0;
    if (h < lists)
      for (int r = 0; r < M; ++r) {
        const uint64_t k = entry(h, r, &second);
        if (k < bound || k == 0) break;
        if (k > bound) first = r + 1; else ++c;
      }
    int total;
    const int at = got + scan_block(c, s_part, &total);
    for (int r = 0; r < c && at + r < M; ++r) {
      s_best[at + r] = entry(h, first + r, &second);
      s_best2[at + r] = second;
    }
    got += total;
  }
  __syncthreads();
  if (tid < M) {
    const int w = key_beam(s_best2[tid]), token = key_token(s_best2[tid]);
    int place = tid;
    if (a.keep) {   // n_out == W
      bool first = true;
      int others = 0;      // candidates before this one that are not their beam's best
      uint64_t used = 0;   // beams that have a child
      for (int j = 0; j < M; ++j) {
        const int wj = key_beam(s_best2[j]);
        if (j < tid) {
          first = first && wj != w;
          others += (used >> wj) & 1;
        }
        used |= 1ull << wj;
      }
      place = w;
      if (!first) {
        uint64_t free_places = ~used;
        for (; others > 0; --others) free_places &= free_places - 1;
        place = __ffsll((long long)free_places) - 1;
      }
    }
    const int64_t o = (int64_t)b * M + place;
    a.out_scores[o] = (float)unordered64(s_best[tid]);
    a.out_parent[o] = (int32_t)(row0 + w);
    a.out_token[o] = token;
    if (a.out_done) a.out_done[o] = s_done[w] || token == a.eos;
  }
}

// Vectors of a thread: as many as leave at least four CTAs an SM, for fewer
// candidates and one selection per more logits.
int vectors_per_thread(int64_t rows, int64_t V, bool f32) {
  const int64_t want = 4 * sm_count();
  for (int nv = 16; nv > 2; nv /= 2) {
    const int64_t per = (int64_t)kChunkThreads * nv * (f32 ? 4 : 8);
    if (rows * ((V + per - 1) / per) >= want) return nv;
  }
  return 2;
}

// Parts of a row, with room for the logits before an unaligned row's start.
int64_t parts_of(int64_t V, int nv, bool f32) {
  const int64_t vec = f32 ? 4 : 8, per = kChunkThreads * nv * vec;
  return (V + vec - 1 + per - 1) / per;
}

size_t beam_bytes(int64_t rows, int64_t S, int n_out, size_t* cand_at) {
  const size_t part = ((size_t)rows * S * sizeof(float2) + 255) / 256 * 256;
  if (cand_at) *cand_at = part;
  return part + (size_t)rows * S * n_out * sizeof(uint64_t);
}

int check_sizes(int B, int W, int64_t V, int n_out) {
  if (B <= 0 || W <= 0 || V <= 0 || n_out <= 0) return TQ_ERR_ARG;
  if (W > kMaxBeams || n_out > kMaxBeams || V > 0x7fffffff / kMaxBeams) return TQ_ERR_UNSUPPORTED;
  if (n_out > W * V) return TQ_ERR_ARG;
  // parts are as small as 1024 logits
  if ((int64_t)B * W * (V / 1024 + 2) > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
  return TQ_OK;
}

template <bool F32>
bool launch_chunks(const BeamArgs& a, int nv, cudaStream_t st) {
  const int64_t grid = (int64_t)a.B * a.W * a.S;
  switch (nv) {
    case 16: return launch(beam_chunk_kernel<F32, 16>, grid, kChunkThreads, false, st, a);
    case 8: return launch(beam_chunk_kernel<F32, 8>, grid, kChunkThreads, false, st, a);
    case 4: return launch(beam_chunk_kernel<F32, 4>, grid, kChunkThreads, false, st, a);
    default: return launch(beam_chunk_kernel<F32, 2>, grid, kChunkThreads, false, st, a);
  }
}

}  // namespace
}  // namespace tq

extern "C" int tq_beam_workspace_bytes(int B, int W, int64_t V, int n_out, size_t* bytes) {
  if (!bytes) return TQ_ERR_ARG;
  const int st = tq::check_sizes(B, W, V, n_out);
  if (st != TQ_OK) return st;
  // fp32 logits are cut into more parts than fp16 ones
  const int64_t rows = (int64_t)B * W;
  size_t most = 0;
  for (int f32 = 0; f32 < 2; ++f32) {
    const size_t n = tq::beam_bytes(rows, tq::parts_of(V, tq::vectors_per_thread(rows, V, f32), f32), n_out, nullptr);
    most = n > most ? n : most;
  }
  *bytes = most;
  return TQ_OK;
}

extern "C" int tq_beam_select(const void* logits, tq_dtype dtype, int B, int W, int64_t V, int64_t row_stride,
                              const float* scores, const uint8_t* done, int64_t eos, int n_out, int keep_place,
                              float* out_scores, int32_t* out_parent, int32_t* out_token, uint8_t* out_done,
                              void* workspace, size_t workspace_bytes, void* stream) {
  if (!logits || !out_scores || !out_parent || !out_token) return TQ_ERR_ARG;
  if (dtype != TQ_F16 && dtype != TQ_F32) return TQ_ERR_ARG;
  int st = tq::check_sizes(B, W, V, n_out);
  if (st != TQ_OK) return st;
  if (row_stride < V || eos < -1 || eos >= V || (done && eos < 0) || (keep_place && n_out != W)) return TQ_ERR_ARG;
  const bool f32 = dtype == TQ_F32;
  const uintptr_t word = f32 ? 3u : 1u;
  if ((reinterpret_cast<uintptr_t>(logits) & word) || (reinterpret_cast<uintptr_t>(scores) & 3u) ||
      (reinterpret_cast<uintptr_t>(out_scores) & 3u) || (reinterpret_cast<uintptr_t>(out_parent) & 3u) ||
      (reinterpret_cast<uintptr_t>(out_token) & 3u))
    return TQ_ERR_ALIGN;
  const int64_t rows = (int64_t)B * W;
  const int nv = tq::vectors_per_thread(rows, V, f32);
  const int64_t S = tq::parts_of(V, nv, f32);
  size_t cand_at;
  if (!workspace || workspace_bytes < tq::beam_bytes(rows, S, n_out, &cand_at)) return TQ_ERR_WORKSPACE;
  if (!tq::aligned16(workspace)) return TQ_ERR_ALIGN;
  const tq::BeamArgs a{logits, row_stride, scores, done, eos, B, W, (int32_t)V, n_out, (int32_t)S, keep_place ? 1 : 0,
                       static_cast<float2*>(workspace),
                       reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + cand_at), out_scores, out_parent,
                       out_token, out_done};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool ok = (f32 ? tq::launch_chunks<true>(a, nv, s) : tq::launch_chunks<false>(a, nv, s)) &&
                  tq::launch(tq::beam_pick_kernel, B, tq::kPickThreads, true, s, a);
  return ok && cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
