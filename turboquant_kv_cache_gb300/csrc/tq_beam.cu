// A beam search's step: of every beam's continuations by every token of the
// vocabulary, the n_out best of each request.
//
// Candidate (w, v) of a request has the score  s_w + (x_wv - lse_w),  with
// lse_w = m + log sum_v exp(x_wv - m), m = max_v x_wv.  Within a row the order
// of the scores is the order of the logits, so the rows need not be
// normalised to be cut down:
//   chunk   one CTA per part of a row, or several, whose logits it reads once:
//           their maximum, the sum of exp(x - maximum), and the n_out largest;
//   pick    one CTA per request: lse of every row from its parts, and the
//           n_out best of all parts' candidates.
//
// The largest M of many values, without sorting them: the M-th largest T of
// the maxima of 2 M groups of threads or more is a bound, since M values are at
// least T; few others are.  What is above T goes to a list, of those equal to T the ones that come
// first fill it up, and a candidate's rank is the number of list entries before
// it.  Equal scores go by place (w V + v, see second_key), so the result does
// not depend on the order in which threads reach the list.
//
// Precision: exp and the parts' sums in 32 bits, log and scores in pairs of 32
// (48 bits); a score is rounded once.  The order in one row is exact, that of two
// rows as exact as their lse.  The term of a row's largest logit is 1 exactly and
// the others are off by 2^-22 and 2^-23 |x - m| of themselves, a change of reference
// by 3 2^-24, so lse is exact where a token leaves the others no weight, and off by
// up to 2e-7 for rows of Gaussian logits and 5e-7 for those with a token 10 or 15
// above (800 rows of 20011 and 128256 each).
// Infinities: a NaN logit counts as -inf and +inf as the largest finite
// number, so a row without any finite logit gives scores of -inf and no NaN.
//
// Bound.  Small: two launches, each a few loads, sorts and rankings in a row, in
// code that runs once (short code is faster here than unrolled code): 8 rows of
// 32000 fp16 logits 6.9 us.  Large: 512 rows of 128256, a fifth of them finished,
// 49 us: 41 for the logits at 5.0 TB/s (a copy's rate would be 31), the rest is
// the second launch.  There a part's bound and the merges of its lists are latency
// that three CTAs of four warps an SM do not cover (16% of the warps are live, 39%
// of the issue slots taken, of fp16 rows 51%): all 512 rows 54 us, of fp16 43 to 46,
// where a copy's rate would be 39 and 19.  Wide: with more than 16 kept the lists of
// few rows do not give the second launch's bound enough groups, and most entries
// pass it; above kPickCap they are selected one after the other.  8 requests of 32
// beams, 32000 fp32: 16 kept 21 us, 32 78, 64 180.
// Steps: selection in registers with 64-bit floating-point scores 177 us; scores in
// pairs of floats, lists without divisions 70; rows streamed through shared memory
// 58; bounds from a sorting network 53; a unit's terms added up behind the branch for
// what goes to the list 49.  Not kept: sums of threads and warps as pairs of floats
// (lse within 3e-7 instead of 5e-7) 55.
#include <cuda_runtime.h>
#include <math.h>

#include "tq_launch.cuh"

namespace tq {

int sm_count();

namespace {

constexpr int kMaxBeams = 64;      // beams of a request, and candidates kept
constexpr int kChunkThreads = 128;
constexpr int kPickThreads = 256;
constexpr int kListCap = 256;      // chunk: entries above the bound, and kSameMost a thread equal to it
constexpr int kSlots = 32;         // chunk: threads whose logits are put where they can be indexed
constexpr int kOwn = 2;            // pick: entries a thread keeps
constexpr int kPickCap = 1536;     // pick: entries above the bound
constexpr int kSameMost = 4;       // entries equal to the bound a thread lists
constexpr float kMost = 3.402823466e38f;

struct BeamArgs {
  const void* logits;
  int64_t row_stride;
  const float* scores;       // [B][W] or NULL: 0
  const uint8_t* done;       // [B][W] or NULL
  int64_t eos;
  int32_t B, W, V, n_out, S, keep;
  int32_t parts, span;       // of a row; of a CTA (S = parts / span, rounded up)
  float2* part;              // [B W][S] maximum, sum
  uint64_t* cand;            // [B W][S][n_out] keys, descending; 0: none
  float* out_scores;
  int32_t* out_parent;
  int32_t* out_token;
  uint8_t* out_done;
};

// A logit's key orders by value, then by the lower beam and token; it is never 0.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);   // -0 is 0
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}
// `row`: (kMaxBeams - 1 - beam) << 26, the same for a row's logits.
constexpr uint32_t kTokenMask = (1u << 26) - 1;
__device__ __forceinline__ uint64_t key_of(float x, int token, uint32_t row) {
  return ((uint64_t)ordered(x) << 32) | row | (kTokenMask - (uint32_t)token);
}
constexpr uint64_t kNothing = (uint64_t)0x007fffff << 32;   // the pair (-inf, none) as a key
constexpr float kLog2 = 0.693147180559945309417f;           // log 2, and what its rounding lost
constexpr float kLog2Rest = (float)(0.693147180559945309417 - (double)kLog2);

// A beam's score with NaN as -inf and +inf as the largest finite number.
__device__ __forceinline__ float beam_score(const BeamArgs& a, int64_t row) {
  return a.scores ? fminf(fmaxf(a.scores[row], -INFINITY), kMost) : 0.f;
}
__device__ __forceinline__ bool beam_done(const BeamArgs& a, int64_t row) { return a.done && a.done[row]; }

// Vectors of 16 bytes as logits, NaN and +inf as they come.
template <bool F32>
struct Vec {
  static constexpr int N = F32 ? 4 : 8;
  uint4 raw;
  __device__ __forceinline__ float at(int e) const {
    const uint32_t w = F32 ? (&raw.x)[e] : (&raw.x)[e >> 1];
    if (F32) return __uint_as_float(w);
    return h2f((uint16_t)((e & 1) ? w >> 16 : w & 0xffffu));
  }
  __device__ __forceinline__ float2 pair(int p) const {   // logits 2p and 2p + 1
    if (F32) return make_float2(__uint_as_float((&raw.x)[2 * p]), __uint_as_float((&raw.x)[2 * p + 1]));
    const uint32_t w = (&raw.x)[p];
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  // The same less m, conversion and difference of a half in one instruction.
  __device__ __forceinline__ float2 pair_less(int p, float m) const {
    if constexpr (F32) {
      return __fadd2_rn(pair(p), make_float2(-m, -m));
    } else {
      float2 d;
      asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\nadd.rn.f32.f16 %0, a, %3;\nadd.rn.f32.f16 %1, b, %3;\n}\n"
          : "=f"(d.x), "=f"(d.y)
          : "r"((&raw.x)[p]), "f"(-m));
      return d;
    }
  }
  // The largest of the vector, -inf where all are NaN.
  __device__ __forceinline__ float most() const {
    if (F32) return fmaxf(fmaxf(fmaxf(at(0), at(1)), fmaxf(at(2), at(3))), -INFINITY);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    const __half2* h = reinterpret_cast<const __half2*>(w);
    const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));   // passes over NaN
    return fmaxf(fmaxf(__low2float(m), __high2float(m)), -INFINITY);
  }
  // The raw words are what is kept: the next pass converts them again, where
  // the compiler would hold the converted ones in twice the registers.
  __device__ __forceinline__ void keep_raw() { asm volatile("" : "+r"(raw.x), "+r"(raw.y), "+r"(raw.z), "+r"(raw.w)); }
};

// NaN as -inf and +inf as the largest finite number.
__device__ __forceinline__ float tame(float x) { return fminf(fmaxf(x, -INFINITY), kMost); }

template <bool F32>
__device__ __forceinline__ float logit_at(const uint8_t* row, int64_t i) {
  return tame(F32 ? reinterpret_cast<const float*>(row)[i] : h2f(reinterpret_cast<const uint16_t*>(row)[i]));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (s, r) += (t, u), what the sum of s and t rounds off going to r.
__device__ __forceinline__ void add_to(float& s, float& r, float t, float u) {
  const float all = s + t, part = all - s;
  r += u + ((s - (all - part)) + (t - part));
  s = all;
}

// exp(from - to) for from <= to, to a step: what makes a sum relative to `from` one
// relative to `to`.  What the difference rounds off counts where it is large.
__device__ __forceinline__ float shrink(float from, float to) {
  if (from == to) return 1.f;
  float d = from, lost = 0.f;
  add_to(d, lost, -to, 0.f);
  if (!(d > -104.f)) return 0.f;   // below the range of 32 bits; -inf
  const float f = expf(d);
  return fmaf(f, lost, f);
}

// The M-th largest of the 32 K values that the lanes of a warp hold, K each
// (equal ones count one by one).  32 are sorted by a network of exchanges, of
// more each is counted against all.
template <int K, class T>
__device__ __forceinline__ T nth_largest(const T (&v)[K], int M) {
  const int lane = threadIdx.x & 31;
  if constexpr (K == 1) {
    T x = v[0];
#pragma unroll
    for (int run = 2; run <= 32; run *= 2)
#pragma unroll
      for (int gap = run / 2; gap; gap /= 2) {
        const T o = __shfl_xor_sync(kFull, x, gap);
        const bool larger = ((lane & run) == 0) == ((lane & gap) == 0);   // the last run descends
        x = larger == (o > x) ? o : x;
      }
    return __shfl_sync(kFull, x, M - 1);
  } else {
    int before[K];
#pragma unroll
    for (int k = 0; k < K; ++k) before[k] = 0;
#pragma unroll(4 / K)
    for (int l = 0; l < 32; ++l)
#pragma unroll
      for (int j = 0; j < K; ++j) {
        const T o = __shfl_sync(kFull, v[j], l);
#pragma unroll
        for (int k = 0; k < K; ++k) before[k] += o > v[k] || (o == v[k] && (j < k || (j == k && l < lane)));
      }
    T found = v[0];
    bool mine = false;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (before[k] == M - 1) {
        found = v[k];
        mine = true;
      }
    return __shfl_sync(kFull, found, __ffs(__ballot_sync(kFull, mine)) - 1);
  }
}

// The vector from logit i0 on of a row of V, -inf outside it.
template <bool F32>
__device__ __noinline__ Vec<F32> edge_vector(const uint8_t* row, int i0, int V) {
  Vec<F32> x;
  if (i0 >= 0 && i0 + Vec<F32>::N <= V) {
    x.raw = __ldcs(reinterpret_cast<const uint4*>(row + (int64_t)i0 * (F32 ? 4 : 2)));
    return x;
  }
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) w[e] = F32 ? 0xff800000u : 0xfc00fc00u;   // -inf
#pragma unroll
  for (int e = 0; e < Vec<F32>::N; ++e) {
    if (i0 + e < 0 || i0 + e >= V) continue;
    if (F32) {
      w[e] = reinterpret_cast<const uint32_t*>(row)[i0 + e];
    } else {
      const uint32_t h = reinterpret_cast<const uint16_t*>(row)[i0 + e];
      w[e >> 1] = (e & 1) ? (w[e >> 1] & 0xffffu) | (h << 16) : (w[e >> 1] & 0xffff0000u) | h;
    }
  }
  x.raw = make_uint4(w[0], w[1], w[2], w[3]);
  return x;
}

// The logits [from, to) of a row that is not read: all -inf, or of a finished
// beam 0 at eos and -inf elsewhere.  The first indexes fill the list.
__device__ __forceinline__ void synthetic_part(const BeamArgs& a, int64_t list, uint32_t beam, int from, int64_t to,
                                               bool at_eos) {
  const int lo = max(from, 0), hi = (int)imin64(to, a.V);
  const bool has = at_eos && a.eos >= lo && a.eos < hi;
  for (int r = threadIdx.x; r < a.n_out; r += blockDim.x) {
    uint64_t key = 0;
    if (has && r == 0) {
      key = key_of(0.f, (int)a.eos, beam);
    } else {
      int i = lo + r - (has ? 1 : 0);
      if (has && i >= a.eos) ++i;
      if (i < hi) key = key_of(-INFINITY, i, beam);
    }
    a.cand[list * a.n_out + r] = key;
  }
}

// sum += exp(x - m) of a thread's logits in pairs.  The difference comes first,
// so that the term of m itself is 1 and no term's exponent is off by more than two
// roundings of its own: one multiply-add, x log2 e less a rounded m log2 e, puts that
// rounding into every term, and from logits of 2^30 on it is a factor that leaves
// the range of 32 bits.
template <bool F32, int NV>
__device__ __forceinline__ void add_exp(const Vec<F32> (&x)[NV], float m, float2 (&sum)[2]) {
  const float2 by = make_float2(kLog2e, kLog2e);
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int q = 0; q < Vec<F32>::N / 2; ++q) {
      const float2 t = __fmul2_rn(x[j].pair_less(q, m), by);
      sum[q & 1] = __fadd2_rn(sum[q & 1], make_float2(ex2(t.x), ex2(t.y)));
    }
}

// Sum of exp(x - m) of a thread's logits, m finite.
template <bool F32, int NV>
__device__ __forceinline__ float sum_exp(Vec<F32> (&x)[NV], float m) {
  float2 sum[2] = {};
#pragma unroll
  for (int j = 0; j < NV; ++j) x[j].keep_raw();
  add_exp(x, m, sum);
  return (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
}

// Shared memory of a chunk CTA.
template <int NV>
struct ChunkShared {
  float max[kChunkThreads];
  float sum[kChunkThreads / 32], ref[kChunkThreads / 32];
  float bound;
  int above, equal, many, slots;
  uint4 slot[kSlots][NV + 1];   // (the odd vector spreads the slots over the banks)
  uint64_t key[kListCap + kSameMost * kChunkThreads];
  uint64_t best[2][kMaxBeams];  // of the parts so far; of one more
};

// Vectors of 128 threads from vector v0 + tid of the row on, 128 apart.
template <bool F32, int N>
__device__ __forceinline__ void load_vectors(Vec<F32> (&x)[N], const uint8_t* base, int first, int lead, int V) {
  constexpr int VEC = Vec<F32>::N;
  const int i0 = first * VEC - lead;   // the first of all threads' logits
  const int mine = (first + (int)threadIdx.x) * VEC - lead;
  if (i0 >= 0 && i0 + N * kChunkThreads * VEC <= V) {   // inside the row
    const uint4* from = reinterpret_cast<const uint4*>(base + (int64_t)mine * (F32 ? 4 : 2));
#pragma unroll
    for (int j = 0; j < N; ++j) x[j].raw = __ldcs(from + j * kChunkThreads);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = edge_vector<F32>(base, mine + j * kChunkThreads * VEC, V);
  }
}

// The maximum of a part, whose vectors are x, and a bound that at least n_out of
// its logits reach: sh.bound, once the CTA's threads have met again.
template <bool F32, int NV>
__device__ __forceinline__ float part_bound(const Vec<F32> (&x)[NV], int n_out, ChunkShared<NV>& sh, float* mine) {
  constexpr int WARPS = kChunkThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float most = -INFINITY;
#pragma unroll
  for (int j = 0; j < NV; ++j) most = fmaxf(most, x[j].most());
  *mine = fminf(most, kMost);
  sh.max[tid] = *mine;
  if (tid == 0) sh.above = sh.equal = sh.many = sh.slots = 0;
  __syncthreads();
  float top[WARPS];
#pragma unroll
  for (int w = 0; w < WARPS; ++w) top[w] = sh.max[32 * w + lane];
  float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  if (warp == 0) {
    // the n_out-th largest of groups' maxima, of at least twice as many groups
    float bound;
    if (n_out <= 16) {
      const float one[1] = {m};
      bound = nth_largest(one, n_out);
    } else if (n_out <= 32) {
      const float two[2] = {fmaxf(top[0], top[1]), fmaxf(top[2], top[3])};
      bound = nth_largest(two, n_out);
    } else {
      bound = nth_largest(top, n_out);
    }
    if (lane == 0) sh.bound = bound;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  return m;
}

// Which of a thread's logits are at least this, a bit each.
template <bool F32, int NV>
__device__ __forceinline__ uint32_t reach(const Vec<F32> (&x)[NV], float least) {
  static_assert(NV * Vec<F32>::N <= 32, "a bit for each logit of a thread");
  uint32_t live = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int e = 0; e < Vec<F32>::N; ++e)
      if (x[j].at(e) >= least) live |= 1u << (j * Vec<F32>::N + e);
  return live;
}

// The n_out largest logits of a part, whose vectors are x, descending to
// out[0 .. n_out) (keys; 0: none).  Returns the part's maximum; sh.sum holds the
// warps' sums of exp(x - maximum).  The CTA's threads meet in it; what they read
// of sh afterwards, or write to out, is not ordered yet.
template <bool F32, int NV>
__device__ __forceinline__ float select_part(Vec<F32> (&x)[NV], const BeamArgs& a, const uint8_t* base, uint32_t beam, int lead,
                                             int s, ChunkShared<NV>& sh, uint64_t* out) {
  constexpr int VEC = Vec<F32>::N, PER = kChunkThreads * NV * VEC, WARPS = kChunkThreads / 32;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int v0 = s * (kChunkThreads * NV) + tid;
  float mine;
  const float m = part_bound(x, a.n_out, sh, &mine);
  const float mref = m == -INFINITY ? 0.f : m;
  float sum = sum_exp(x, mref);
  if (!(sum < INFINITY)) {   // NaN or +inf among them
    sum = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      x[j].keep_raw();
#pragma unroll
      for (int e = 0; e < VEC; ++e) sum += ex2((tame(x[j].at(e)) - mref) * kLog2e);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
  if (lane == 0) sh.sum[warp] = sum;
  __syncthreads();
  const float bound = sh.bound;
  if (mine >= bound && mine != -INFINITY) {
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j].keep_raw();
    uint32_t live = reach(x, fmaxf(bound, -kMost));   // -inf (places outside the row too) never
    // registers have no indexes: the logits go to shared memory, those of a thread
    // without a slot are read again
    const int slot = atomicAdd(&sh.slots, 1);
    if (slot < kSlots) {
#pragma unroll
      for (int j = 0; j < NV; ++j) sh.slot[slot][j] = x[j].raw;
    }
    int same = 0;
    for (; live; live &= live - 1) {
      const int k = __ffs(live) - 1;
      const int i = (v0 + k / VEC * kChunkThreads) * VEC + k % VEC - lead;
      const float v = slot < kSlots ? logit_at<F32>(reinterpret_cast<const uint8_t*>(sh.slot[slot]), k)
                                    : logit_at<F32>(base, i);
      if (v > bound) {
        const int at = atomicAdd(&sh.above, 1);
        if (at < kListCap) sh.key[at] = key_of(v, i, beam);
      } else if (++same <= kSameMost) {
        sh.key[kListCap + atomicAdd(&sh.equal, 1)] = key_of(v, i, beam);
      } else {
        sh.many = 1;   // the rest of the loop looks for those above it
      }
    }
  }
  __syncthreads();
  const int above = sh.above;
  const int lo = max(s * PER - lead, 0), hi = (int)imin64((int64_t)(s + 1) * PER - lead, a.V);
  if (above > kListCap) {
    // a few threads hold most of the large values: one after the other, each
    // the largest below the last.  There are more than n_out above the bound
    uint64_t last = ~0ull;
    for (int r = 0; r < a.n_out; ++r) {
      uint64_t best = 0;
#pragma unroll 4
      for (int i = lo + tid; i < hi; i += kChunkThreads) {
        const uint64_t k = key_of(logit_at<F32>(base, i), i, beam);
        if (k < last && k > best) best = k;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const uint64_t k = __shfl_xor_sync(kFull, best, o);
        best = k > best ? k : best;
      }
      __syncthreads();   // the last round's results have been read
      if (lane == 0) sh.key[warp] = best;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < WARPS; ++w) best = sh.key[w] > best ? sh.key[w] : best;
      if (tid == 0) out[r] = best;
      last = best;
    }
    return m;
  }
  for (int i = tid; i < above; i += kChunkThreads) {
    const uint64_t k = sh.key[i];
    int r = 0;
#pragma unroll 8
    for (int u = 0; u < above; ++u) r += sh.key[u] > k;
    if (r < a.n_out) out[r] = k;
  }
  if (above >= a.n_out) return m;
  if (bound != -INFINITY && !sh.many) {
    const int equal = sh.equal;   // with those above at least n_out
    for (int i = tid; i < equal; i += kChunkThreads) {
      const uint64_t k = sh.key[kListCap + i];
      int r = above;
      for (int u = 0; u < equal; ++u) r += sh.key[kListCap + u] > k;
      if (r < a.n_out) out[r] = k;
    }
  } else if (warp == 0) {
    // many logits are the bound itself (a mask's value, or -inf): the first of
    // them, which are among the part's first few then
    int r = above;
    for (int i0 = lo; i0 < hi && r < a.n_out; i0 += 64) {
      float v[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = i0 + 32 * u + lane;
        v[u] = i < hi ? logit_at<F32>(base, i) : NAN;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t found = __ballot_sync(kFull, v[u] == bound);
        const int at = r + __popc(found & ((1u << lane) - 1));
        if (((found >> lane) & 1u) && at < a.n_out) out[at] = key_of(bound, i0 + 32 * u + lane, beam);
        r += __popc(found);
      }
    }
    for (r += lane; r < a.n_out; r += 32) out[r] = 0;   // a part of fewer logits
  }
  return m;
}

// Part t to sh.best[1], for what seldom happens: a call keeps its registers out
// of the kernel's.
template <bool F32, int NV>
__device__ __noinline__ float select_again(const BeamArgs& a, const uint8_t* base, uint32_t beam, int lead, int t,
                                           ChunkShared<NV>& sh) {
  Vec<F32> x[NV];
  load_vectors(x, base, t * kChunkThreads * NV, lead, a.V);
  return select_part<F32, NV>(x, a, base, beam, lead, t, sh, sh.best[1]);
}

// sh.best[0] := the n_out largest of its keys, the first n of sh.key and, with
// `more`, sh.best[1].
template <int NV>
__device__ __forceinline__ void merge_best(ChunkShared<NV>& sh, int n_out, int n, bool more) {
  constexpr int MOST = (kListCap + 2 * kMaxBeams + kChunkThreads - 1) / kChunkThreads;
  const int best = more ? 2 * n_out : n_out, all = n + best;
  auto at = [&](int i) {
    return i >= best ? sh.key[i - best] : i >= n_out ? sh.best[1][i - n_out] : sh.best[0][i];
  };
  uint64_t k[MOST];
  int rank[MOST];
#pragma unroll
  for (int q = 0; q < MOST; ++q) {
    const int i = (int)threadIdx.x + q * kChunkThreads;
    k[q] = i < all ? at(i) : 0;
    rank[q] = kMaxBeams;
    if (k[q]) {
      rank[q] = 0;
#pragma unroll 8
      for (int u = 0; u < n_out; ++u) rank[q] += sh.best[0][u] > k[q];
      if (more)
        for (int u = 0; u < n_out; ++u) rank[q] += sh.best[1][u] > k[q];
#pragma unroll 8
      for (int u = 0; u < n; ++u) rank[q] += sh.key[u] > k[q];
    }
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < MOST; ++q)
    if (rank[q] < n_out) sh.best[0][rank[q]] = k[q];
  if (threadIdx.x == 0) sh.above = 0;
  __syncthreads();
}

// A thread's own 16 bytes of shared memory, loaded asynchronously.
__device__ __forceinline__ void copy_async(uint4* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;\n" ::"r"((uint32_t)__cvta_generic_to_shared(to)), "l"(from)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;\n" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;\n" ::"n"(N) : "memory"); }

constexpr int kUnit = 4;        // stream: vectors of a thread in a unit (four are written out)
constexpr int kStages = 4;      // stream: units of a thread in flight or worked on
constexpr int kStreamBits = 32; // logits of a thread in a part that streams

// One CTA for `span` parts of a row.  The first gives a bound and a maximum; the
// rest streams through shared memory that each thread loads for itself, so no
// thread waits for another: what is above the bound goes to the list (a later
// equal one loses by its index).  A thread's terms are relative to the largest
// logit that it knows of, the CTA's at the last merge or its own since: one above
// that is above the bound too, so only the branch for what goes to the list looks
// for it, and the sum so far follows.  After two parts, and as their number doubles
// or quadruples, the list is merged, the bound rises, so that about one to three
// times n_out logits pass it each time, and the threads' sums are added up relative
// to the largest logit of all of them.
// Where more pass than the list holds, or NaN or +inf are among them, or the first
// part leaves less than n_out, the parts since the last merge are selected from one
// by one.
template <bool F32, int NV>
__global__ void __launch_bounds__(kChunkThreads, 5) beam_chunk_kernel(const BeamArgs a) {
  constexpr int VEC = Vec<F32>::N, PER = kChunkThreads * NV * VEC;   // logits of a part
  constexpr bool STREAMS = NV * VEC == kStreamBits;
  __shared__ ChunkShared<NV> sh;
  __shared__ uint4 s_ring[STREAMS ? kStages : 1][kUnit][STREAMS ? kChunkThreads : 1];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int list = blockIdx.x, at_row = list / a.S, s = list - at_row * a.S;
  const int64_t row = at_row;
  const int p0 = s * a.span, p1 = min(p0 + a.span, a.parts);
  const int esz = F32 ? 4 : 2;
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + row * a.row_stride * esz;
  // vectors lie on 16-byte boundaries; the first of a row starts `lead` logits before it
  const int lead = (int)((reinterpret_cast<uintptr_t>(base) & 15u) / esz);
  const uint32_t beam = (uint32_t)(kMaxBeams - 1 - at_row % a.W) << 26;
  uint64_t* out = a.cand + (int64_t)list * a.n_out;
  const float score = beam_score(a, row);
  const bool done = beam_done(a, row);
  if (done || score == -INFINITY) {   // a row that is not read
    if (tid == 0) a.part[list] = make_float2(-INFINITY, 0.f);
    synthetic_part(a, list, beam, p0 * PER - lead, (int64_t)p1 * PER - lead, done && score != -INFINITY);
    return;
  }
  // units of the stream, unit u in ring stage u % kStages; but for an unaligned
  // row's first they lie inside the row up to u_in
  const int u_end = p1 * (NV / kUnit), u_in = (int)(((int64_t)a.V + lead) / (kChunkThreads * kUnit * VEC));
  const uint4* vectors = reinterpret_cast<const uint4*>(base - lead * esz) + tid;
  auto fetch = [&](int u) {
    uint4* to = &s_ring[u % kStages][0][tid];
    if (u < min(u_in, u_end) && (u > 0 || lead == 0)) {
#pragma unroll
      for (int j = 0; j < kUnit; ++j) copy_async(to + j * kChunkThreads, vectors + (u * kUnit + j) * kChunkThreads);
    } else if (u < u_end) {
#pragma unroll
      for (int j = 0; j < kUnit; ++j)
        to[j * kChunkThreads] = edge_vector<F32>(base, ((u * kUnit + j) * kChunkThreads + tid) * VEC - lead, a.V).raw;
    }
    copy_commit();
  };
  Vec<F32> x[NV];
  float m, l;
  if (!STREAMS || p1 - p0 == 1) {
    load_vectors(x, base, p0 * kChunkThreads * NV, lead, a.V);
    m = select_part<F32, NV>(x, a, base, beam, lead, p0, sh, out);
    l = (sh.sum[0] + sh.sum[1]) + (sh.sum[2] + sh.sum[3]);
  } else {
    constexpr int FIRST = STREAMS ? NV / kUnit : 1;   // units of a part
    const int u0 = p0 * FIRST;
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(u0 + k);
    for (int r = tid; r < a.n_out; r += kChunkThreads) sh.best[0][r] = 0;
    copy_wait<kStages - 1 - FIRST>();
    auto in_ring = [&](int j) { return &s_ring[(u0 + j / kUnit) % kStages][j % kUnit][tid]; };   // the first part's
#pragma unroll
    for (int j = 0; j < NV; ++j) x[j].raw = *in_ring(j);
    float mine;
    m = part_bound(x, a.n_out, sh, &mine);
    l = 0.f;
    // a unit's terms are added up by themselves, and the units' sums as a pair:
    // however long the row, the sum is off by a few steps
    float total = 0.f, rest = 0.f;
    auto add_unit = [&](float2 (&sums)[2]) { add_to(total, rest, (sums[0].x + sums[0].y) + (sums[1].x + sums[1].y), 0.f); };
    {
      float2 sums[2] = {};
      add_exp(x, m, sums);
      add_unit(sums);
    }
    __syncthreads();
    float bound = sh.bound;
    const bool found = bound != -INFINITY;   // else the first part leaves less than n_out
    if (found && mine >= bound) {
      for (uint32_t live = reach(x, bound); live; live &= live - 1) {
        const int k = __ffs(live) - 1, i = ((p0 * NV + k / VEC) * kChunkThreads + tid) * VEC + k % VEC - lead;
        const int at = atomicAdd(&sh.above, 1);
        if (at < kListCap)
          sh.key[at] = key_of(logit_at<F32>(reinterpret_cast<const uint8_t*>(in_ring(k / VEC)), k % VEC), i, beam);
      }
    }
#pragma unroll
    for (int k = 0; k < FIRST; ++k) fetch(u0 + kStages - 1 + k);   // into the first part's stages and the one before
    // parts [p, q), of which the first of all is in the list already.  Up to 32
    // candidates the list holds what passes the bound while the parts quadruple
    const int grow = a.n_out <= 32 ? 4 : 2;
    for (int p = p0, q = min(p0 + 2, p1); p < p1; p = q, q = min(p0 + grow * (q - p0), p1)) {
      const bool fits = m != -INFINITY && (p > p0 || found);
      float ref = m;   // this thread's terms are relative to it
      for (int u = (p > p0 ? p : p0 + 1) * (NV / kUnit); u < q * (NV / kUnit); ++u) {
        copy_wait<kStages - 2>();
        const uint4* from = &s_ring[u % kStages][0][tid];
        Vec<F32> y[kUnit];
#pragma unroll
        for (int j = 0; j < kUnit; ++j) y[j].raw = from[j * kChunkThreads];
        fetch(u + kStages - 1);   // into the stage before this one, whose logits have been used
        const float most = fmaxf(fmaxf(y[0].most(), y[1].most()), fmaxf(y[2].most(), y[3].most()));
        if (most > bound) {
          if (most > ref) {   // so it is above the bound too, which is at most m
            const float to = fminf(most, kMost), f = shrink(ref, to);
            total *= f;
            rest *= f;
            ref = to;
          }
          for (uint32_t live = reach(y, bound); live; live &= live - 1) {
            const int k = __ffs(live) - 1;
            const float v = logit_at<F32>(reinterpret_cast<const uint8_t*>(from + k / VEC * kChunkThreads), k % VEC);
            if (v == bound) continue;
            const int at = atomicAdd(&sh.above, 1);
            if (at < kListCap) sh.key[at] = key_of(v, ((u * kUnit + k / VEC) * kChunkThreads + tid) * VEC + k % VEC - lead, beam);
          }
        }
        float2 sums[2] = {};
        add_exp(y, ref, sums);
        add_unit(sums);
      }
      // the sum of all threads, relative to the largest logit so far
      float top = ref;
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
      float sum = (total + rest) * shrink(ref, top);
      total = rest = 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kFull, sum, o);
      if (lane == 0) {
        sh.sum[warp] = sum;
        sh.ref[warp] = top;
      }
      __syncthreads();
      const int n = sh.above;
      top = fmaxf(fmaxf(sh.ref[0], sh.ref[1]), fmaxf(sh.ref[2], sh.ref[3]));
      const float part = (sh.sum[0] * shrink(sh.ref[0], top) + sh.sum[1] * shrink(sh.ref[1], top)) +
                         (sh.sum[2] * shrink(sh.ref[2], top) + sh.sum[3] * shrink(sh.ref[3], top));
      if (fits && part < INFINITY && n <= kListCap) {   // else NaN or +inf among them
        merge_best(sh, a.n_out, n, false);
        l = l * shrink(m, top) + part;
        m = top;
      } else {
        if (p == p0) m = -INFINITY;
        for (int t = p; t < q; ++t) {
          __syncthreads();
          const float mt = select_again<F32, NV>(a, base, beam, lead, t, sh);
          const float lt = (sh.sum[0] + sh.sum[1]) + (sh.sum[2] + sh.sum[3]);
          const float both = fmaxf(m, mt);
          if (both != -INFINITY) l = l * shrink(m, both) + lt * shrink(mt, both);
          m = both;
          __syncthreads();
          merge_best(sh, a.n_out, 0, true);
        }
      }
      bound = unordered((uint32_t)(sh.best[0][a.n_out - 1] >> 32));
    }
    for (int r = tid; r < a.n_out; r += kChunkThreads) out[r] = sh.best[0][r];
  }
  if (tid == 0) a.part[list] = make_float2(m, l);
  // the second launch's blocks come late, when there is room on every SM: early
  // ones gather on the first that has some, and take twice the time
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
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
// that the pair does not tell them apart), then the lower token.
__device__ __forceinline__ uint64_t second_key(uint64_t key) {
  const uint32_t low = (uint32_t)key;
  return ((uint64_t)(low >> 26) << 58) | ((key >> 32) << 26) | (low & kTokenMask);
}
__device__ __forceinline__ int key_beam(uint64_t second) { return kMaxBeams - 1 - (int)(second >> 58); }
__device__ __forceinline__ int key_token(uint64_t second) { return (int)(kTokenMask - ((uint32_t)second & kTokenMask)); }

// An entry's score as an ordered key; 0: none.  A pair is brought into the one form
// in which it orders as (first, second).  `row`: of each beam, its maximum and what a
// logit less that lacks of its score.
__device__ __forceinline__ uint64_t score_key(const float4* row, uint64_t k) {
  if (!k) return 0;
  const float x = unordered((uint32_t)(k >> 32));
  if (x == -INFINITY) return kNothing;
  const float4 q = row[kMaxBeams - 1 - ((uint32_t)k >> 26)];
  float hi = x, lo = 0.f;
  add_to(hi, lo, -q.x, 0.f);
  add_to(hi, lo, q.y, q.z);
  const float top = hi + lo;
  if (!(top > -INFINITY)) return kNothing + 1;   // out of the range of 32 bits
  return ((uint64_t)ordered(top) << 32) | ordered(lo - (top - hi));
}

// The entries [*first, *end) of a list (M, descending) whose score is `bound`.
__device__ __forceinline__ void equal_range(const float4* row, const uint64_t* list, int M, uint64_t bound, int* first, int* end) {
  int lo = 0, hi = M;   // the first that is not above it
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (score_key(row, list[mid]) > bound) lo = mid + 1; else hi = mid;
  }
  *first = lo;
  hi = M;               // the first that is below it, or none
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    const uint64_t k = score_key(row, list[mid]);
    if (k >= bound && k != 0) lo = mid + 1; else hi = mid;
  }
  *end = lo;
}

// Whether entries of one beam have the score `bound` and different logits (tiny
// differences beside a large score, which a pair does not hold).
__device__ __forceinline__ bool equal_of_many(const float4* row, const uint64_t* cand, int M, int W, int S, uint64_t bound) {
  __shared__ uint32_t s_low[kMaxBeams], s_high[kMaxBeams];
  const int tid = threadIdx.x;
  if (tid < kMaxBeams) {
    s_low[tid] = 0xffffffffu;
    s_high[tid] = 0;
  }
  __syncthreads();
  for (int h = tid; h < W * S; h += kPickThreads) {
    const uint64_t* list = cand + (int64_t)h * M;
    int first, end;
    equal_range(row, list, M, bound, &first, &end);
    if (first < end) {
      atomicMax(&s_high[h / S], (uint32_t)(list[first] >> 32));
      atomicMin(&s_low[h / S], (uint32_t)(list[end - 1] >> 32));
    }
  }
  __syncthreads();
  return __syncthreads_or(tid < W && s_low[tid] < s_high[tid]);
}

// The M best entries from `least` on, one after the other, each the best behind the
// last, to `to` and `to2` (scores and what orders equal ones); `mine`: the best of this
// thread's lists.
__device__ __forceinline__ void one_by_one(const float4* row, const uint64_t* cand, int M, int lists, uint64_t least, uint64_t mine,
                                        uint64_t* to, uint64_t* to2) {
  constexpr int WARPS = kPickThreads / 32;
  __shared__ uint64_t s_top[WARPS], s_top2[WARPS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint64_t last = ~0ull, last2 = ~0ull;
  for (int r0 = 0; r0 < M; ++r0) {
    uint64_t best = 0, best2 = 0;
    if (mine >= least)
      for (int h = tid; h < lists; h += kPickThreads)
        for (int r = 0; r < M; ++r) {
          const uint64_t raw = cand[(int64_t)h * M + r], k = score_key(row, raw), second = second_key(raw);
          if (k < least || k < best) break;
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
    __syncthreads();   // the last round's results have been read
    if (lane == 0) {
      s_top[warp] = best;
      s_top2[warp] = best2;
    }
    __syncthreads();
    for (int w = 0; w < WARPS; ++w) {
      if (s_top[w] > best || (s_top[w] == best && s_top2[w] > best2)) {
        best = s_top[w];
        best2 = s_top2[w];
      }
    }
    if (tid == 0) {
      to[r0] = best;
      to2[r0] = best2;
    }
    last = best;
    last2 = best2;
  }
}

// (Four blocks an SM: 64 registers instead of 40, which the compiler takes by itself.
// 2 requests of 4 beams 7.2 -> 7.1 us, 12 of 32 beams and 64 kept 220 -> 214; with two
// blocks 1000 requests of 4 beams take 100 us instead of 98)
__global__ void __launch_bounds__(kPickThreads, 4) beam_pick_kernel(const BeamArgs a) {
  constexpr int WARPS = kPickThreads / 32;
  __shared__ float4 s_row[kMaxBeams];   // see score_key
  __shared__ uint32_t s_max[kPickThreads];
  __shared__ int s_list[kPickThreads], s_lists;
  __shared__ uint64_t s_score[kPickCap], s_second[kPickCap];
  __shared__ uint64_t s_best[kMaxBeams], s_best2[kMaxBeams];
  __shared__ int s_n, s_part[WARPS], s_from[kMaxBeams];
  __shared__ uint8_t s_done[kMaxBeams];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int b = blockIdx.x, M = a.n_out, lists = a.W * a.S;
  const int64_t row0 = (int64_t)b * a.W;
  const uint64_t* cand = a.cand + row0 * a.S * M;
  // few entries: each thread keeps up to kOwn of them; else the lists' first ones
  const bool own = lists * M <= kOwn * kPickThreads;
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  uint64_t raw[kOwn];   // on their way during the sums
#pragma unroll
  for (int e = 0; e < kOwn; ++e) {
    const int i = tid + e * kPickThreads;
    raw[e] = own ? (i < lists * M ? cand[i] : 0) : (i < lists ? cand[(int64_t)i * M] : 0);
  }
  if (tid == 0) s_n = 0;
  if (tid < kMaxBeams) s_from[tid] = 0;
  // A score is (x - m) + (s - log sum) in pairs of floats: 64-bit sums are slow
  // here.  log of 2^e f with f in [3/4, 3/2) is e log 2 + log f, whose second
  // part is below 0.41 and so off by 3e-8 at most
  for (int w = warp; w < a.W; w += WARPS) {
    const float score = beam_score(a, row0 + w);
    const bool done = beam_done(a, row0 + w);
    const float2* p = a.part + (row0 + w) * a.S;
    const float2 first = lane < a.S ? p[lane] : make_float2(-INFINITY, 0.f);
    // parts' sums relative to the row's maximum, as a pair of floats
    float m = first.x, sum = 0.f, rest = 0.f;
    for (int i = lane + 32; i < a.S; i += 32) m = fmaxf(m, p[i].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
    if (first.x != -INFINITY) sum = first.y * shrink(first.x, m);
    for (int i = lane + 32; i < a.S; i += 32) {
      const float2 q = p[i];
      if (q.x != -INFINITY) add_to(sum, rest, q.y * shrink(q.x, m), 0.f);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float s2 = __shfl_xor_sync(kFull, sum, o), r2 = __shfl_xor_sync(kFull, rest, o);
      add_to(sum, rest, s2, r2);
    }
    if (lane == 0) {
      float add = score, low = 0.f, most = 0.f;   // of a finished beam lse is 0
      if (!done && score != -INFINITY && m != -INFINITY) {
        const int e = (__float_as_int(sum) - 0x3f400000) >> 23;   // the sum is 1 at least
        const float f = __int_as_float(__float_as_int(sum) - (e << 23)), n = (float)e;
        const float by_two = n * kLog2, lost = fmaf(n, kLog2, -by_two) + n * kLog2Rest;
        add_to(add, low, -by_two, -lost);
        add_to(add, low, -logf(f), -(rest / sum));
        most = m;
      }
      s_row[w] = make_float4(most, add, low, 0.f);
      s_done[w] = done;
    }
  }
  __syncthreads();
  auto score_of = [&](uint64_t k) { return score_key(s_row, k); };
  // entry r of list h (descending in r)
  auto entry = [&](int h, int r, uint64_t* second) {
    const uint64_t k = cand[(int64_t)h * M + r];
    *second = second_key(k);
    return score_of(k);
  };
  uint64_t mine = 0, second;
  uint64_t key[kOwn];
#pragma unroll
  for (int e = 0; e < kOwn; ++e) {
    key[e] = score_of(raw[e]);
    mine = key[e] > mine ? key[e] : mine;
  }
  if (!own)
    for (int h = tid + kOwn * kPickThreads; h < lists; h += kPickThreads) {
      const uint64_t k = score_of(cand[(int64_t)h * M]);
      mine = k > mine ? k : mine;
    }
  s_max[tid] = (uint32_t)(mine >> 32);
  __syncthreads();
  // the M-th largest of groups' maxima, of at least twice as many groups, by the
  // keys' first words: few more have the same.  0 is the maximum of a group
  // without a list: then everything is above the bound
  uint32_t first_word;
  auto group = [&](int i, int n) {   // the largest of n warps' values from warp i on
    uint32_t g = s_max[32 * i + lane];
    for (int w = 1; w < n; ++w) g = max(g, s_max[32 * (i + w) + lane]);
    return g;
  };
  if (M <= 16) {
    const uint32_t one[1] = {group(0, 8)};
    first_word = nth_largest(one, M);
  } else if (M <= 32) {
    const uint32_t two[2] = {group(0, 4), group(4, 4)};
    first_word = nth_largest(two, M);
  } else {
    const uint32_t four[4] = {group(0, 2), group(2, 2), group(4, 2), group(6, 2)};
    first_word = nth_largest(four, M);
  }
  uint64_t bound = (uint64_t)first_word << 32;
  const int span = M <= 16 ? 16 : M <= 32 ? 32 : 64;   // threads of a list
  auto push = [&](uint64_t k, uint64_t k2) {
    const int at = atomicAdd(&s_n, 1);
    if (at < kPickCap) {
      s_score[at] = k;
      s_second[at] = k2;
    }
  };
  // entries from `least` on to the list; returns how many there are
  auto gather = [&](uint64_t least) {
    if (own) {
#pragma unroll
      for (int e = 0; e < kOwn; ++e)
        if (key[e] >= least) push(key[e], second_key(raw[e]));
    } else {
      for (int h0 = 0; h0 < lists; h0 += kPickThreads) {
        // lists that have some
        __syncthreads();
        if (tid == 0) s_lists = 0;
        __syncthreads();
        const int h = h0 + tid;
        if (mine >= least && h < lists && score_of(cand[(int64_t)h * M]) >= least)
          s_list[atomicAdd(&s_lists, 1)] = h;
        __syncthreads();
        const int found = s_lists;
        for (int i = tid / span; i < found; i += kPickThreads / span) {
          const int r = tid % span;
          if (r >= M) continue;
          const uint64_t k = entry(s_list[i], r, &second);
          if (k >= least) push(k, second);
        }
      }
    }
    __syncthreads();
    return s_n;
  };
  // with those equal to it, but for -inf, which many may be
  int n = gather(bound > kNothing ? bound : bound + 1);
  if (n > kPickCap && bound > kNothing) {
    // many are equal to the bound, or nearly: the threads' M-th largest maximum itself
    __syncthreads();
    s_score[tid] = mine;
    if (tid == 0) s_n = 0;
    __syncthreads();
    int before = 0;
    for (int u = 0; u < kPickThreads; ++u) before += s_score[u] > mine || (s_score[u] == mine && u < tid);
    if (before == M - 1) s_best[0] = mine;
    __syncthreads();
    bound = s_best[0];
    __syncthreads();
    n = gather(bound + 1);
  }
  // more are equal to the bound than the list takes: those of one logit go by place,
  // as the lists do; different ones of a beam may lie in any of its lists
  const bool of_many = n < M && bound > kNothing && equal_of_many(s_row, cand, M, a.W, a.S, bound);
  if (n > kPickCap || of_many) {
    one_by_one(s_row, cand, M, lists, of_many ? bound : bound + 1, mine, s_best, s_best2);
    n = M;
  } else {
    for (int i = tid; i < n; i += kPickThreads) {
      const uint64_t k = s_score[i], k2 = s_second[i];
      int r = 0;
#pragma unroll 4
      for (int u = 0; u < n; ++u) r += s_score[u] > k || (s_score[u] == k && s_second[u] > k2);
      if (r < M) {
        s_best[r] = k;
        s_best2[r] = k2;
      }
    }
  }
  // what is equal to the bound, in order of place, as lists and their equal entries of one logit are
  if (n < M) {
    for (int h0 = 0, got = n; got < M && h0 < lists; h0 += kPickThreads) {
      const int h = h0 + tid;
      int first = 0, end = 0;
      if (h < lists) equal_range(s_row, cand + (int64_t)h * M, M, bound, &first, &end);
      int total;
      const int at = got + scan_block(end - first, s_part, &total);
      for (int r = first; r < end && at + r - first < M; ++r) s_from[at + r - first] = h * M + r;
      got += total;
    }
    __syncthreads();
    if (tid >= n && tid < M) {
      s_best[tid] = entry(s_from[tid] / M, s_from[tid] % M, &second);
      s_best2[tid] = second;
    }
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
    a.out_scores[o] = unordered((uint32_t)(s_best[tid] >> 32));
    a.out_parent[o] = (int32_t)(row0 + w);
    a.out_token[o] = token;
    if (a.out_done) a.out_done[o] = s_done[w] || token == a.eos;
  }
}

// How a row is cut up.
struct Cut {
  int nv;           // vectors of a thread in a part
  int64_t parts;    // of a row, with room for the logits before an unaligned row's start
  int64_t span;     // parts of a CTA
  int64_t lists;    // CTAs of a row
};

Cut cut_of(int64_t rows, int64_t V, bool f32) {
  const int64_t vec = f32 ? 4 : 8, sms = sm_count();
  // as many vectors as leave at least four CTAs an SM, for fewer candidates and
  // one selection per more logits; at most kStreamBits logits of a thread.  Whole
  // calls with four, two and eight CTAs an SM: 64 rows of 32000 fp32 7.6, 8.4, 8.8
  // us, 16 of 128256 8.1, 7.8, 11.0
  Cut c{f32 ? 2 : 1, 0, 1, 0};
  for (int64_t nv = kStreamBits / vec; nv > c.nv; nv /= 2) {
    const int64_t per = kChunkThreads * nv * vec;
    if (rows * ((V + per - 1) / per) >= 4 * sms) c.nv = (int)nv;
  }
  const int64_t per = kChunkThreads * c.nv * vec;
  c.parts = (V + vec - 1 + per - 1) / per;
  if (c.nv * vec == kStreamBits) {
    // the CTAs that run at a time, whole rows where there are more of those.  512
    // rows of 128256: one CTA a row 54 us, two 66
    const int64_t most = 5 * sms, lists = rows < most ? most / rows : 1;
    c.span = (c.parts + lists - 1) / lists;
  }
  c.lists = (c.parts + c.span - 1) / c.span;
  return c;
}

size_t beam_bytes(int64_t rows, int64_t S, int n_out, size_t* cand_at) {
  const size_t part = ((size_t)rows * S * sizeof(float2) + 255) / 256 * 256;
  if (cand_at) *cand_at = part;
  return part + (size_t)rows * S * n_out * sizeof(uint64_t);
}

int check_sizes(int B, int W, int64_t V, int n_out) {
  if (B <= 0 || W <= 0 || V <= 0 || n_out <= 0) return TQ_ERR_ARG;
  if (W > kMaxBeams || n_out > kMaxBeams || V > 0x7fffffff / kMaxBeams)   // tokens in 26 bits, places in 31
    return TQ_ERR_UNSUPPORTED;
  if (n_out > W * V) return TQ_ERR_ARG;
  // parts are as small as 1024 logits
  if ((int64_t)B * W * (V / 1024 + 2) > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
  return TQ_OK;
}

template <bool F32>
bool launch_chunks(const BeamArgs& a, int nv, cudaStream_t st) {
  const int64_t grid = (int64_t)a.B * a.W * a.S;
  constexpr int MOST = kStreamBits / Vec<F32>::N;
  if (nv == MOST) return launch(beam_chunk_kernel<F32, MOST>, grid, kChunkThreads, false, st, a);
  if (nv == MOST / 2) return launch(beam_chunk_kernel<F32, MOST / 2>, grid, kChunkThreads, false, st, a);
  return launch(beam_chunk_kernel<F32, MOST / 4>, grid, kChunkThreads, false, st, a);
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
    const size_t n = tq::beam_bytes(rows, tq::cut_of(rows, V, f32).lists, n_out, nullptr);
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
  const tq::Cut cut = tq::cut_of(rows, V, f32);
  const int64_t S = cut.lists;
  size_t cand_at;
  if (!workspace || workspace_bytes < tq::beam_bytes(rows, S, n_out, &cand_at)) return TQ_ERR_WORKSPACE;
  if (!tq::aligned16(workspace)) return TQ_ERR_ALIGN;
  const tq::BeamArgs a{logits, row_stride, scores, done, eos, B, W, (int32_t)V, n_out, (int32_t)S, keep_place ? 1 : 0,
                       (int32_t)cut.parts, (int32_t)cut.span,
                       static_cast<float2*>(workspace),
                       reinterpret_cast<uint64_t*>(static_cast<uint8_t*>(workspace) + cand_at), out_scores, out_parent,
                       out_token, out_done};
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool ok = (f32 ? tq::launch_chunks<true>(a, cut.nv, s) : tq::launch_chunks<false>(a, cut.nv, s)) &&
                  tq::launch(tq::beam_pick_kernel, B, tq::kPickThreads, true, s, a);
  return ok && cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
