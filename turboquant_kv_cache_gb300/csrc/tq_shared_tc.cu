// Attention of a batch over one shared packed prefix and each sequence's own
// tokens on the tensor cores (tcgen05, TMEM accumulators): tq_decode_attn_shared
// for 1..4 bits without QJL.
//
// Rows: the B sequences' queries of one KV head, R = B*G rows (sequence b,
// head h -> row b*G + h), all of which attend to the same prefix.  A prefix CTA
// owns a tile of up to NR rows, one KV head and a slice of the prefix, which it
// walks in tiles of 128 tokens; its codes are decoded once for all its rows.
// The sequences' own tokens are the same work with other rows: a CTA then has
// one sequence, its G rows and a slice of its tokens.  Both kinds are one
// launch; every CTA writes a partial (m, l, O) per row, and the combine kernel
// joins a row's partials and turns O out of the rotated domain.
//
//   S^T [128 tokens x NR]  = K^ (A, smem, K-major) . Q^ (B, smem, K-major)
//   P^T                    = exp2(S^T - m), fp16, to shared memory
//   O^T [d x NR]          += V^ (A, smem, MN-major) . P^T (B, smem, MN-major)
//
// Tokens are on the 128 TMEM lanes and rows on the columns, so the tensor
// work and the softmax cost what the rows there are cost (a multiple of 32),
// not the 128 of a row-per-lane tile.  (Rows on the lanes with Q^ and P in
// TMEM reads less shared memory, but one thread then has 64 tokens of a row in
// sequence: 53.5 us against 52.2 us for 128 rows over 32768 tokens, 28.6
// against 26.1 us for 16.)  A softmax thread has one token's p for half of the
// rows; the sums l over tokens come from the same rounded p that multiplies V:
// two warps read P back as mma.sync operands and multiply it by a matrix of
// ones, in fp32.
// The reference of a row only moves when a score passes it by more than 2^10
// (it starts as the largest of 32 scores): the common step needs no maximum
// over tokens, only one barrier vote; the rare one takes the maxima and scales
// O and l.  What is kept as m lies 5 below the reference, so p is 2^5 there and
// at most 2^15: a part of fp16's range for what is larger, the rest for what is
// smaller.  (7 below and moves past 2^8: where scores have twice the unit
// deviation, 128 rows over 32768 tokens, references then move often enough to
// cost 55.5 us against 53.4; 3 and 2^12 53.3.)
//
// Roundings.  Scores, m, l and O are fp32.  Q^, K^ and V^ are rounded once to
// fp16 (half a step, 2^-11 relative to each value) and p once (2^-11): the
// tensor cores' operands, the same as the prefill's.  Their errors are
// independent over d values and over the tokens: with Gaussian vectors the
// outputs are 6e-4 to 9e-4 (relative, as norms) from attention in 64 bits, of
// which 2.1e-4 are the output's own rounding; a score of s (in e-folds) is off
// by up to 2^-10 sum |q k|, so weights of large scores by as much.  p is kept to
// 2^-30 of the reference's and dropped below: at most that per token, 2^-13 of a
// softmax over a slice of 131072 tokens.
//
// Warps: 0-7 softmax (warps 0-3 rows [0, NR/2), 4-7 the rest), which also
// rotate the queries while the first loads are in flight, 8 issues S, 9 issues
// O, 10 and 11 sum half of the rows each, 12-27 decode.  A decoder thread
// takes one 32-code group (two at head_dim 256) of the K tile and of the V
// tile, its packed words loaded a tile ahead; at head_dim 64 half of the
// decoder warps take K, half V.  Handoffs are mbarriers:
//   q_full      Q^ is written
//   kfull[b]    K^(t) is decoded; its buffer is free when S(t) is done
//   vfull[b]/vfree[b]  V^(t) is decoded / O(t) is done with it
//               (two buffers of each; one at head_dim 256)
//   s_full[i]   S(t), t & 1 = i, is in TMEM
//   p_full[i]   P(t) is written and S(t) has been read
//   o_done[i]   O += V(t) P(t) and l are done
// Every wait is bounded at two levels, as in tq_tc.cuh; a CTA that gives up
// stops decoding and issuing, waits for the products in flight and frees its
// TMEM.
//
// Measured (GB300; graph replays of the call, the combine in it).  128 rows
// over 32768 shared tokens and 512 own ones of 32 sequences, 8 KV heads,
// head_dim 128, 3 bits: 53.3 us for 40.9 MB of cache and 17.2 GFLOP (floors
// 6.1 and 8.8 us).  16 rows in 32 over 131072 shared tokens, 4 KV heads,
// head_dim 256, 4 and 3 bits: 78.9 us for 136 MB (floor 20.3 us).  Neither the
// memory nor the tensor cores bound it but the decode and the softmax on the
// way between them: at 128 rows a tile takes 3400 cycles, of which 2400 the
// softmax's exponentials, with issue slots 55 % and the shared-memory pipe
// 49 % busy over the kernel (the products' operand reads on top); at head_dim
// 256 it takes 4750, of which 2900 a decoder's two sides.  Sixteen softmax and
// eight decoder warps: 57.9 us against 54.7 before the query rotation's
// change.  Packed words through shared memory by asynchronous copies of 16
// bytes a thread 62.8, by bulk copies 69.3.  Two CTAs of half the size on an
// SM for 32 rows: as fast per tile (1.5 us against 1.4).
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>

#include "tq_device.cuh"
#include "tq_lut.cuh"
#include "tq_tc.cuh"

namespace tq {

int sm_count();

namespace {

using namespace tcq;

constexpr int kTile = 128;          // tokens per tile (MMA M of S^T)
constexpr int kSoftWarps = 8;
constexpr int kDecWarps = 16;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDec0 = 32 * (kSoftWarps + 4);          // first decoder thread (whole warpgroups)
constexpr int kThreadsSh = kDec0 + kDecThreads;       // 896
constexpr int kLaunchRegs = 72;     // registers a thread at launch (896 threads of 65536)
// log2 of p at a row's reference, and the log2 units a score may pass it by: p
// stays below 2^15, inside fp16, and sums of p * v inside fp32
constexpr float kHeadSh = 5.0f, kLazySh = 10.0f;

// first failure status of a launch since the last read (0 = none)
__device__ int g_shared_status;

template <int D>
struct ShCfg {
  static constexpr int NB = D == 256 ? 1 : 2;          // buffers of K and of V
  static constexpr int DV = D < 128 ? 128 : D;         // V tile width: whole M tiles of 128
  static constexpr int OT = DV / 128;                  // M tiles of O^T
  static constexpr int MAXR = D == 256 ? 64 : 128;     // rows of a CTA, by shared memory and registers
  static constexpr uint32_t KB = kTile * D * 2, VB = kTile * DV * 2;
  static constexpr int G8 = D / 32;                    // 32-code groups per token
  static constexpr bool SPLIT = D == 64;               // K and V on half of the decoder warps each
  static constexpr int SIDE = SPLIT ? kDecThreads / 2 : kDecThreads;   // threads on one side
  static constexpr int N = kTile * G8 / SIDE;          // groups per thread and side
  // registers of the softmax warps and of the others after the split: shares
  // of the launch's (a decoder thread of two groups needs the more)
  static constexpr int SOFT = N > 1 ? 88 : 104, OTHER = N > 1 ? 64 : 56;
  static_assert(32 * kSoftWarps * SOFT + (kThreadsSh - 32 * kSoftWarps) * OTHER <= kThreadsSh * kLaunchRegs,
                "the register split fits the launch's");
  static_assert(N * SIDE == kTile * G8, "every decoder thread has the same number of groups");
};

// One cache pair as the decoders read it.
struct Source {
  const uint8_t* kc;
  const uint8_t* ks;
  const uint8_t* vc;
  const uint8_t* vs;
  const int32_t* len;          // device lengths ([1] of the prefix, [B] of the sequences) or NULL
  PageMap pages;
  int64_t S_cap, ctx;
  int64_t per;                 // tokens per split (multiple of kTile)
  int splits, slot0;
  uint32_t div_mul, div_shift;   // unit / splits (FastDiv)
};

// n / d for n < 2^31 by a multiplication (d >= 1)
struct FastDiv {
  uint32_t mul, shift;   // mul 0: d is 1
};
FastDiv fast_div(uint32_t d) {
  if (d <= 1) return {0u, 0u};
  uint32_t l = 1;
  while (l < 31 && (1u << l) < d) ++l;   // 2^(l-1) < d <= 2^l
  return {(uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d), l - 1};
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, FastDiv f) { return f.mul ? __umulhi(n, f.mul) >> f.shift : n; }

struct SharedArgs {
  Source pre, own;
  const uint16_t* q;
  float* part;                 // [B*Hq][slots][D + 4]
  uint64_t report_ns, hard_ns;
  FastDiv by_heads;            // unit / Hkv
  int B, Hq, Hkv, G, lg, slots;   // G = 1 << lg
  int NR;                      // rows of a prefix CTA (multiple of 32)
  int row_tiles;               // prefix CTAs along the rows
  int n_pre;                   // prefix CTAs, ahead of the sequences' own
  float qscale;
};

#define TQ_LD4(taddr, v)                                                                       \
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];\n"                 \
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])                               \
               : "r"(taddr))
#define TQ_LD16(taddr, v)                                                                                          \
  asm volatile(                                                                                                    \
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n"    \
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),            \
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])       \
      : "r"(taddr))

__device__ __forceinline__ void ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ void st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
__device__ __forceinline__ float ex2s(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void sts16b(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
// barrier of one half of the softmax warps (128 threads), alone or with a vote
__device__ __forceinline__ void half_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool half_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n barrier.cta.red.or.pred p, %2, 128, q;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_init(uint32_t bar, int count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ bool bar_done(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}
// Wait of a whole warp for a phase of an mbarrier: one poll and a vote when it
// has completed.  Otherwise try_wait suspends the warp until it completes (no
// sleep between polls: a handoff of this kernel is due within a microsecond);
// past report_ns of wall time it sets `late` and goes on, past hard_ns, or
// once the CTA has given up, it returns false.
__device__ __forceinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, uint64_t report_ns, uint64_t hard_ns,
                                           volatile int& abort, int& late) {
  const uint64_t t0 = global_ns();
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
    const uint64_t el = global_ns() - t0;
    if (el > report_ns) late = 1;
    if (__all_sync(kFull, done)) return true;
    if (__any_sync(kFull, el > hard_ns || abort)) {
      abort = 1;
      return false;
    }
  }
}
// maximum over the warp, in every lane
__device__ __forceinline__ float warp_max_f(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// D += ones B for a 16 x 8 block of B (every row of D: the sums of its columns)
__device__ __forceinline__ void hmma_sum(float* d, uint32_t b0, uint32_t b1) {
  const uint32_t one = 0x3C003C00u;
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%4,%4,%4}, {%5,%6}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(one), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void ldsm4_trans(uint32_t* v, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// The packed words and norm of one 32-code group, loaded a tile ahead.
struct Group {
  uint32_t w[4];
  uint32_t sc;
};

// A group's packed words as the 8-byte word at or 4 bytes before it and, past
// two bits, the next one: the same two loads whatever the bit width, with no
// branch or predicate, so that no load is waited for at a join.  Groups of
// 4 * bits bytes come in pairs that start on 8 bytes (d / 32 is even), so both
// words lie in the record.  1 and 3 bits: an odd group starts with the second
// 4-byte word (`shifted`).
__device__ __forceinline__ void load_group_g(const uint8_t* c8, int next, const uint8_t* s, Group& g) {
  asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(g.w[0]), "=r"(g.w[1]) : "l"(c8));
  asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(g.w[2]), "=r"(g.w[3]) : "l"(c8 + next));
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(g.sc) : "l"(s));
}

// Keeps what is computed from a group behind this point: otherwise the first
// steps of its decode are scheduled right after its loads, a tile too early,
// and wait for them there.
__device__ __forceinline__ void pin(Group& g) {
  asm volatile("" : "+r"(g.w[0]), "+r"(g.w[1]), "+r"(g.w[2]), "+r"(g.w[3]), "+r"(g.sc));
}

// Four fp16x2 registers of a nibble word of 4-bit codes.  The codebook is
// symmetric, c(15 - k) = -c(k): the upper eight levels in the byte tables, a
// lower code looked up as 15 - k and its sign bit set in the high byte.
__device__ __forceinline__ void lut8_sym(uint32_t n, const Tab& T, uint32_t* o) {
  const uint32_t low = ~n & 0x88888888u;                        // nibbles of lower codes
  const uint32_t idx = (n ^ (low - (low >> 3))) & 0x77777777u;  // their three bits flipped
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint32_t s = half ? __umulhi(idx, 1u << 16) : idx;
    const uint32_t b = half ? n >> 17 : n >> 1;   // bit 3 of each code as bit 2 of a byte selector
    const uint32_t lo = lut_prmt(T.t[0], T.t[1], s);
    const uint32_t neg = lut_prmt(0xffffffffu, 0u, b);
    const uint32_t hi = lut_prmt(T.t[2], T.t[3], s) ^ (neg & 0x80808080u);
    o[2 * half] = lut_prmt(lo, hi, 0x5140);
    o[2 * half + 1] = lut_prmt(lo, hi, 0x7362);
  }
}

// A thread's N groups, 32 values each (centroid * norm, fp16), to the
// core-matrix tile: four 16-byte chunks, one per core matrix.  Each (token,
// block) table holds the fp32 products of centroids and norm, rounded once to
// fp16.  A token past the slice (not live) takes norm 0: zero rows, since 0 * p
// must be 0.  One branch on the bit width around all groups, so that their
// instructions interleave.
template <int BITS, int N>
__device__ __forceinline__ void decode_groups_b(const Group* g, bool shifted, const float* cent, const bool* live,
                                                uint32_t dst, uint32_t step) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    uint32_t n[4];
    if (BITS & 1) {
      const uint32_t w3[3] = {shifted ? g[k].w[1] : g[k].w[0], shifted ? g[k].w[2] : g[k].w[1],
                              shifted ? g[k].w[3] : g[k].w[2]};
      chunk_words<BITS>(w3, n);
    } else {
      chunk_words<BITS>(g[k].w, n);
    }
    const float norm = live[k] ? h2f((uint16_t)g[k].sc) : 0.f;
    const Tab T = make_tab_f32<BITS == 4 ? 3 : BITS>(BITS == 4 ? cent + 8 : cent, norm);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t o[4];
      if (BITS == 4) lut8_sym(n[c], T, o);
      else lut8<BITS>(n[c], T, o);
      sts16b(dst + k * step + 128 * c, o[0], o[1], o[2], o[3]);
    }
  }
}

template <int N>
__device__ __forceinline__ void decode_groups(int bits, const Group* g, bool odd, const float* cent, const bool* live,
                                              uint32_t dst, uint32_t step) {
  switch (bits) {
    case 4: decode_groups_b<4, N>(g, odd, cent, live, dst, step); break;
    case 3: decode_groups_b<3, N>(g, odd, cent, live, dst, step); break;
    case 2: decode_groups_b<2, N>(g, odd, cent, live, dst, step); break;
    default: decode_groups_b<1, N>(g, odd, cent, live, dst, step); break;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreadsSh, 1) shared_prefix_kernel(const CodecParams PK, const CodecParams PV,
                                                                      const __grid_constant__ SharedArgs a) {
  using C = ShCfg<D>;
  constexpr int NB = C::NB, OT = C::OT;
  constexpr uint32_t kKGroup = (D / 8) * 128;       // bytes of 8 tokens of K, 8 rows of Q
  constexpr uint32_t kVGroup = (C::DV / 8) * 128;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[3 * NB + 8];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int s_abort;
  __shared__ int s_late;
  __shared__ __align__(16) float s_m[C::MAXR];      // kHeadSh below the rows' softmax references
  __shared__ float s_al[C::MAXR];
  __shared__ int64_t s_dst[C::MAXR];                // where the rows' partials go
  __shared__ __align__(8) float s_l[C::MAXR];                    // the rows' sums of p

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // a prefix CTA: split fastest, then KV head, then row tile; behind them a
  // sequence's own: split, KV head, sequence
  const bool pre = (int)blockIdx.x < a.n_pre;
  const Source& src = pre ? a.pre : a.own;
  const uint32_t unit = pre ? blockIdx.x : blockIdx.x - a.n_pre;
  const uint32_t unit_h = div_by(unit, {src.div_mul, src.div_shift}), unit_z = div_by(unit_h, a.by_heads);
  const int split = unit - unit_h * src.splits, kvh = unit_h - unit_z * a.Hkv, grp_z = unit_z;
  const int NR = pre ? a.NR : 32;
  const int row0 = pre ? grp_z * a.NR : grp_z * a.G;
  const int rows = pre ? min(NR, a.B * a.G - row0) : a.G;
  const int seq = pre ? 0 : grp_z;
  const int slot = src.slot0 + split;
  int64_t len = src.ctx;
  if (src.len) len = imin64(len, (int64_t)src.len[seq]);
  const int64_t t_lo = (int64_t)split * src.per;
  const int64_t t_hi = imin64(t_lo + src.per, len);
  const int n_tok = t_hi > t_lo ? (int)(t_hi - t_lo) : 0;
  const int n_tiles = (n_tok + kTile - 1) / kTile;

  // P(t) is written once O(t - 2) and l are done with its buffer: up to 64 rows
  // S(t) is issued only then, so that a softmax warp has one wait a tile (16
  // rows, head_dim 256: 77.0 us against 78.7); past them the sums take longer
  // and the softmax waits itself (128 rows: 52.5 us against 54.2)
  const bool s_waits = NR <= 64;
  // K, V buffers, Q^, two P buffers
  const uint32_t pbytes = (uint32_t)NR * kTile * 2;
  const uint32_t aK = su32(smem), aV = aK + NB * C::KB, aQ = aV + NB * C::VB, aP = aQ + (uint32_t)NR * D * 2;
  const uint32_t b0 = su32(&bars[0]);
  const uint32_t q_full = b0, s_full = b0 + 8, p_full = b0 + 24, o_done = b0 + 40, drained = b0 + 56,
                 kfull = b0 + 64, vfull = kfull + 8 * NB, vfree = vfull + 8 * NB;
  // TMEM columns: S twice, then O
  const uint32_t cO = 2u * NR;
  const uint32_t tused = cO + (uint32_t)OT * NR;
  const uint32_t tcols = tused > 256 ? 512u : (tused > 128 ? 256u : 128u);

  auto wait = [&](uint32_t bar, uint32_t parity) -> bool {
    if (__all_sync(kFull, bar_done(bar, parity))) return true;
    int late = 0;
    const bool ok = bar_wait_slow(bar, parity, a.report_ns, a.hard_ns, s_abort, late);
    if (late) s_late = 1;
    return ok;
  };

  // ---- before the CTA's first barrier: each role's own preparations
  if (warp == kSoftWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(&tmem_base)),
                 "r"(tcols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  } else if (tid == 32 * (kSoftWarps + 1)) {
    s_abort = 0;
    s_late = 0;
    constexpr int kSide = C::SIDE / 32;   // decoder warps that fill one side
    bar_init(q_full, kSoftWarps);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      bar_init(s_full + 8 * i, 1);
      bar_init(p_full + 8 * i, kSoftWarps);
      bar_init(o_done + 8 * i, 3);   // the product's commit and the two summing warps
    }
    bar_init(drained, 2);
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      bar_init(kfull + 8 * i, kSide);
      bar_init(vfull + 8 * i, kSide);
      bar_init(vfree + 8 * i, 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  } else if (tid < NR) {
    const int r = row0 + tid;
    s_m[tid] = -INFINITY;
    s_l[tid] = 0.f;
    s_dst[tid] = (((int64_t)(r >> a.lg) * a.Hq + kvh * a.G + (r & (a.G - 1))) * a.slots + slot) * (D + 4);
  }
  uint32_t tmem;
  auto begin = [&]() {   // every warp, once
    fence_before();
    asm volatile("bar.sync 0;\n" ::: "memory");
    fence_after();
    tmem = tmem_base;
  };

  // Q^ = H D q per K block, times softmax_scale * log2 e, by the softmax warps:
  // a lane has 32 values of one row, a warp QR = 1024 / D rows at a time, the
  // rows on consecutive lanes, so that eight lanes write one core matrix.
  constexpr int QL = D / 32, QR = 32 / QL;
  uint4 qv[4];
  auto fetch_query = [&](int i) {   // rows [QR * i, QR * (i + 1))
    const int r = QR * i + lane % QR;
#pragma unroll
    for (int e = 0; e < 4; ++e) qv[e] = make_uint4(0u, 0u, 0u, 0u);
    if (r < rows) {
      const int rr = row0 + r, b = rr >> a.lg, h = kvh * a.G + (rr & (a.G - 1));
      const uint4* qr = reinterpret_cast<const uint4*>(a.q + ((int64_t)b * a.Hq + h) * D + 32 * (lane / QR));
#pragma unroll
      for (int e = 0; e < 4; ++e) qv[e] = qr[e];
    }
  };
  auto rotate_queries = [&](int w) {   // after fetch_query(w)
    const float qn = PK.inv_sqrt_blk * a.qscale;
    const uint32_t sb = PK.sign_bits[lane / QR];
#pragma unroll 1
    for (int i = w; QR * i < NR; i += kSoftWarps) {
      float v[32];
#pragma unroll
      for (int e = 0; e < 32; e += 2) {
        const uint4& x = qv[e >> 3];
        const uint32_t u = (e & 6) == 0 ? x.x : (e & 6) == 2 ? x.y : (e & 6) == 4 ? x.z : x.w;
        const uint32_t us = u ^ ((sb >> e & 1u) << 15 | (sb >> (e + 1) & 1u) << 31);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&us));
        v[e] = f.x * qn;
        v[e + 1] = f.y * qn;
      }
      fetch_query(i + kSoftWarps);
#pragma unroll
      for (int hs = 1; hs < 32; hs <<= 1) {   // blocks are 32 values at least
#pragma unroll
        for (int e = 0; e < 32; ++e)
          if ((e & hs) == 0) {
            const float p = v[e], q = v[e + hs];
            v[e] = p + q;
            v[e + hs] = p - q;
          }
      }
#pragma unroll 1
      for (int hs = 32; hs < PK.blk; hs <<= 1) {
        const int lo = hs / 32 * QR;
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const float p = __shfl_xor_sync(kFull, v[e], lo);
          v[e] = (lane & lo) ? (p - v[e]) : (v[e] + p);
        }
      }
      const uint32_t dst = aQ + cm_off(QR * i + lane % QR, 32 * (lane / QR), D);
#pragma unroll
      for (int c = 0; c < 4; ++c)
        sts16b(dst + 128 * c, pack2(v[8 * c], v[8 * c + 1]), pack2(v[8 * c + 2], v[8 * c + 3]),
               pack2(v[8 * c + 4], v[8 * c + 5]), pack2(v[8 * c + 6], v[8 * c + 7]));
    }
    fence_async_smem();
    __syncwarp();
    if (lane == 0) arrive(q_full);
  };

  if (warp >= kSoftWarps) {
    // whole warpgroups (4 warps) execute one instruction each
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(C::OTHER));
    if (warp >= kDec0 / 32) {
      // ================= decoders
      if (n_tiles == 0) {
        begin();
      } else {
        const int dt = tid - kDec0;
        const int st = C::SPLIT ? dt % C::SIDE : dt;    // thread within its side
        const bool do_k = !C::SPLIT || dt < C::SIDE, do_v = !C::SPLIT || dt >= C::SIDE;
        // the thread's groups: number grp of the tokens tok0 and, at head_dim
        // 256, kStep tokens on.  A group's number turns with its token, so that
        // the eight lanes of one access hit different banks whatever the
        // records' pitch.
        constexpr int kStep = C::SIDE / C::G8;
        static_assert(C::N == 1 || kStep % 8 == 0, "a thread's groups have one number");
        const int tok0 = 8 * (st / (8 * C::G8)) + (st & 7), grp = ((st >> 3) + (C::G8 == 8 ? st : st >> 1)) % C::G8;
        const bool odd = grp & 1;
        const int kbits = PK.bits, vbits = PV.bits;
        const bool paged = src.pages.table != nullptr;
        const uint32_t kwb = PK.code_bytes, vwb = PV.code_bytes, knb = 2 * PK.nb, vnb = 2 * PV.nb;
        const uint32_t kw0 = grp * 4 * kbits - ((kbits & 1) && odd ? 4 : 0), kn0 = 32 * grp / PK.blk * 2;
        const uint32_t vw0 = grp * 4 * vbits - ((vbits & 1) && odd ? 4 : 0), vn0 = 32 * grp / PV.blk * 2;
        const int knext = kbits > 2 ? 8 : 0, vnext = vbits > 2 ? 8 : 0;
        const int64_t rec0 = paged ? 0 : ((int64_t)seq * a.Hkv + kvh) * src.S_cap + t_lo;
        const uint8_t *kc = src.kc + rec0 * kwb + kw0, *ks = src.ks + rec0 * knb + kn0;
        const uint8_t *vc = src.vc + rec0 * vwb + vw0, *vs = src.vs + rec0 * vnb + vn0;
        const int32_t* table = paged ? src.pages.table + (int64_t)seq * src.pages.pages_per_seq : nullptr;
        const uint32_t psize = src.pages.page_size;
        const int last_page = paged ? ((uint32_t)t_lo + n_tok - 1) / psize : 0;
        // record (contiguous: token) of each group in the tile to be loaded; a
        // token past the slice takes the last one's place (paged: some record
        // of the last page), and its values are not used
        int32_t page[C::N], off[C::N];
        int64_t rec[C::N];
#pragma unroll
        for (int k = 0; k < C::N; ++k) {
          const uint32_t t = (uint32_t)t_lo + tok0 + k * kStep;
          page[k] = paged ? t / psize : 0;
          off[k] = paged ? t - page[k] * psize : 0;
        }
        auto place = [&](int at) {   // the records of the tile `at` tokens into the slice
#pragma unroll
          for (int k = 0; k < C::N; ++k) {
            if (paged) {
              rec[k] = ((int64_t)table[min(page[k], last_page)] * a.Hkv + kvh) * psize + off[k];
              off[k] += kTile;
              while ((uint32_t)off[k] >= psize) {
                off[k] -= psize;
                ++page[k];
              }
            } else {
              rec[k] = min(at + tok0 + k * kStep, n_tok - 1);
            }
          }
        };
        Group gk[C::N], gv[C::N];
        auto load_k = [&]() {
#pragma unroll
          for (int k = 0; k < C::N; ++k) load_group_g(kc + rec[k] * kwb, knext, ks + rec[k] * knb, gk[k]);
        };
        auto load_v = [&]() {
#pragma unroll
          for (int k = 0; k < C::N; ++k) load_group_g(vc + rec[k] * vwb, vnext, vs + rec[k] * vnb, gv[k]);
        };
        place(0);
        load_k();
        load_v();
        begin();
        for (int t = 0; t < n_tiles; ++t) {
          const int bf = t % NB, at = t * kTile;
          bool live[C::N];
#pragma unroll
          for (int k = 0; k < C::N; ++k) live[k] = at + tok0 + k * kStep < n_tok;
          if (do_k) {
            if (t >= NB) wait(s_full + 8 * ((t - NB) & 1), (uint32_t)((t - NB) >> 1) & 1);   // S(t - NB) is done
#pragma unroll
            for (int k = 0; k < C::N; ++k) pin(gk[k]);
            if (!s_abort)
              decode_groups<C::N>(kbits, gk, odd, PK.centroids, live, aK + bf * C::KB + cm_off(tok0, 32 * grp, D),
                                  cm_off(kStep, 0, D));
            fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive(kfull + 8 * bf);
            place(at + kTile);
            load_k();
          }
          if (do_v) {
            if (t >= NB) wait(vfree + 8 * bf, (uint32_t)(t / NB - 1) & 1);
#pragma unroll
            for (int k = 0; k < C::N; ++k) pin(gv[k]);
            if (!s_abort)
              decode_groups<C::N>(vbits, gv, odd, PV.centroids, live, aV + bf * C::VB + cm_off(tok0, 32 * grp, C::DV),
                                  cm_off(kStep, 0, C::DV));
            fence_async_smem();
            __syncwarp();
            if (lane == 0) arrive(vfull + 8 * bf);
            if (C::SPLIT) place(at + kTile);
            load_v();
          }
        }
      }
    } else if (warp == kSoftWarps) {
      // ================= S^T(t) = K^(t) Q^
      begin();
      const uint32_t idesc = (1u << 4) | ((uint32_t)(NR >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
      const uint64_t dq = sdesc(aQ, 128, kKGroup);
      bool ok = n_tiles > 0 && wait(q_full, 0);
      for (int t = 0; t < n_tiles && ok; ++t) {
        const int bf = t % NB;
        ok = wait(kfull + 8 * bf, (uint32_t)(t / NB) & 1) &&
             (t < 2 || wait((s_waits ? o_done : p_full) + 8 * (t & 1), (uint32_t)((t >> 1) - 1) & 1));
        if (!ok) break;
        fence_after();
        __syncwarp();
        const uint64_t dk = sdesc(aK + bf * C::KB, 128, kKGroup);
#pragma unroll
        for (int s = 0; s < D / 16; ++s)
          mma_ss_elect(tmem + (t & 1) * NR, dk + (uint64_t)(16 * s), dq + (uint64_t)(16 * s), idesc, s > 0);
        commit_elect(s_full + 8 * (t & 1));
      }
      __syncwarp();
      commit_elect(drained);
    } else if (warp == kSoftWarps + 1) {
      // ================= O^T += V^(t)^T P(t)^T
      begin();
      const uint32_t idesc = (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(NR >> 3) << 17) |
                             ((uint32_t)(128 >> 4) << 24);
      const uint32_t pg = (uint32_t)(NR >> 3) * 128;   // bytes of 8 tokens of P
      for (int t = 0; t < n_tiles; ++t) {
        const int vb = t % NB, pb = t & 1;
        if (!wait(vfull + 8 * vb, (uint32_t)(t / NB) & 1)) break;
        if (!wait(p_full + 8 * pb, (uint32_t)(t >> 1) & 1)) break;
        fence_after();
        __syncwarp();
        const uint64_t dp = sdesc(aP + pb * pbytes, pg, 128);
#pragma unroll
        for (int m = 0; m < OT; ++m) {
          const uint64_t dv = sdesc(aV + vb * C::VB + m * 16 * 128, kVGroup, 128);
#pragma unroll
          for (int s = 0; s < kTile / 16; ++s)
            mma_ss_elect(tmem + cO + m * NR, dv + (uint64_t)(s * (2 * kVGroup >> 4)),
                         dp + (uint64_t)(s * (2 * pg >> 4)), idesc, t > 0 || s > 0);
        }
        commit_elect(o_done + 8 * pb);
        commit_elect(vfree + 8 * vb);
      }
      __syncwarp();
      commit_elect(drained);
    } else {
      // ================= l += ones P(t)^T: rows [0, NR/2) or the rest, 8 at a time
      begin();
      const int nc = NR / 2, col0 = (warp - kSoftWarps - 2) * nc;
      // lane i's row of the four 8 x 8 matrices of 32 tokens: token i, 8 rows
      const uint32_t row = cm_off(lane, col0, NR);
      const uint32_t step = (uint32_t)(NR >> 3) * 512;   // 32 tokens on
      for (int t = 0; t < n_tiles; ++t) {
        const int pb = t & 1;
        if (!wait(p_full + 8 * pb, (uint32_t)(t >> 1) & 1)) break;
        __syncwarp();
        for (int c = 0; c < nc; c += 16) {   // two blocks of 8 rows, four chains of products
          float d[2][2][4] = {};
          const uint32_t at = aP + pb * pbytes + row + (uint32_t)(c >> 3) * 128;
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t b[4];
              ldsm4_trans(b, at + k * step + x * 128);
              hmma_sum(d[x][0], b[0], b[1]);
              hmma_sum(d[x][1], b[2], b[3]);
            }
          if (lane < 4) {   // columns 2 lane, 2 lane + 1 of each block
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              float2* l = reinterpret_cast<float2*>(&s_l[col0 + c + 8 * x + 2 * lane]);
              const float2 o = *l;
              *l = make_float2(o.x + (d[x][0][0] + d[x][1][0]), o.y + (d[x][0][1] + d[x][1][1]));
            }
          }
        }
        __syncwarp();
        if (lane == 0) arrive(o_done + 8 * pb);
      }
    }
  } else {
    // ================= softmax: thread = token (TMEM lane) x half of the rows
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(C::SOFT));
    if (n_tiles > 0) fetch_query(warp);
    begin();
    if (n_tiles > 0) rotate_queries(warp);
    const int quarter = warp & 3, half = warp >> 2, bid = 1 + half;
    const int nc = NR / 2, col0 = half * nc;
    const int tk = 32 * quarter + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t pdst0 = aP + cm_off(tk, col0, NR);
    constexpr int NCH = C::MAXR / 32;       // column chunks of 16
    const uint32_t kOver = 0x78007800u;     // 2^15 twice in fp16
    static_assert(kHeadSh + kLazySh == 15.0f, "kOver is p where the reference moves");
    for (int t = 0; t < n_tiles; ++t) {
      const uint32_t sS = lanes + (t & 1) * NR + col0;
      const uint32_t pdst = pdst0 + (t & 1) * pbytes;
      const bool whole = (t + 1) * kTile <= n_tok, live = t * kTile + tk < n_tok;
      // p of every column from its score, to P; returns whether one passes
      // 2^15.  A token past the slice has p = 0.
      auto emit = [&]() {
        uint32_t vv[2][16], mx = 0u;
        TQ_LD16(sS, vv[0]);
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          if (16 * i >= nc) break;
          uint32_t o[8];
          uint32_t* v = vv[i & 1];
          ld_wait();
          if (16 * (i + 1) < nc) TQ_LD16(sS + 16 * (i + 1), vv[(i + 1) & 1]);   // in flight during this chunk
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 m = *reinterpret_cast<const float4*>(&s_m[col0 + 16 * i + j]);
            o[j / 2] = pack2(ex2s(__uint_as_float(v[j]) - m.x), ex2s(__uint_as_float(v[j + 1]) - m.y));
            o[j / 2 + 1] = pack2(ex2s(__uint_as_float(v[j + 2]) - m.z), ex2s(__uint_as_float(v[j + 3]) - m.w));
          }
          if (!whole) {
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = live ? o[j] : 0u;
          }
          mx = hmax2(mx, hmax2(hmax2(hmax2(o[0], o[1]), hmax2(o[2], o[3])), hmax2(hmax2(o[4], o[5]), hmax2(o[6], o[7]))));
          sts16b(pdst + 256 * i, o[0], o[1], o[2], o[3]);
          sts16b(pdst + 256 * i + 128, o[4], o[5], o[6], o[7]);
        }
        return hmax2(mx, kOver) != kOver;
      };
      wait(s_full + 8 * (t & 1), (uint32_t)(t >> 1) & 1);
      if (!s_waits && t >= 2) wait(o_done + 8 * (t & 1), (uint32_t)((t >> 1) - 1) & 1);
      fence_after();
      __syncwarp();
      if (t == 0) {
        // the first references: a row's largest score over 32 tokens, each
        // quarter's tokens for a quarter of the rows
        for (int c = 4 * quarter; c < nc; c += 16) {
          uint32_t v[4];
          TQ_LD4(sS + c, v);
          ld_wait();
          float mine = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x = warp_max_f(live ? __uint_as_float(v[j]) : -INFINITY);
            if (lane == j) mine = x;
          }
          if (lane < 4) s_m[col0 + c + lane] = mine - kHeadSh;
        }
        half_sync(bid);
      }
      if (half_any(bid, emit())) {
        // some row's reference moves: its maximum over the tile, O and l
        // scaled, P written again
        if (t >= 1) {
          wait(o_done + 8 * ((t - 1) & 1), (uint32_t)((t - 1) >> 1) & 1);   // O and l stand still
          fence_after();
        }
        __syncwarp();
        // the maxima by TMEM lane quarter, in this half's part of the first
        // eight tokens of P(t), which is written again below
        float* wm = reinterpret_cast<float*>(smem + (aP - aK) + (t & 1) * pbytes + (col0 >> 3) * 128);
        for (int c = 0; c < nc; c += 16) {
          uint32_t v[16];
          TQ_LD16(sS + c, v);
          ld_wait();
          float mine = 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float x = warp_max_f(live ? __uint_as_float(v[j]) : -INFINITY);
            if (lane == j) mine = x;
          }
          if (lane < 16) wm[quarter * nc + c + lane] = mine;
        }
        half_sync(bid);
        if ((tid & 127) < nc) {
          const int i = tid & 127, r = col0 + i;
          const float x = fmaxf(fmaxf(wm[i], wm[nc + i]), fmaxf(wm[2 * nc + i], wm[3 * nc + i]));
          const float mo = s_m[r], mn = x > mo + (kHeadSh + kLazySh) || mo == -INFINITY ? x - kHeadSh : mo;
          const float al = mo == -INFINITY ? 0.f : ex2s(mo - mn);
          s_m[r] = mn;
          s_al[r] = al;
          s_l[r] *= al;
        }
        half_sync(bid);
        if (t >= 1) {
#pragma unroll 1
          for (int m = 0; m < OT; ++m) {
#pragma unroll 1
            for (int c = 0; c < nc; c += 16) {
              uint32_t v[16];
              const uint32_t at = lanes + cO + m * NR + col0 + c;
              TQ_LD16(at, v);
              ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * s_al[col0 + c + j]);
              TQ_ST16(at, v);
            }
          }
          st_wait();
        }
        emit();
      }
      fence_async_smem();
      fence_before();
      __syncwarp();
      if (lane == 0) arrive(p_full + 8 * (t & 1));
    }
  }
  // the next kernel may be scheduled; it waits for this grid before it ends
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  __syncthreads();
  if (n_tiles > 0) wait(o_done + 8 * ((n_tiles - 1) & 1), (uint32_t)((n_tiles - 1) >> 1) & 1);
  fence_after();
  // partials: lane = dimension of O^T, column = row; six groups of four warps
  // (a TMEM lane quarter each) take 16 columns of one M tile at a time
  const bool ok = n_tiles > 0 && !__any_sync(kFull, s_abort);
  if (warp < 24) {
    const int quarter = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    for (int w = warp >> 2; w < OT * (NR / 16); w += 6) {
      const int m = OT > 1 ? w % OT : 0, c = w / OT * 16;
      uint32_t v[16];
      if (ok) {
        TQ_LD16(lanes + cO + m * NR + c, v);
        ld_wait();
      }
      const int dim = 128 * m + 32 * quarter + lane;
      float* base = a.part + 2 + dim;
      if (dim < D) {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (c + j < rows) base[s_dst[c + j]] = ok ? __uint_as_float(v[j]) : 0.f;
      }
    }
  } else {
    for (int r = tid - 24 * 32; r < rows; r += kThreadsSh - 24 * 32)
      *reinterpret_cast<float2*>(a.part + s_dst[r]) = make_float2(ok ? s_m[r] : -INFINITY, ok ? s_l[r] : 0.f);
  }
  fence_before();
  __syncthreads();
  if (warp == kSoftWarps) {
    fence_after();
    // every product has been committed and, on the normal path, has ended
    if (!__all_sync(kFull, bar_done(drained, 0))) {
      int late = 0;
      s_abort = 0;   // the others have left: wait for the products themselves
      __syncwarp();
      if (!bar_wait_slow(drained, 0, a.report_ns, a.hard_ns, s_abort, late) || late) s_late = 1;
    }
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(tcols) : "memory");
    if (lane == 0 && (s_abort || s_late)) atomicCAS(&g_shared_status, 0, (int)TQ_ERR_TIMEOUT);
  }
}

template <int D>
size_t shared_smem(int NR) {
  using C = ShCfg<D>;
  return (size_t)C::NB * (C::KB + C::VB) + (size_t)NR * D * 2 + (size_t)2 * NR * kTile * 2;
}

template <int D>
int launch_shared(const CodecParams& PK, const CodecParams& PV, const SharedArgs& a, unsigned grid, cudaStream_t st) {
  const size_t sm = shared_smem<D>(a.n_pre ? a.NR : 32);
  auto kern = shared_prefix_kernel<D>;
  // once per device; a build with fewer registers than the split shares out
  // would wait for them without end, so it is refused
  static std::atomic<bool> ready[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TQ_ERR_CUDA;
  if (!ready[dev].load(std::memory_order_acquire)) {
    cudaFuncAttributes fa;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared_smem<D>(ShCfg<D>::MAXR)) ||
        cudaFuncGetAttributes(&fa, kern) || fa.numRegs < kLaunchRegs)
      return TQ_ERR_CUDA;
    ready[dev].store(true, std::memory_order_release);
  }
  kern<<<grid, kThreadsSh, sm, st>>>(PK, PV, a);
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}

// Row tiles of R rows and the rows each has (a multiple of 32).
void shared_rows(int d, int64_t R, int* tiles, int* NR) {
  const int most = d == 256 ? ShCfg<256>::MAXR : ShCfg<128>::MAXR;
  *tiles = (int)((R + most - 1) / most);
  *NR = (int)(((R + *tiles - 1) / *tiles + 31) / 32 * 32);
}

Source source_of(const tq_kv_view* K, const tq_kv_view* V, const int32_t* len, int64_t S_cap, int64_t ctx, int splits,
                 int slot0) {
  Source s{};
  s.kc = K->codes;
  s.ks = reinterpret_cast<const uint8_t*>(K->scales);
  s.vc = V->codes;
  s.vs = reinterpret_cast<const uint8_t*>(V->scales);
  s.len = len;
  s.pages = {K->page_table, K->page_table ? K->page_size : 0, K->page_table ? K->pages_per_seq : 0};
  s.S_cap = S_cap;
  s.ctx = ctx;
  const int64_t tiles = (ctx + kTile - 1) / kTile;
  s.per = (tiles + splits - 1) / splits * kTile;
  s.splits = splits;
  const FastDiv f = fast_div((uint32_t)splits);
  s.div_mul = f.mul;
  s.div_shift = f.shift;
  s.slot0 = slot0;
  return s;
}

}  // namespace

// Layouts the tensor-core kernel takes: 1..4 bits without QJL.
bool shared_tc_eligible(const CodecParams& PK, const CodecParams& PV) {
  return !PK.m && !PV.m && PK.bits <= 4 && PV.bits <= 4;
}

// Splits of the prefix and of each sequence's own tokens.  An SM holds one CTA
// at a time and a CTA's start and end cost about two tiles (kSetup), so there
// are two ways.  One wave: every CTA on an SM of its own, with the fewest
// tiles at which they all have one.  Or the prefix over all SMs and the own
// tokens in waves behind it, which is shorter when there is much prefix or
// there are many sequences.
// 7 sequences of 333 tokens, 2011 shared ones, 8 KV heads at head_dim 64: one
// wave of 3 tiles 10.6 us, two of 1 and 2 tiles 15.6 us.  8 sequences of 256 and
// 131072 shared ones, 4 KV heads at head_dim 256: one wave of 35 tiles 93.6 us,
// two of 27 and 1 tiles 82.8 us.
void shared_tc_splits(int d, int B, int G, int Hkv, int64_t prefix_ctx, int64_t ctx, int* n_prefix, int* n_own) {
  constexpr int64_t kSetup = 2;
  int row_tiles, NR;
  shared_rows(d, (int64_t)B * G, &row_tiles, &NR);
  const int64_t sms = sm_count(), up = (int64_t)row_tiles * Hkv, uo = (int64_t)B * Hkv;
  const int64_t tp = (prefix_ctx + kTile - 1) / kTile, to = (ctx + kTile - 1) / kTile;
  auto parts = [](int64_t tiles, int64_t most) { return most > 0 ? (tiles + most - 1) / most : 0; };
  auto waves = [&](int64_t units, int64_t ns, int64_t tiles) {
    return ns > 0 ? parts(units * ns, sms) * (parts(tiles, ns) + kSetup) : 0;
  };
  // the prefix over all SMs, then the own tokens
  const int64_t np = tp > 0 ? imin64(tp, up < sms ? sms / up : 1) : 0;
  int64_t no = to > 0 ? 1 : 0;
  for (int64_t n = 2; n <= imin64(to, 64) && uo * n <= 2 * sms; ++n)
    if (waves(uo, n, to) < waves(uo, no, to)) no = n;
  const int64_t two = waves(up, np, tp) + waves(uo, no, to);
  *n_prefix = (int)np;
  *n_own = (int)no;
  // one wave of CTAs of at most `most` tiles
  auto fits = [&](int64_t most) { return up * parts(tp, most) + uo * parts(to, most) <= sms; };
  int64_t lo = 1, hi = tp > to ? tp : to;
  if (hi < 1 || !fits(hi)) return;
  while (lo < hi) {
    const int64_t mid = (lo + hi) / 2;
    if (fits(mid)) hi = mid;
    else lo = mid + 1;
  }
  if (lo + kSetup > two) return;
  *n_prefix = (int)parts(tp, lo);
  *n_own = (int)parts(to, lo);
}

// At least the splits above, and no fewer for longer lengths: a workspace for
// the longest lengths serves shorter ones.
void shared_tc_most_splits(int d, int B, int G, int Hkv, int64_t prefix_ctx, int64_t ctx, int* n_prefix, int* n_own) {
  int row_tiles, NR;
  shared_rows(d, (int64_t)B * G, &row_tiles, &NR);
  const int64_t sms = sm_count(), up = (int64_t)row_tiles * Hkv, uo = (int64_t)B * Hkv;
  auto most = [&](int64_t tokens, int64_t ctas, int64_t units) {
    return (int)imin64((tokens + kTile - 1) / kTile, ctas > units ? ctas / units : 1);
  };
  *n_prefix = most(prefix_ctx, sms, up);
  *n_own = most(ctx, 2 * sms, uo);
}

// Writes the partials of the own tokens to slots [0, n_own) and those of the
// prefix to [n_own, n_own + n_prefix).
int launch_shared_tc(const CodecParams& PK, const CodecParams& PV, const tq_kv_view* Kp, const tq_kv_view* Vp,
                     int64_t P_cap, const int32_t* prefix_len, int64_t prefix_ctx, int n_prefix, const tq_kv_view* K,
                     const tq_kv_view* V, int64_t S_cap, const int32_t* kv_len, int64_t ctx, int n_own,
                     const uint16_t* q, float* part, int B, int Hq, int Hkv, float qscale, cudaStream_t st) {
  const WaitLimits wl = wait_limits();
  SharedArgs a{};
  if (n_prefix) a.pre = source_of(Kp, Vp, prefix_len, P_cap, prefix_ctx, n_prefix, n_own);
  if (n_own) a.own = source_of(K, V, kv_len, S_cap, ctx, n_own, 0);
  a.q = q;
  a.part = part;
  a.report_ns = wl.report_ns;
  a.hard_ns = wl.hard_ns;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.by_heads = fast_div((uint32_t)Hkv);
  a.G = Hq / Hkv;
  while ((1 << a.lg) < a.G) ++a.lg;
  a.slots = n_own + n_prefix;
  a.qscale = qscale;
  shared_rows(PK.d, (int64_t)B * a.G, &a.row_tiles, &a.NR);
  const int64_t n_pre = (int64_t)n_prefix * Hkv * a.row_tiles, all = n_pre + (int64_t)n_own * Hkv * B;
  // 32-bit units and token numbers
  if (all > 0x7fffffff || prefix_ctx > 0x7fffff00 || ctx > 0x7fffff00) return TQ_ERR_UNSUPPORTED;
  a.n_pre = (int)n_pre;
  switch (PK.d) {
    case 64: return launch_shared<64>(PK, PV, a, (unsigned)all, st);
    case 128: return launch_shared<128>(PK, PV, a, (unsigned)all, st);
    default: return launch_shared<256>(PK, PV, a, (unsigned)all, st);
  }
}

// First failure status a launch recorded since the last read with clear set.
int shared_tc_status(int clear, int* status) {
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_shared_status, sizeof(int)) != cudaSuccess) return TQ_ERR_CUDA;
  if (clear && v != 0) {
    const int zero = 0;
    if (cudaMemcpyToSymbol(g_shared_status, &zero, sizeof(int)) != cudaSuccess) return TQ_ERR_CUDA;
  }
  *status = v;
  return TQ_OK;
}

}  // namespace tq
