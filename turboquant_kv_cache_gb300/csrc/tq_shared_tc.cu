// Attention of many queries over one shared packed prefix on the tensor cores
// (tcgen05, TMEM accumulators): the prefix part of tq_decode_attn_shared.
//
// Rows: the B sequences' queries of one KV head, R = B*G rows (sequence b,
// head h -> row b*G + h), all of which attend to the same tokens.  A CTA owns
// a tile of up to NR rows, one KV head and a slice of the prefix, which it
// walks in tiles of 128 tokens; its codes are decoded once for all its rows.
//
//   S^T [128 tokens x NR]  = K^ (A, smem, K-major) . Q^ (B, smem, K-major)
//   P^T                    = exp2(S^T - m), fp16, to shared memory
//   O^T [d x NR]          += V^ (A, smem, MN-major) . P^T (B, smem, MN-major)
//   L   [64 x NR]         += ones . P^T      (every lane the sum of a row's p)
//
// Tokens are on the 128 TMEM lanes and rows on the columns, so the tensor
// work and the softmax cost what the rows there are cost (a multiple of 32),
// not the 128 of a row-per-lane tile.  The sum l comes from the same rounded
// p that multiplies V, as one more product with a tile of ones, so a softmax
// thread (a token, half of the rows) keeps no per-row sums.  The reference m
// of a row only moves when a score passes it by more than 2^12 (the first tile
// always does): the common step needs no maximum over tokens, only one
// barrier vote; the rare one takes the maxima and scales O and L.
//
// Warps: 0-7 softmax (warps 0-3 rows [0, NR/2), 4-7 the rest), 8 issues S,
// 9 issues O and L, 10-25 decode.  A decoder thread takes one 32-code group
// (two at head_dim 256) of the K tile and of the V tile, its packed words
// loaded a tile ahead; at head_dim 64 half of the decoder warps take K, half
// V.  Handoffs are mbarriers:
//   kfull/vfull[b] a decoded tile is in buffer b   kfree/vfree[b] its products are done
//   s_full[i] S(t), t & 1 = i, is in TMEM          s_free[i] it has been read
//   p_full    P(t) is written                      o_done    O += P(t) V(t) is done
// Every wait is bounded at two levels, as in tq_tc.cuh; a CTA that gives up
// stops decoding and issuing, waits for the products in flight and frees its
// TMEM.
#include <cuda_runtime.h>
#include <math.h>

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
constexpr int kDec0 = 32 * (kSoftWarps + 2);          // first decoder thread
constexpr int kThreadsSh = kDec0 + kDecThreads;       // 832
// log2 units a score may pass its row's reference by: p stays below 2^12, far
// inside fp16, and sums of p * v inside fp32
constexpr float kLazySh = 12.0f;

// first failure status of a launch since the last read (0 = none)
__device__ int g_shared_status;

template <int D>
struct ShCfg {
  static constexpr int NB = D == 256 ? 1 : 2;          // buffers of K and of V
  static constexpr int DV = D < 128 ? 128 : D;         // V tile width: whole M tiles of 128
  static constexpr int OT = DV / 128;                  // M tiles of O^T
  static constexpr int MAXR = D == 256 ? 96 : 128;     // rows of a CTA: TMEM columns (2 + OT + 1) NR <= 512
  static constexpr uint32_t KB = kTile * D * 2, VB = kTile * DV * 2;
  static constexpr int G8 = D / 32;                    // 32-code groups per token
  static constexpr bool SPLIT = D == 64;               // K and V on half of the decoder warps each
  static constexpr int SIDE = SPLIT ? kDecThreads / 2 : kDecThreads;   // threads on one side
  static constexpr int N = kTile * G8 / SIDE;          // groups per thread and side
  static_assert(N * SIDE == kTile * G8, "every decoder thread has the same number of groups");
};

struct SharedArgs {
  const uint8_t* kc;
  const uint8_t* ks;
  const uint8_t* vc;
  const uint8_t* vs;
  const uint16_t* q;
  const int32_t* prefix_len;   // device [1] or NULL
  float* part;                 // [B*Hq][slots][D + 4]
  PageMap pages;
  int64_t S_cap, ctx, per;     // per: tokens per split (multiple of kTile)
  uint64_t report_ns, hard_ns;
  int B, Hq, Hkv, G, lg, NR, slots, slot0;   // G = 1 << lg
  float qscale;
};

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

// Wait for a phase of an mbarrier as tq_tc.cuh's, but without a sleep between
// polls: try_wait suspends the warp until the phase completes, and a handoff
// of this kernel is due within a microsecond.
__device__ __forceinline__ bool bar_wait_near(uint32_t bar, uint32_t parity, uint64_t report_ns, uint64_t hard_ns,
                                              int& late) {
  uint32_t done = 0;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  if (done) return true;
  const uint64_t t0 = global_ns();
  for (;;) {
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(bar), "r"(parity), "r"(1000000u)
        : "memory");
    const uint64_t el = global_ns() - t0;
    if (el > report_ns) late = 1;
    if (done) return true;
    if (el > hard_ns) return false;
  }
}
// maximum over the warp, in every lane
__device__ __forceinline__ float warp_max_f(float x) {
  float y;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}

// The packed words and norm of one 32-code group, loaded a tile ahead.
struct Group {
  uint32_t w[4];
  uint32_t sc;
};

__device__ __forceinline__ void load_group_g(int bits, const uint8_t* c, uint32_t odd, const uint8_t* s, Group& g) {
  switch (bits) {
    case 4:
      asm volatile("ld.global.nc.v4.u32 {%0,%1,%2,%3}, [%4];"
                   : "=r"(g.w[0]), "=r"(g.w[1]), "=r"(g.w[2]), "=r"(g.w[3])
                   : "l"(c));
      break;
    case 3: {
      // 12 bytes, 8-byte aligned for even groups and 4 bytes past that for
      // odd ones: the 16 bytes around them (an even group is never a row's
      // last, so they are inside the row)
      const uint8_t* c8 = c - (odd ? 4 : 0);
      asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(g.w[0]), "=r"(g.w[1]) : "l"(c8));
      asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(g.w[2]), "=r"(g.w[3]) : "l"(c8 + 8));
      break;
    }
    case 2:
      asm volatile("ld.global.nc.v2.u32 {%0,%1}, [%2];" : "=r"(g.w[0]), "=r"(g.w[1]) : "l"(c));
      break;
    default: asm volatile("ld.global.nc.b32 %0, [%1];" : "=r"(g.w[0]) : "l"(c)); break;
  }
  asm volatile("ld.global.nc.u16 %0, [%1];" : "=r"(g.sc) : "l"(s));
}

// One group's 32 values (centroid * norm, fp16) to the core-matrix tile: four
// 16-byte chunks, one per core matrix.  Each (token, block) table holds the
// fp32 products of centroids and norm, rounded once to fp16.
template <int BITS>
__device__ __forceinline__ void decode_group_b(const Group& g, uint32_t odd, const float* cent, uint32_t dst) {
  uint32_t n[4];
  if (BITS == 3) {
    const uint32_t w3[3] = {odd ? g.w[1] : g.w[0], odd ? g.w[2] : g.w[1], odd ? g.w[3] : g.w[2]};
    chunk_words<3>(w3, n);
  } else {
    chunk_words<BITS>(g.w, n);
  }
  const Tab T = make_tab_f32<BITS>(cent, h2f((uint16_t)g.sc));
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t o[4];
    lut8<BITS>(n[c], T, o);
    sts16b(dst + 128 * c, o[0], o[1], o[2], o[3]);
  }
}

__device__ __forceinline__ void decode_group(int bits, const Group& g, uint32_t odd, const float* cent, bool live,
                                             uint32_t dst) {
  if (!live) {   // past the slice: zero rows (their p is zero too, but 0 * NaN is not)
#pragma unroll
    for (int c = 0; c < 4; ++c) sts16b(dst + 128 * c, 0u, 0u, 0u, 0u);
    return;
  }
  switch (bits) {
    case 4: decode_group_b<4>(g, odd, cent, dst); break;
    case 3: decode_group_b<3>(g, odd, cent, dst); break;
    case 2: decode_group_b<2>(g, odd, cent, dst); break;
    default: decode_group_b<1>(g, odd, cent, dst); break;
  }
}

template <int D, bool PAGED>
__global__ void __launch_bounds__(kThreadsSh, 1) shared_prefix_kernel(const CodecParams PK, const CodecParams PV,
                                                                      const SharedArgs a) {
  using C = ShCfg<D>;
  constexpr int NB = C::NB, OT = C::OT;
  constexpr uint32_t kKGroup = (D / 8) * 128;       // bytes of 8 tokens of K, 8 rows of Q
  constexpr uint32_t kVGroup = (C::DV / 8) * 128;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ __align__(8) uint64_t bars[4 * NB + 7];
  __shared__ uint32_t tmem_base;
  __shared__ volatile int s_abort;
  __shared__ int s_late;
  __shared__ __align__(16) float s_m[C::MAXR];      // the rows' softmax references
  __shared__ float s_al[C::MAXR];
  __shared__ float s_wm[4][C::MAXR];                // maxima by TMEM lane quarter (rare path)

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int NR = a.NR;
  const int split = blockIdx.x, kvh = blockIdx.y, rt = blockIdx.z;
  const int row0 = rt * NR;
  const int rows = min(NR, a.B * a.G - row0);
  int64_t len = a.ctx;
  if (a.prefix_len) len = imin64(len, (int64_t)a.prefix_len[0]);
  const int64_t t_lo = (int64_t)split * a.per;
  const int64_t t_hi = imin64(t_lo + a.per, len);
  const int n_tiles = t_hi > t_lo ? (int)((t_hi - t_lo + kTile - 1) / kTile) : 0;

  // K buffers, V buffers, Q^, P, ones
  const uint32_t aK = su32(smem), aV = aK + NB * C::KB, aQ = aV + NB * C::VB, aP = aQ + (uint32_t)NR * D * 2,
                 aOnes = aP + (uint32_t)NR * kTile * 2;
  const uint32_t kfull = su32(&bars[0]), vfull = su32(&bars[NB]), kfree = su32(&bars[2 * NB]),
                 vfree = su32(&bars[3 * NB]), s_full = su32(&bars[4 * NB]), s_free = su32(&bars[4 * NB + 2]),
                 p_full = su32(&bars[4 * NB + 4]), o_done = su32(&bars[4 * NB + 5]), drained = su32(&bars[4 * NB + 6]);
  // TMEM columns
  const uint32_t cO = 2u * NR, cL = cO + (uint32_t)OT * NR;
  const uint32_t tcols = cL + NR > 256 ? 512u : (cL + NR > 128 ? 256u : 128u);

  auto wait = [&](uint32_t bar, uint32_t parity) {
    if (__any_sync(kFull, s_abort)) return false;   // one decision per warp
    int late = 0;
    const bool ok = __all_sync(kFull, bar_wait_near(bar, parity, a.report_ns, a.hard_ns, late));
    if (late) s_late = 1;
    if (!ok) s_abort = 1;
    return ok;
  };

  if (tid == 0) {
    s_abort = 0;
    s_late = 0;
    constexpr int kSide = C::SIDE / 32;   // decoder warps that fill one side
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      bar_init(kfull + 8 * i, kSide);
      bar_init(vfull + 8 * i, kSide);
      bar_init(kfree + 8 * i, 1);
      bar_init(vfree + 8 * i, 1);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      bar_init(s_full + 8 * i, 1);
      bar_init(s_free + 8 * i, kSoftWarps);
    }
    bar_init(p_full, kSoftWarps);
    bar_init(o_done, 1);
    bar_init(drained, 2);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(su32(&tmem_base)),
                 "r"(tcols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  if (tid < NR) s_m[tid] = -INFINITY;
  if (tid < 128) sts16b(aOnes + 16 * tid, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u, 0x3C003C00u);
  // Q^ = H D q per K block, times softmax_scale * log2 e: a warp per row, a
  // lane the D/32 consecutive values from E*lane on
  if (n_tiles > 0) {
    constexpr int E = D / 32;
    const float qn = PK.inv_sqrt_blk * a.qscale;
    for (int r = warp; r < NR; r += kThreadsSh / 32) {
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = 0.f;
      if (r < rows) {
        const int rr = row0 + r, b = rr >> a.lg, h = kvh * a.G + (rr & (a.G - 1));
        const uint16_t* src = a.q + ((int64_t)b * a.Hq + h) * D + E * lane;
        uint32_t u[E / 2];
        if constexpr (E == 8) {
          const uint4 x = *reinterpret_cast<const uint4*>(src);
          u[0] = x.x; u[1] = x.y; u[2] = x.z; u[3] = x.w;
        } else if constexpr (E == 4) {
          const uint2 x = *reinterpret_cast<const uint2*>(src);
          u[0] = x.x; u[1] = x.y;
        } else {
          u[0] = *reinterpret_cast<const uint32_t*>(src);
        }
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const int i = E * lane + e;
          v[e] = flip(h2f((uint16_t)(u[e / 2] >> (16 * (e & 1)))), (PK.sign_bits[i >> 5] >> (i & 31)) & 1u);
        }
        for (int hs = 1; hs < E && hs < PK.blk; hs <<= 1) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if ((e & hs) == 0 && e + hs < E) {
              const float x = v[e], y = v[e + hs];
              v[e] = x + y;
              v[e + hs] = x - y;
            }
          }
        }
        for (int hs = E; hs < PK.blk; hs <<= 1) {
          const int lo = hs / E;
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const float x = __shfl_xor_sync(kFull, v[e], lo);
            v[e] = (lane & lo) ? (x - v[e]) : (v[e] + x);
          }
        }
      }
      const uint32_t dst = aQ + cm_off(r, E * lane, D);
      uint32_t o[E / 2];
#pragma unroll
      for (int e = 0; e < E / 2; ++e) o[e] = pack2(v[2 * e] * qn, v[2 * e + 1] * qn);
      if constexpr (E == 8) {
        sts16b(dst, o[0], o[1], o[2], o[3]);
      } else if constexpr (E == 4) {
        asm volatile("st.shared.v2.b32 [%0], {%1,%2};" ::"r"(dst), "r"(o[0]), "r"(o[1]) : "memory");
      } else {
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst), "r"(o[0]) : "memory");
      }
    }
  }
  fence_async_smem();
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = tmem_base;

  if (warp >= kSoftWarps + 2) {
    // ================= decoders
    const int dt = tid - kDec0;
    const int st = C::SPLIT ? dt % C::SIDE : dt;    // thread within its side
    const bool do_k = !C::SPLIT || dt < C::SIDE, do_v = !C::SPLIT || dt >= C::SIDE;
    // the thread's groups: number grp of the tokens tok0 and, at head_dim 256,
    // kStep tokens on.  Contiguous: pointers of the first that move on by a
    // tile; paged: page and place in it of each.
    constexpr int kStep = C::SIDE / C::G8;
    static_assert(C::N == 1 || kStep % 8 == 0, "a thread's groups have one number");
    const int tok0 = 8 * (st / (8 * C::G8)) + (st & 7), grp = (st >> 3) % C::G8;
    const int kbits = PK.bits, vbits = PV.bits;
    const uint8_t *kw = a.kc + grp * 4 * kbits, *kn = a.ks + 32 * grp / PK.blk * 2;
    const uint8_t *vw = a.vc + grp * 4 * vbits, *vn = a.vs + 32 * grp / PV.blk * 2;
    int32_t page[C::N], off[C::N];
    if (PAGED) {
#pragma unroll
      for (int k = 0; k < C::N; ++k) {
        const int64_t t = t_lo + tok0 + k * kStep;
        page[k] = (int32_t)(t / a.pages.page_size);
        off[k] = (int32_t)(t - (int64_t)page[k] * a.pages.page_size);
      }
    } else {
      const int64_t r = (int64_t)kvh * a.S_cap + t_lo + tok0;
      kw += r * PK.code_bytes;
      vw += r * PV.code_bytes;
      kn += r * PK.nb * 2;
      vn += r * PV.nb * 2;
    }
    Group gk[C::N], gv[C::N];
    auto left_of = [&](int t) { return (int)imin64(kTile, t_hi - (t_lo + (int64_t)t * kTile)); };
    auto load = [&](int t) {
      const int left = left_of(t);
#pragma unroll
      for (int k = 0; k < C::N; ++k) {
        if (tok0 + k * kStep < left) {
          int64_t r = k * kStep;
          if (PAGED) r = ((int64_t)a.pages.table[page[k]] * a.Hkv + kvh) * a.pages.page_size + off[k];
          if (do_k) load_group_g(kbits, kw + r * PK.code_bytes, grp & 1, kn + r * (PK.nb * 2), gk[k]);
          if (do_v) load_group_g(vbits, vw + r * PV.code_bytes, grp & 1, vn + r * (PV.nb * 2), gv[k]);
        }
        if (PAGED) {
          off[k] += kTile;
          while (off[k] >= a.pages.page_size) {
            off[k] -= a.pages.page_size;
            ++page[k];
          }
        }
      }
      if (!PAGED) {
        kw += kTile * PK.code_bytes;
        vw += kTile * PV.code_bytes;
        kn += kTile * PK.nb * 2;
        vn += kTile * PV.nb * 2;
      }
    };
    if (n_tiles > 0) load(0);
    for (int t = 0; t < n_tiles; ++t) {
      const int bf = t % NB;
      const int left = left_of(t);
      const uint32_t ph = (uint32_t)(t / NB - 1) & 1;
      if (do_k) {
        if (t >= NB) wait(kfree + 8 * bf, ph);
        if (!s_abort) {
#pragma unroll
          for (int k = 0; k < C::N; ++k)
            decode_group(kbits, gk[k], grp & 1, PK.centroids, tok0 + k * kStep < left,
                         aK + bf * C::KB + cm_off(tok0 + k * kStep, 32 * grp, D));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive(kfull + 8 * bf);
      }
      if (do_v) {
        if (t >= NB) wait(vfree + 8 * bf, ph);
        if (!s_abort) {
#pragma unroll
          for (int k = 0; k < C::N; ++k)
            decode_group(vbits, gv[k], grp & 1, PV.centroids, tok0 + k * kStep < left,
                         aV + bf * C::VB + cm_off(tok0 + k * kStep, 32 * grp, C::DV));
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0) arrive(vfull + 8 * bf);
      }
      if (t + 1 < n_tiles) load(t + 1);
    }
  } else if (warp == kSoftWarps) {
    // ================= S^T(t) = K^(t) Q^
    const uint32_t idesc = (1u << 4) | ((uint32_t)(NR >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
    const uint64_t dq = sdesc(aQ, 128, kKGroup);
    for (int t = 0; t < n_tiles; ++t) {
      const int bf = t % NB;
      if (!wait(kfull + 8 * bf, (uint32_t)(t / NB) & 1)) break;
      if (t >= 2 && !wait(s_free + 8 * (t & 1), (uint32_t)((t >> 1) - 1) & 1)) break;
      fence_after();
      __syncwarp();
      const uint64_t dk = sdesc(aK + bf * C::KB, 128, kKGroup);
#pragma unroll
      for (int s = 0; s < D / 16; ++s)
        mma_ss_elect(tmem + (t & 1) * NR, dk + (uint64_t)(16 * s), dq + (uint64_t)(16 * s), idesc, s > 0);
      commit_elect(s_full + 8 * (t & 1));
      commit_elect(kfree + 8 * bf);
    }
    __syncwarp();
    commit_elect(drained);
  } else if (warp == kSoftWarps + 1) {
    // ================= O^T += V^(t)^T P(t)^T, L += ones P(t)^T
    const uint32_t idesc = (1u << 4) | (1u << 15) | (1u << 16) | ((uint32_t)(NR >> 3) << 17) |
                           ((uint32_t)(128 >> 4) << 24);
    const uint32_t idesc_l = (1u << 4) | (1u << 16) | ((uint32_t)(NR >> 3) << 17) | ((uint32_t)(64 >> 4) << 24);
    const uint32_t pg = (uint32_t)(NR >> 3) * 128;   // bytes of 8 tokens of P
    const uint64_t dp = sdesc(aP, pg, 128), done = sdesc(aOnes, 128, 256);
    for (int t = 0; t < n_tiles; ++t) {
      const int bf = t % NB;
      if (!wait(vfull + 8 * bf, (uint32_t)(t / NB) & 1)) break;
      if (!wait(p_full, (uint32_t)t & 1)) break;
      fence_after();
      __syncwarp();
#pragma unroll
      for (int m = 0; m < OT; ++m) {
        const uint64_t dv = sdesc(aV + bf * C::VB + m * 16 * 128, kVGroup, 128);
#pragma unroll
        for (int s = 0; s < kTile / 16; ++s)
          mma_ss_elect(tmem + cO + m * NR, dv + (uint64_t)(s * (2 * kVGroup >> 4)),
                       dp + (uint64_t)(s * (2 * pg >> 4)), idesc, t > 0 || s > 0);
      }
#pragma unroll
      for (int s = 0; s < kTile / 16; ++s)
        mma_ss_elect(tmem + cL, done, dp + (uint64_t)(s * (2 * pg >> 4)), idesc_l, t > 0 || s > 0);
      commit_elect(o_done);
      commit_elect(vfree + 8 * bf);
    }
    __syncwarp();
    commit_elect(drained);
  } else {
    // ================= softmax: thread = token (TMEM lane) x half of the rows
    const int quarter = warp & 3, half = warp >> 2, bid = 1 + half;
    const int nc = NR / 2, col0 = half * nc;
    const int tk = 32 * quarter + lane;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16);
    const uint32_t pdst = aP + cm_off(tk, col0, NR);
    // p of 16 columns from c on, from their scores: stored to P; returns the
    // largest s - m.  A token past the slice has p = 0.
    auto emit = [&](uint32_t* v, int c, bool live) {
      float mx = -INFINITY;
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 16; j += 4) {
        const float4 m = *reinterpret_cast<const float4*>(&s_m[col0 + c + j]);
        const float x0 = __uint_as_float(v[j]) - m.x, x1 = __uint_as_float(v[j + 1]) - m.y;
        const float x2 = __uint_as_float(v[j + 2]) - m.z, x3 = __uint_as_float(v[j + 3]) - m.w;
        mx = fmaxf(mx, fmaxf(fmaxf(x0, x1), fmaxf(x2, x3)));
        o[j / 2] = pack2(ex2s(x0), ex2s(x1));
        o[j / 2 + 1] = pack2(ex2s(x2), ex2s(x3));
      }
      if (!live) {
        mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = 0u;
      }
      sts16b(pdst + (c >> 3) * 128, o[0], o[1], o[2], o[3]);
      sts16b(pdst + (c >> 3) * 128 + 128, o[4], o[5], o[6], o[7]);
      return mx;
    };
    for (int t = 0; t < n_tiles; ++t) {
      const bool live = tk < t_hi - (t_lo + (int64_t)t * kTile);
      const uint32_t sS = lanes + (t & 1) * NR + col0;
      wait(s_full + 8 * (t & 1), (uint32_t)(t >> 1) & 1);
      if (t >= 1) wait(o_done, (uint32_t)(t - 1) & 1);   // P is free, O and L stand still
      fence_after();
      bool moved = t == 0;
      if (!moved) {
        float mx = -INFINITY;
        for (int c = 0; c < nc; c += 16) {
          uint32_t v[16];
          TQ_LD16(sS + c, v);
          ld_wait();
          mx = fmaxf(mx, emit(v, c, live));
        }
        moved = half_any(bid, mx > kLazySh);
      }
      if (moved) {
        // some row's reference moves (the first tile sets them): its maximum
        // over the tile, O and L scaled, P written again
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
          if (lane < 16) s_wm[quarter][col0 + c + lane] = mine;
        }
        half_sync(bid);
        if ((tid & 127) < nc) {
          const int r = col0 + (tid & 127);
          const float x = fmaxf(fmaxf(s_wm[0][r], s_wm[1][r]), fmaxf(s_wm[2][r], s_wm[3][r]));
          const float mo = s_m[r], mn = x > mo + kLazySh || mo == -INFINITY ? x : mo;
          s_m[r] = mn;
          s_al[r] = mo == -INFINITY ? 0.f : ex2s(mo - mn);
        }
        half_sync(bid);
        if (t >= 1) {
#pragma unroll 1
          for (int m = 0; m <= OT; ++m) {   // O's M tiles, then L
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
        for (int c = 0; c < nc; c += 16) {
          uint32_t v[16];
          TQ_LD16(sS + c, v);
          ld_wait();
          emit(v, c, live);
        }
      }
      fence_async_smem();
      fence_before();
      __syncwarp();
      if (lane == 0) {
        arrive(p_full);
        arrive(s_free + 8 * (t & 1));
      }
    }
    if (n_tiles > 0) wait(o_done, (uint32_t)(n_tiles - 1) & 1);
    fence_after();
    const bool ok = n_tiles > 0 && !__any_sync(kFull, s_abort);
    // partials: lane = dimension of O^T, column = row
    for (int c = 0; c < nc; c += 16) {
      uint32_t l[16];
      if (ok && quarter == 0) {
        TQ_LD16(lanes + cL + col0 + c, l);
        ld_wait();
      }
#pragma unroll 1
      for (int m = 0; m < OT; ++m) {
        uint32_t v[16];
        if (ok) {
          TQ_LD16(lanes + cO + m * NR + col0 + c, v);
          ld_wait();
        }
        const int dim = 128 * m + tk;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int r = col0 + c + j;
          if (r >= rows) continue;
          const int rr = row0 + r, b = rr >> a.lg, h = kvh * a.G + (rr & (a.G - 1));
          float* dst = a.part + (((int64_t)b * a.Hq + h) * a.slots + a.slot0 + split) * (D + 4);
          if (dim < D) dst[2 + dim] = ok ? __uint_as_float(v[j]) : 0.f;
          if (m == 0 && quarter == 0 && lane == j) {
            dst[0] = ok ? s_m[r] : -INFINITY;
            dst[1] = ok ? __uint_as_float(l[j]) : 0.f;
          }
        }
      }
    }
  }
  // the next kernel may be scheduled; it waits for this grid before it ends
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  fence_before();
  __syncthreads();
  if (warp == 0) {
    fence_after();
    // every product has been committed and, on the normal path, has ended
    int late = 0;
    __all_sync(kFull, bar_wait_near(drained, 0, a.report_ns, a.hard_ns, late));
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(tcols) : "memory");
    if (lane == 0 && (s_abort || s_late || late)) atomicCAS(&g_shared_status, 0, (int)TQ_ERR_TIMEOUT);
  }
}

template <int D>
size_t shared_smem(int NR) {
  return (size_t)ShCfg<D>::NB * (ShCfg<D>::KB + ShCfg<D>::VB) + (size_t)NR * D * 2 + (size_t)NR * kTile * 2 + 2048;
}

template <int D, bool PAGED>
int launch_shared(const CodecParams& PK, const CodecParams& PV, const SharedArgs& a, dim3 grid, cudaStream_t st) {
  auto kern = shared_prefix_kernel<D, PAGED>;
  const size_t sm = shared_smem<D>(a.NR);
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return TQ_ERR_CUDA;
  if (!attr_set[dev]) {
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)shared_smem<D>(ShCfg<D>::MAXR)) !=
        cudaSuccess)
      return TQ_ERR_CUDA;
    attr_set[dev] = true;
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

}  // namespace

// Layouts whose prefix the tensor-core kernel takes: 1..4 bits without QJL,
// norms on their own alignment.
bool shared_tc_eligible(const CodecParams& PK, const CodecParams& PV) {
  return !PK.m && !PV.m && PK.bits <= 4 && PV.bits <= 4;
}

// Prefix splits: one wave of a CTA per SM, each at least a tile.
int shared_tc_splits(int d, int B, int G, int Hkv, int64_t ctx) {
  int tiles, NR;
  shared_rows(d, (int64_t)B * G, &tiles, &NR);
  const int64_t most = (ctx + kTile - 1) / kTile;
  int64_t ns = sm_count() / ((int64_t)tiles * Hkv);
  if (ns > most) ns = most;
  return ns < 1 ? 1 : (int)ns;
}

// Writes the partials of the prefix to slots [slot0, slot0 + n_split).
int launch_shared_tc(const CodecParams& PK, const CodecParams& PV, const tq_kv_view* K, const tq_kv_view* V,
                     const uint16_t* q, const int32_t* prefix_len, float* part, int B, int Hq, int Hkv, int64_t S_cap,
                     int64_t ctx, int n_split, int slots, int slot0, float qscale, cudaStream_t st) {
  const WaitLimits wl = wait_limits();
  SharedArgs a{};
  a.kc = K->codes;
  a.ks = reinterpret_cast<const uint8_t*>(K->scales);
  a.vc = V->codes;
  a.vs = reinterpret_cast<const uint8_t*>(V->scales);
  a.q = q;
  a.prefix_len = prefix_len;
  a.part = part;
  a.pages = {K->page_table, K->page_table ? K->page_size : 0, K->page_table ? K->pages_per_seq : 0};
  a.S_cap = S_cap;
  a.ctx = ctx;
  const int64_t tiles_all = (ctx + kTile - 1) / kTile;
  a.per = (tiles_all + n_split - 1) / n_split * kTile;
  a.report_ns = wl.report_ns;
  a.hard_ns = wl.hard_ns;
  a.B = B;
  a.Hq = Hq;
  a.Hkv = Hkv;
  a.G = Hq / Hkv;
  while ((1 << a.lg) < a.G) ++a.lg;
  a.slots = slots;
  a.slot0 = slot0;
  a.qscale = qscale;
  int tiles;
  shared_rows(PK.d, (int64_t)B * a.G, &tiles, &a.NR);
  const dim3 grid((unsigned)n_split, (unsigned)Hkv, (unsigned)tiles);
  switch (PK.d) {
    case 64: return a.pages.table ? launch_shared<64, true>(PK, PV, a, grid, st) : launch_shared<64, false>(PK, PV, a, grid, st);
    case 128: return a.pages.table ? launch_shared<128, true>(PK, PV, a, grid, st) : launch_shared<128, false>(PK, PV, a, grid, st);
    default: return a.pages.table ? launch_shared<256, true>(PK, PV, a, grid, st) : launch_shared<256, false>(PK, PV, a, grid, st);
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
