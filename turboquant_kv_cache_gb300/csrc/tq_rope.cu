// Rows of a model's query/key/value projection made ready for the cache and
// the attention: RMS norm of every query and key head, rotary position, and
// the [batch, head, token] layout, in one pass.
//
// Mathematics, per head row x of d values (queries and keys):
//   y_i = x_i / sqrt(sum x^2 / d + eps) * w_i            (when w is given)
//   (y_a, y_b) -> (y_a cos - y_b sin, y_b cos + y_a sin)  for each rotated pair
// in fp32 whatever the input's type, rounded to fp16 once at the end.  Value
// rows are only converted.
//
// Mapping: a thread owns 16 values of a row, 8 of the rotated lower half and
// the 8 that they are paired with, or 16 consecutive ones behind the rotated
// part: no value crosses threads but for the sum of squares, a shuffle
// reduction over the row's d/16 threads.  A row is read and written in pieces
// of 16 bytes a thread.  (8 consecutive values a thread and the pair's other
// value by shuffle: 153 us against 132 for 32768 tokens; the shuffles, and the
// weights read anew for every row, kept the load/store pipe 75 % busy.)
//
// Bound: memory once there are many tokens, since a row is read and written
// once and nothing else is (822 MB for 32768 tokens of 48 heads, head_dim 128,
// fp16: 130.5 us, 6.3 TB/s, 94 % of a copy's rate); for a few tokens the launch
// (8 tokens 2.4 us in a graph, 15 tokens of fp32 rows at head_dim 256 2.5).
#include <cuda_runtime.h>

#include "tq_device.cuh"

namespace tq {

int sm_count();

namespace {

constexpr int kThreads = 64;

struct RopeArgs {
  const void* x;
  int64_t row_stride;      // elements between token rows
  const float* wq;
  const float* wk;
  const float* rope;       // [n_pos][rot]: rot/2 cosines, then rot/2 sines
  const int32_t* pos;      // [B] or NULL
  const int32_t* new_len;  // [B] or NULL
  const int32_t* slot;     // [B] or NULL
  uint16_t* q;
  uint16_t* k;
  uint16_t* v;
  int64_t n_pos, kv_cap;
  int64_t tokens;          // B * T
  int T, Hq, Hkv, rot;
  float eps;
};

// 8 values of a row as they lie in memory, and as floats
template <bool F32>
struct Raw {
  uint4 u[F32 ? 2 : 1];
};
template <bool F32>
__device__ __forceinline__ Raw<F32> load8(const void* x, int64_t at) {
  Raw<F32> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) + at * (F32 ? 4 : 2));
  r.u[0] = __ldcs(p);
  if constexpr (F32) r.u[1] = __ldcs(p + 1);
  return r;
}
template <bool F32>
__device__ __forceinline__ void floats(const Raw<F32>& r, float* v) {
  if constexpr (F32) {
    const uint32_t w[8] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w, r.u[1].x, r.u[1].y, r.u[1].z, r.u[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {r.u[0].x, r.u[0].y, r.u[0].z, r.u[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

template <int N>
__device__ __forceinline__ void load_floats(const float* p, float* v) {
#pragma unroll
  for (int i = 0; i < N; i += 4) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p + i));
    v[i] = a.x; v[i + 1] = a.y; v[i + 2] = a.z; v[i + 3] = a.w;
  }
}

// NEXT: rotated pairs are neighbours (2i, 2i+1); otherwise (i, i + rot/2).
// A block's kThreads / (D/16) thread groups take consecutive token rows b*T + j
// (grid x) and the same R heads (grid y): a group has R rows of one token in
// flight, contiguous in the input, and reads the token's cosines and sines
// once for all of them, and the weights once for heads of one kind; the
// block's outputs of a head are one run.
template <int D, bool F32, bool NEXT, int R>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const __grid_constant__ RopeArgs a) {
  constexpr int TPR = D / 16;             // threads per row
  constexpr int HPB = kThreads / TPR;     // groups per block
  // the thread's chunks of 8 values: one of the rotated lower half and its
  // counterpart of the upper half, or two neighbours behind the rotated part
  const int sub = threadIdx.x % TPR, lows = a.rot / 16;
  const bool in = sub < lows;
  const int e0 = in ? 8 * sub : 16 * sub, e1 = in ? e0 + a.rot / 2 : e0 + 8;
  const int64_t tok_at = (int64_t)blockIdx.x * HPB + threadIdx.x / TPR, tok = imin64(tok_at, a.tokens - 1);
  const int h0 = blockIdx.y * R;
  const int H = a.Hq + 2 * a.Hkv, HT = a.Hq + a.Hkv;   // all heads, and those with a position
  Raw<F32> raw[R][2];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int64_t row = tok * a.row_stride + (int64_t)min(h0 + i, H - 1) * D;
    raw[i][0] = load8<F32>(a.x, row + e0);
    raw[i][1] = load8<F32>(a.x, row + e1);
  }
  const int b = (int)(tok / a.T), j = (int)(tok - (int64_t)b * a.T);
  const int n_new = a.new_len ? a.new_len[b] : a.T;
  const int64_t p = (a.pos ? (int64_t)a.pos[b] : 0) + j;
  const int64_t at = (a.slot ? (int64_t)a.slot[b] : 0) + j;
  // a token behind its batch's length, or whose position has no row in the
  // table, is left out (its lanes stay for the shuffles of their warp)
  const bool ok = tok_at < a.tokens && j < n_new && (!a.rot || (p >= 0 && p < a.n_pos));
  // cosines and sines of the thread's pairs: (e0 + k, e1 + k), or four
  // neighbouring pairs of each chunk
  float c[8], s[8];
  if (in && ok) {
    const float* row = a.rope + p * a.rot;
    const int half = a.rot / 2;
    if constexpr (NEXT) {
      load_floats<4>(row + e0 / 2, c);
      load_floats<4>(row + e1 / 2, c + 4);
      load_floats<4>(row + half + e0 / 2, s);
      load_floats<4>(row + half + e1 / 2, s + 4);
    } else {
      load_floats<8>(row + e0, c);
      load_floats<8>(row + half + e0, s);
    }
  }
  const float* have = nullptr;   // the weights in wv
  float wv[16];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int h = h0 + i;
    const float* w = h < a.Hq ? a.wq : (h < HT ? a.wk : nullptr);
    float v[16];
    floats<F32>(raw[i][0], v);
    floats<F32>(raw[i][1], v + 8);
    if (w) {   // the same for the whole block
      if (w != have) {
        load_floats<8>(w + e0, wv);
        load_floats<8>(w + e1, wv + 8);
        have = w;
      }
      float s0 = 0.f, s1 = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        s0 = fmaf(v[k], v[k], s0);
        s1 = fmaf(v[8 + k], v[8 + k], s1);
      }
      float ss = s0 + s1;
#pragma unroll
      for (int o = 1; o < TPR; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = v[k] * r * wv[k];
    }
    if (in && h < HT) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int x = NEXT ? 2 * k : k, y = NEXT ? 2 * k + 1 : k + 8;
        const float vx = v[x], vy = v[y];
        v[x] = vx * c[k] - vy * s[k];
        v[y] = vy * c[k] + vx * s[k];
      }
    }
    if (h >= H || !ok) continue;
    uint16_t* dst;
    if (h < a.Hq) {
      dst = a.q + (((int64_t)b * a.Hq + h) * a.T + j) * D;
    } else {
      if (at < 0 || at >= a.kv_cap) continue;
      const int kv = h - a.Hq;
      dst = kv < a.Hkv ? a.k + (((int64_t)b * a.Hkv + kv) * a.kv_cap + at) * D
                       : a.v + (((int64_t)b * a.Hkv + kv - a.Hkv) * a.kv_cap + at) * D;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      uint32_t o[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2 y = __floats2half2_rn(v[8 * x + 2 * k], v[8 * x + 2 * k + 1]);
        o[k] = *reinterpret_cast<const uint32_t*>(&y);
      }
      *reinterpret_cast<uint4*>(dst + (x ? e1 : e0)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int D, bool F32, bool NEXT>
void launch_rows(const RopeArgs& a, int64_t tokens, cudaStream_t st) {
  constexpr int HPB = kThreads / (D / 16);
  const int H = a.Hq + 2 * a.Hkv;
  // Rows per thread group: one while that does not fill the GPU (latency
  // counts), else the number from 4 down to 2 that leaves the fewest without
  // a head: several rows in flight and the cosines and sines read once for
  // them.  8 tokens of 48 heads: 1 or 2 rows 2.2 us, 4 rows 2.5; 32768 tokens:
  // 1 row 151 us, 2 rows 136, 3 rows 141, 4 rows 132.
  const int64_t blocks = (tokens + HPB - 1) / HPB;
  int R = 1;
  if (blocks * H > 16 * sm_count()) {
    int best = 1 << 30;
    for (int r = 4; r >= 2; --r) {
      const int idle = (H + r - 1) / r * r - H;
      if (idle < best) {
        best = idle;
        R = r;
      }
    }
  }
  const dim3 grid((unsigned)blocks, (unsigned)((H + R - 1) / R));
  switch (R) {
    case 1: norm_rope_kernel<D, F32, NEXT, 1><<<grid, kThreads, 0, st>>>(a); break;
    case 2: norm_rope_kernel<D, F32, NEXT, 2><<<grid, kThreads, 0, st>>>(a); break;
    case 3: norm_rope_kernel<D, F32, NEXT, 3><<<grid, kThreads, 0, st>>>(a); break;
    default: norm_rope_kernel<D, F32, NEXT, 4><<<grid, kThreads, 0, st>>>(a); break;
  }
}

template <int D>
void launch(const RopeArgs& a, bool f32, bool next, int64_t tokens, cudaStream_t st) {
  if (f32) {
    if (next) launch_rows<D, true, true>(a, tokens, st);
    else launch_rows<D, true, false>(a, tokens, st);
  } else {
    if (next) launch_rows<D, false, true>(a, tokens, st);
    else launch_rows<D, false, false>(a, tokens, st);
  }
}

}  // namespace
}  // namespace tq

extern "C" int tq_qkv_norm_rope(const void* qkv, tq_dtype x_dtype, int B, int T, int Hq, int Hkv, int head_dim,
                                int64_t row_stride, const float* q_weight, const float* k_weight, float eps,
                                const float* rope, int64_t n_pos, int rot_dim, int interleaved, const int32_t* pos,
                                const int32_t* new_len, uint16_t* q_out, uint16_t* k_out, uint16_t* v_out,
                                int64_t kv_cap, const int32_t* slot, void* stream) {
  if (B < 0 || T < 0 || Hq <= 0 || Hkv <= 0 || Hq > 4096 || Hkv > 4096 || kv_cap < 0 || n_pos < 0) return TQ_ERR_ARG;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return TQ_ERR_UNSUPPORTED;
  if (x_dtype != TQ_F16 && x_dtype != TQ_F32) return TQ_ERR_ARG;
  if (interleaved != 0 && interleaved != 1) return TQ_ERR_ARG;
  if (rot_dim < 0 || rot_dim > head_dim || (rot_dim && (!rope || n_pos <= 0))) return TQ_ERR_ARG;
  if (rot_dim % 16) return TQ_ERR_UNSUPPORTED;
  if ((q_weight || k_weight) && !(eps > 0.f)) return TQ_ERR_ARG;
  const int64_t width = (int64_t)(Hq + 2 * Hkv) * head_dim;
  if (row_stride < width) return TQ_ERR_ARG;
  if ((int64_t)B * T == 0) return TQ_OK;
  if ((int64_t)B * T > 0x7fffffff) return TQ_ERR_UNSUPPORTED;
  if (!qkv || !q_out || (kv_cap && (!k_out || !v_out))) return TQ_ERR_ARG;
  if (!tq::aligned16(qkv) || (row_stride * (x_dtype == TQ_F32 ? 4 : 2)) % 16 || !tq::aligned16(q_out) ||
      !tq::aligned16(k_out) || !tq::aligned16(v_out) || !tq::aligned16(q_weight) || !tq::aligned16(k_weight) ||
      !tq::aligned16(rope))
    return TQ_ERR_ALIGN;
  const tq::RopeArgs a{qkv, row_stride, q_weight, k_weight, rope, pos, new_len, slot, q_out, k_out, v_out,
                       n_pos, kv_cap, (int64_t)B * T, T, Hq, Hkv, rot_dim, eps};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t tokens = (int64_t)B * T;
  switch (head_dim) {
    case 64: tq::launch<64>(a, x_dtype == TQ_F32, interleaved, tokens, st); break;
    case 128: tq::launch<128>(a, x_dtype == TQ_F32, interleaved, tokens, st); break;
    default: tq::launch<256>(a, x_dtype == TQ_F32, interleaved, tokens, st); break;
  }
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
