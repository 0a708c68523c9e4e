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
// Mapping: a thread owns 8 consecutive values of a row, d/8 threads a row, so
// a row is one coalesced read and write of 16 bytes a thread; the sum of
// squares is a shuffle reduction and a half-split pair's other value comes by
// shuffle from the lane that owns it.
#include <cuda_runtime.h>

#include "tq_device.cuh"

namespace tq {
namespace {

constexpr int kThreads = 128;

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
  int T, Hq, Hkv, rot;
  float eps;
};

template <bool F32>
__device__ __forceinline__ void load8(const void* x, int64_t at, float* v) {
  if constexpr (F32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(x) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}

// NEXT: rotated pairs are neighbours (2i, 2i+1); otherwise (i, i + rot/2).
// Grid: x = token rows b*T + j, y = groups of kThreads / (D/8) heads.
template <int D, bool F32, bool NEXT>
__global__ void __launch_bounds__(kThreads) norm_rope_kernel(const RopeArgs a) {
  constexpr int TPR = D / 8;              // threads per row
  constexpr int HPB = kThreads / TPR;     // heads per block
  const int64_t tok = blockIdx.x;
  const int b = (int)(tok / a.T), j = (int)(tok - (int64_t)b * a.T);
  if (a.new_len && j >= a.new_len[b]) return;
  const int64_t p = (a.pos ? (int64_t)a.pos[b] : 0) + j;
  if (a.rot && (p < 0 || p >= a.n_pos)) return;   // no such row of the table: the token is left out
  const int h = blockIdx.y * HPB + threadIdx.x / TPR;
  const int H = a.Hq + 2 * a.Hkv;
  const int sub = threadIdx.x % TPR, e0 = 8 * sub;
  const bool live = h < H;
  float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live) load8<F32>(a.x, tok * a.row_stride + (int64_t)h * D + e0, v);
  const bool turned = live && h < a.Hq + a.Hkv;   // queries and keys
  const float* w = h < a.Hq ? a.wq : a.wk;
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
#pragma unroll
  for (int o = 1; o < TPR; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
  if (turned && w) {
    const float r = rsqrtf(ss * (1.f / D) + a.eps);
    float wv[8];
    load4(w + e0, wv);
    load4(w + e0 + 4, wv + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = v[i] * r * wv[i];
  }
  if (a.rot) {
    const int half = a.rot / 2;
    const float* row = a.rope + p * a.rot;
    if constexpr (NEXT) {
      if (turned && e0 < a.rot) {
        float c[4], s[4];
        load4(row + e0 / 2, c);
        load4(row + half + e0 / 2, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = v[2 * i], y = v[2 * i + 1];
          v[2 * i] = x * c[i] - y * s[i];
          v[2 * i + 1] = y * c[i] + x * s[i];
        }
      }
    } else {
      // the other value of each pair is `half` further or back: rot is a
      // multiple of 16, so it is one other lane's same place
      const bool lower = e0 < half, in = e0 < a.rot;
      const int lane = threadIdx.x & 31;
      const int other = in ? (lower ? lane + half / 8 : lane - half / 8) : lane;
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = __shfl_sync(kFull, v[i], other);
      if (turned && in) {
        const int at = lower ? e0 : e0 - half;
        float c[8], s[8];
        load4(row + at, c);
        load4(row + at + 4, c + 4);
        load4(row + half + at, s);
        load4(row + half + at + 4, s + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = lower ? v[i] * c[i] - o[i] * s[i] : v[i] * c[i] + o[i] * s[i];
      }
    }
  }
  if (!live) return;
  uint16_t* dst;
  if (h < a.Hq) {
    dst = a.q + (((int64_t)b * a.Hq + h) * a.T + j) * D;
  } else {
    const int64_t at = (a.slot ? (int64_t)a.slot[b] : 0) + j;
    if (at < 0 || at >= a.kv_cap) return;
    const int kv = h - a.Hq;
    dst = kv < a.Hkv ? a.k + (((int64_t)b * a.Hkv + kv) * a.kv_cap + at) * D
                     : a.v + (((int64_t)b * a.Hkv + kv - a.Hkv) * a.kv_cap + at) * D;
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = (uint32_t)f2h(v[2 * i]) | ((uint32_t)f2h(v[2 * i + 1]) << 16);
  *reinterpret_cast<uint4*>(dst + e0) = make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
void launch(const RopeArgs& a, bool f32, bool next, int64_t tokens, cudaStream_t st) {
  constexpr int HPB = kThreads / (D / 8);
  const dim3 grid((unsigned)tokens, (unsigned)((a.Hq + 2 * a.Hkv + HPB - 1) / HPB));
  if (f32) {
    if (next) norm_rope_kernel<D, true, true><<<grid, kThreads, 0, st>>>(a);
    else norm_rope_kernel<D, true, false><<<grid, kThreads, 0, st>>>(a);
  } else {
    if (next) norm_rope_kernel<D, false, true><<<grid, kThreads, 0, st>>>(a);
    else norm_rope_kernel<D, false, false><<<grid, kThreads, 0, st>>>(a);
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
                       n_pos, kv_cap, T, Hq, Hkv, rot_dim, eps};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int64_t tokens = (int64_t)B * T;
  switch (head_dim) {
    case 64: tq::launch<64>(a, x_dtype == TQ_F32, interleaved, tokens, st); break;
    case 128: tq::launch<128>(a, x_dtype == TQ_F32, interleaved, tokens, st); break;
    default: tq::launch<256>(a, x_dtype == TQ_F32, interleaved, tokens, st); break;
  }
  return cudaGetLastError() == cudaSuccess ? TQ_OK : TQ_ERR_CUDA;
}
