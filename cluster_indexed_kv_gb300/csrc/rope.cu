// rope.cu -- rotary positions: lkv_rope_init and lkv_rope_apply.
#include <cmath>
#include <cstdio>

#include "../../include/lkv.h"
#include "cache8.cuh"

namespace lkv {

// A thread turns V pairs (2 V values) of one token's row, or copies 2 V of
// the values that do not rotate, for a run of heads: the sines and cosines of
// its pairs are the same for every head of the token, so it takes them once.
// V = 8 (16-byte vectors in both layouts) needs rotary_dim % 16 == 0; V = 1
// takes every other even size.
//
// The angle of pair i at position p is p * turn[i] turns. turn[i] is held in
// units of 2^-64, so the product modulo 2^64 is the exact fraction of a turn,
// in two's complement within half a turn of zero; its top 32 bits go to
// sincospif, which needs no argument reduction. Against an angle formed in
// fp32 (wrong by whole radians past position 2^24) this costs one 64-bit
// multiplication a pair, and no fp64 instruction.
//
// Bound: the tensors' bytes, once in and once out.
constexpr int kRopeThreads = 128;

template <int DT, int N>
struct Vals {
  float x[N];
  __device__ __forceinline__ void load(const void *base, int64_t i) {
    if constexpr (N == 1) {
      x[0] = load_elem<DT>(base, i);
    } else if constexpr (DT == 1) {
      const uint4 w = *(const uint4 *)((const uint16_t *)base + i);
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        x[2 * e] = __uint_as_float(u[e] << 16);
        x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
      }
    } else {
#pragma unroll
      for (int h = 0; h < N / 4; ++h) {
        const float4 w = *(const float4 *)((const float *)base + i + 4 * h);
        x[4 * h] = w.x; x[4 * h + 1] = w.y; x[4 * h + 2] = w.z; x[4 * h + 3] = w.w;
      }
    }
  }
  __device__ __forceinline__ void store(void *base, int64_t i) const {
    if constexpr (N == 1) {
      store_elem<DT>(base, i, x[0]);
    } else if constexpr (DT == 1) {
      uint4 w;
      w.x = pack_bf16(x[0], x[1]); w.y = pack_bf16(x[2], x[3]);
      w.z = pack_bf16(x[4], x[5]); w.w = pack_bf16(x[6], x[7]);
      *(uint4 *)((uint16_t *)base + i) = w;
    } else {
#pragma unroll
      for (int h = 0; h < N / 4; ++h)
        *(float4 *)((float *)base + i + 4 * h) = make_float4(x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]);
    }
  }
};

struct RopeArgs {
  lkv_rope r;
  const void *q, *k;
  void *q_out, *k_out;
  const int32_t *positions;
  int32_t heads, kv_heads, n;
  int32_t per;       // heads (of q and k together) that a thread walks
  int64_t tokens;    // B * n
};

template <int DT, int INTER, int V>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const __grid_constant__ RopeArgs a) {
  constexpr int TPR = 64 / V;  // threads of a row
  constexpr int HB = DT == 1 ? 4 : 2;  // heads whose loads are in flight together
  __shared__ uint64_t turn[64];
  if (threadIdx.x < 64) turn[threadIdx.x] = a.r.turn[threadIdx.x];
  __syncthreads();
  const int64_t id = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
  const int64_t tok = id / TPR;
  if (tok >= a.tokens) return;
  const int t = (int)(id % TPR);
  const int rd = a.r.rotary_dim, half = rd / 2;
  const int64_t b = tok / a.n, i = tok % a.n;
  const bool rot = t * V < half;
  float c[V], s[V];
  int o1, o2;  // the two runs of V values
  if (rot) {
    const int64_t pos = a.positions[tok];
#pragma unroll
    for (int e = 0; e < V; ++e) {
      const int32_t frac = (int32_t)(((uint64_t)pos * turn[t * V + e]) >> 32);
      sincospif((float)frac * 0x1p-31f, &s[e], &c[e]);
      s[e] *= a.r.gain;
      c[e] *= a.r.gain;
    }
    o1 = INTER ? 2 * V * t : V * t;
    o2 = INTER ? o1 + V : half + V * t;
  } else {
    o1 = rd + 2 * V * (t - half / V);
    o2 = o1 + V;
  }
  const int h1 = min((int)(blockIdx.y + 1) * a.per, a.heads + a.kv_heads);
  for (int h0 = (int)blockIdx.y * a.per; h0 < h1; h0 += HB) {
    Vals<DT, V> x[HB], y[HB];
    const void *src[HB];
    void *dst[HB];
    int64_t row[HB];
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      const int h = h0 + j;
      if (h >= h1) break;
      const bool isq = h < a.heads;
      src[j] = isq ? a.q : a.k;
      dst[j] = isq ? a.q_out : a.k_out;
      row[j] = ((isq ? b * a.heads + h : b * a.kv_heads + (h - a.heads)) * a.n + i) * kHeadDim;
      x[j].load(src[j], row[j] + o1);
      y[j].load(src[j], row[j] + o2);
    }
#pragma unroll
    for (int j = 0; j < HB; ++j) {
      if (h0 + j >= h1) break;
      if (rot) {
        if constexpr (INTER && V > 1) {
          // V consecutive pairs lie in x, then y
#pragma unroll
          for (int e = 0; e < V / 2; ++e) {
            const float a0 = x[j].x[2 * e], a1 = x[j].x[2 * e + 1], b0 = y[j].x[2 * e], b1 = y[j].x[2 * e + 1];
            x[j].x[2 * e] = a0 * c[e] - a1 * s[e];
            x[j].x[2 * e + 1] = a1 * c[e] + a0 * s[e];
            y[j].x[2 * e] = b0 * c[V / 2 + e] - b1 * s[V / 2 + e];
            y[j].x[2 * e + 1] = b1 * c[V / 2 + e] + b0 * s[V / 2 + e];
          }
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) {
            const float x1 = x[j].x[e], x2 = y[j].x[e];
            x[j].x[e] = x1 * c[e] - x2 * s[e];
            y[j].x[e] = x2 * c[e] + x1 * s[e];
          }
        }
      } else if (src[j] == dst[j]) {
        continue;  // in place: nothing to copy
      }
      x[j].store(dst[j], row[j] + o1);
      y[j].store(dst[j], row[j] + o2);
    }
  }
}

template <int DT, int INTER, int V>
static cudaError_t launch_rope(RopeArgs &a, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int64_t threads = a.tokens * (64 / V);
  const int64_t blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  // few tokens: the heads are split over CTAs until the GPU is filled once
  const int all = a.heads + a.kv_heads;
  const int64_t want = ((int64_t)sms * 8 + blocks - 1) / blocks;
  a.per = (int)((all + want - 1) / want);
  const int gy = (all + a.per - 1) / a.per;
  if (gy > 65535) return cudaErrorInvalidValue;
  k_rope<DT, INTER, V><<<dim3((unsigned)blocks, (unsigned)gy), kRopeThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace lkv

extern "C" lkv_status lkv_rope_init(const lkv_rope_params *p, lkv_rope *rope) {
  using namespace lkv;
  if (!p || !rope) return refuse("lkv_rope_init: null argument");
  const int rd = p->rotary_dim;
  if (rd < 2 || rd > kHeadDim || rd % 2 != 0) return refuse("lkv_rope_init: rotary_dim must be even, 2..128");
  if (p->layout != LKV_ROPE_HALF && p->layout != LKV_ROPE_INTERLEAVED) return refuse("lkv_rope_init: unknown layout");
  if (p->scaling < LKV_ROPE_NONE || p->scaling > LKV_ROPE_YARN) return refuse("lkv_rope_init: unknown scaling");
  if (!(p->base >= 1.0) || !std::isfinite(p->base)) return refuse("lkv_rope_init: base must be finite and >= 1");
  double base = p->base, gain = 1.0;
  const double factor = p->factor;
  if (p->scaling != LKV_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return refuse("lkv_rope_init: factor must be finite and >= 1");
  if (p->scaling == LKV_ROPE_NTK) {
    if (rd == 2) return refuse("lkv_rope_init: LKV_ROPE_NTK needs rotary_dim > 2");
    base *= std::pow(factor, (double)rd / (rd - 2));
    if (!std::isfinite(base)) return refuse("lkv_rope_init: base * factor^(rotary_dim / (rotary_dim - 2)) overflows");
  }
  if (p->scaling == LKV_ROPE_YARN) {
    if (p->orig_len < 1) return refuse("lkv_rope_init: LKV_ROPE_YARN needs orig_len >= 1");
    if (!(p->beta_fast > p->beta_slow) || !(p->beta_slow >= 0.0) || !std::isfinite(p->beta_fast))
      return refuse("lkv_rope_init: LKV_ROPE_YARN needs beta_fast > beta_slow >= 0");
    gain = 0.1 * std::log(factor) + 1.0;
  }
  const double two_pi = 6.283185307179586476925;
  rope->rotary_dim = rd;
  rope->layout = p->layout;
  rope->gain = (float)gain;
  rope->reserved = 0;
  for (int i = 0; i < 64; ++i) {
    rope->turn[i] = 0;
    if (i >= rd / 2) continue;
    double f = std::pow(base, -2.0 * i / rd);
    if (p->scaling == LKV_ROPE_LINEAR) f /= factor;
    if (p->scaling == LKV_ROPE_YARN) {
      const double r = p->orig_len * f / two_pi;
      const double g = std::fmin(1.0, std::fmax(0.0, (r - p->beta_slow) / (p->beta_fast - p->beta_slow)));
      f = f * g + f * (1.0 - g) / factor;
    }
    rope->turn[i] = (uint64_t)std::nearbyint(std::ldexp(f / two_pi, 64));  // f <= 1: below 2^62
  }
  return LKV_OK;
}

extern "C" lkv_status lkv_rope_apply(const lkv_rope *rope, int32_t dtype, int32_t batch, int32_t n_heads,
                                     int32_t n_kv_heads, int32_t n, const void *q, const void *k,
                                     const int32_t *positions, void *q_out, void *k_out, void *stream) {
  using namespace lkv;
  if (!rope) return refuse("lkv_rope_apply: null table");
  if (rope->rotary_dim < 2 || rope->rotary_dim > kHeadDim || rope->rotary_dim % 2 != 0 ||
      (rope->layout != LKV_ROPE_HALF && rope->layout != LKV_ROPE_INTERLEAVED))
    return refuse("lkv_rope_apply: the table was not filled by lkv_rope_init");
  if (dtype != LKV_DTYPE_FP32 && dtype != LKV_DTYPE_BF16) return refuse("lkv_rope_apply: bad dtype");
  if (batch < 0 || n < 0 || n_heads < 0 || n_kv_heads < 0) return refuse("lkv_rope_apply: negative size");
  if (n_heads > 32768 || n_kv_heads > 32768) return refuse("lkv_rope_apply: at most 32768 heads");
  const int64_t tokens = (int64_t)batch * n;
  if (tokens == 0 || n_heads + n_kv_heads == 0) return LKV_OK;
  if (!positions || (n_heads && (!q || !q_out)) || (n_kv_heads && (!k || !k_out)))
    return refuse("lkv_rope_apply: null tensor");
  if (!aligned(positions, 4) || (n_heads && (!aligned(q, 16) || !aligned(q_out, 16))) ||
      (n_kv_heads && (!aligned(k, 16) || !aligned(k_out, 16))))
    return refuse("lkv_rope_apply: tensors must be 16-byte aligned, positions 4-byte aligned");
  if (tokens > (int64_t(1) << 31)) return refuse("lkv_rope_apply: more than 2^31 tokens");
  const int64_t es = dtype == LKV_DTYPE_BF16 ? 2 : 4;
  const int64_t qb = tokens * n_heads * kHeadDim * es, kb = tokens * n_kv_heads * kHeadDim * es;
  const int64_t pb = tokens * 4;
  if ((q_out != q && overlap(q_out, qb, q, qb)) || (k_out != k && overlap(k_out, kb, k, kb)) ||
      overlap(q_out, qb, k, kb) || overlap(k_out, kb, q, qb) || overlap(q_out, qb, k_out, kb) ||
      overlap(q_out, qb, positions, pb) || overlap(k_out, kb, positions, pb))
    return refuse("lkv_rope_apply: an output overlaps another tensor (in place: the same pointer)");
  RopeArgs a{};
  a.r = *rope;
  a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
  a.positions = positions;
  a.heads = n_heads; a.kv_heads = n_kv_heads; a.n = n;
  a.tokens = tokens;
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf = dtype == LKV_DTYPE_BF16, in = rope->layout == LKV_ROPE_INTERLEAVED;
  const bool wide = rope->rotary_dim % 16 == 0;
  cudaError_t e;
  if (bf) e = in ? (wide ? launch_rope<1, 1, 8>(a, st) : launch_rope<1, 1, 1>(a, st))
                 : (wide ? launch_rope<1, 0, 8>(a, st) : launch_rope<1, 0, 1>(a, st));
  else e = in ? (wide ? launch_rope<0, 1, 8>(a, st) : launch_rope<0, 1, 1>(a, st))
              : (wide ? launch_rope<0, 0, 8>(a, st) : launch_rope<0, 0, 1>(a, st));
  return e == cudaSuccess ? LKV_OK : cuda_refuse("lkv_rope_apply", e);
}
