// rope.cu -- rotary positions: lkv_rope_init, lkv_rope_apply and lkv_rope_apply_axes.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <type_traits>

#include "../../include/lkv.h"
#include "cache8.cuh"

namespace lkv {

// A thread turns the pairs of one or two 16-byte vectors of one token's row
// (two where the pairs lie rotary_dim / 2 apart, one where they are
// neighbours), or copies values that do not rotate, for a run of heads: the
// sines and cosines of its pairs are the same for every head of the token, so
// it takes them once. Sizes whose pairs do not fill whole vectors go pair by
// pair (WIDE = 0).
//
// The angle of pair i at position p is p * turn[i] turns. turn[i] is held in
// units of 2^-64, so the product modulo 2^64 is the exact fraction of a turn,
// in two's complement within half a turn of zero; its top 32 bits go to
// sincospif, which needs no argument reduction. Against an angle formed in
// fp32 (wrong by whole radians past position 2^24) this costs one 64-bit
// multiplication a pair, and no fp64 instruction.
//
// Bound: the tensors' bytes, once in and once out. On a GB300, 40 heads x 32K
// tokens of bf16 take 100 us, 98% of the measured copy rate, in either layout
// (148 us before each thread kept eight vectors' loads in flight); one token of
// 8 sequences 1.9 us. Positions on several axes cost a select a pair: 40 heads x
// 32K tokens on three axes 102 us, 97% of the copy rate; 32 heads x 5476 patches
// in fp32 28.6 us, 92%.
constexpr int kRopeThreads = 128;

struct RopeArgs {
  lkv_rope r;
  const void *q, *k;
  void *q_out, *k_out;
  const int32_t *positions;
  int32_t heads, kv_heads, n;
  int32_t per;       // heads (of q and k together) that a thread walks
  int64_t tokens;    // B * n
};

// Positions on several axes, [axes][B][n]: pair i turns by the one on axis[i].
struct RopeAxesArgs : RopeArgs {
  int32_t axes;
  uint8_t axis[64];
};

// A thread's piece of a row: V values at o1 and, for NV = 2, at o2.
template <int DT, int INTER, int WIDE>
struct RopePiece {
  static constexpr int V = !WIDE ? 1 : DT == 1 ? 8 : 4;
  static constexpr int NV = WIDE && INTER ? 1 : 2;
  static constexpr int PAIRS = V * NV / 2;
  static constexpr int TPR = kHeadDim / (V * NV);   // threads of a row
  static constexpr int HB = WIDE ? 8 / NV : 4;      // heads whose loads are in flight together
  float c[PAIRS], s[PAIRS];
  int o1, o2;
  bool rot;

  struct Raw { uint4 w[NV]; float f[2]; };
  __device__ __forceinline__ void load(Raw &r, const void *row) const {
    if constexpr (WIDE) {
      r.w[0] = *(const uint4 *)((const char *)row + o1 * (DT == 1 ? 2 : 4));
      if constexpr (NV == 2) r.w[NV - 1] = *(const uint4 *)((const char *)row + o2 * (DT == 1 ? 2 : 4));
    } else {
      r.f[0] = load_elem<DT>(row, o1);
      r.f[1] = load_elem<DT>(row, o2);
    }
  }
  static __device__ __forceinline__ void unpack(const uint4 &w, float *x) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (DT == 1) {
        x[2 * e] = __uint_as_float(u[e] << 16);
        x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
      } else {
        x[e] = __uint_as_float(u[e]);
      }
    }
  }
  static __device__ __forceinline__ uint4 pack(const float *x) {
    if constexpr (DT == 1)
      return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
    else
      return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  __device__ __forceinline__ void turn(float &x1, float &x2, int e) const {
    const float y = x1 * c[e] - x2 * s[e];
    x2 = x2 * c[e] + x1 * s[e];
    x1 = y;
  }
  __device__ __forceinline__ void store(const Raw &r, void *row) const {
    if constexpr (WIDE) {
      Raw o = r;
      if (rot) {
        float x[V * NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) unpack(r.w[v], x + v * V);
#pragma unroll
        for (int e = 0; e < PAIRS; ++e) turn(x[INTER ? 2 * e : e], x[INTER ? 2 * e + 1 : V * (NV - 1) + e], e);
#pragma unroll
        for (int v = 0; v < NV; ++v) o.w[v] = pack(x + v * V);
      }
      *(uint4 *)((char *)row + o1 * (DT == 1 ? 2 : 4)) = o.w[0];
      if constexpr (NV == 2) *(uint4 *)((char *)row + o2 * (DT == 1 ? 2 : 4)) = o.w[NV - 1];
    } else {
      float x1 = r.f[0], x2 = r.f[1];
      if (rot) turn(x1, x2, 0);
      store_elem<DT>(row, o1, x1);
      store_elem<DT>(row, o2, x2);
    }
  }
};

template <int DT, int INTER, int WIDE, class Args>
__global__ void __launch_bounds__(kRopeThreads) k_rope(const __grid_constant__ Args a) {
  using P = RopePiece<DT, INTER, WIDE>;
  constexpr bool AXES = std::is_same_v<Args, RopeAxesArgs>;
  __shared__ uint64_t turn[64];
  __shared__ uint8_t axis[AXES ? 64 : 1];
  if (threadIdx.x < 64) {
    turn[threadIdx.x] = a.r.turn[threadIdx.x];
    if constexpr (AXES) axis[threadIdx.x] = a.axis[threadIdx.x];
  }
  __syncthreads();
  wait_prerequisites();
  launch_dependents();
  const int64_t id = (int64_t)blockIdx.x * kRopeThreads + threadIdx.x;
  const int64_t tok = id / P::TPR;
  if (tok >= a.tokens) return;
  const int t = (int)(id % P::TPR);
  const int rd = a.r.rotary_dim, half = rd / 2;
  const int64_t b = tok / a.n, i = tok % a.n;
  P p;
  p.rot = t * P::PAIRS < half;
  if (INTER) {
    p.o1 = t * P::V * P::NV;
    p.o2 = p.o1 + P::V;
  } else if (p.rot) {
    p.o1 = t * P::V;
    p.o2 = p.o1 + half;
  } else {  // the rest of the row, in two halves too
    p.o1 = rd + (t - half / P::V) * P::V;
    p.o2 = p.o1 + (kHeadDim - rd) / 2;
  }
  if (p.rot) {
    const int32_t pos = a.positions[tok];
    int32_t pos1 = 0, pos2 = 0, pos3 = 0;
    if constexpr (AXES) {
      static_assert(LKV_ROPE_AXES == 4);
      if (a.axes > 1) pos1 = a.positions[a.tokens + tok];
      if (a.axes > 2) pos2 = a.positions[2 * a.tokens + tok];
      if (a.axes > 3) pos3 = a.positions[3 * a.tokens + tok];
    }
#pragma unroll
    for (int e = 0; e < P::PAIRS; ++e) {
      int64_t at = pos;
      if constexpr (AXES) {
        const int x = axis[t * P::PAIRS + e];
        const int32_t low = x & 1 ? pos1 : pos, high = x & 1 ? pos3 : pos2;
        at = x & 2 ? high : low;
      }
      const int32_t frac = (int32_t)(((uint64_t)at * turn[t * P::PAIRS + e]) >> 32);
      sincospif((float)frac * 0x1p-31f, &p.s[e], &p.c[e]);
      p.s[e] *= a.r.gain;
      p.c[e] *= a.r.gain;
    }
  }
  const int64_t step = (int64_t)a.n * kHeadDim * (DT == 1 ? 2 : 4);  // bytes from head to head
  auto walk = [&](const void *in, void *out, int heads, int h0, int h1) {
    if (!p.rot && in == out) return;  // in place: nothing to copy
    const int64_t at = (b * heads + h0) * step + i * kHeadDim * (DT == 1 ? 2 : 4);
    const char *src = (const char *)in + at;
    char *dst = (char *)out + at;
    for (int h = h0; h < h1; h += P::HB) {
      typename P::Raw r[P::HB];
#pragma unroll
      for (int j = 0; j < P::HB; ++j)
        if (h + j < h1) p.load(r[j], src + j * step);
#pragma unroll
      for (int j = 0; j < P::HB; ++j)
        if (h + j < h1) p.store(r[j], dst + j * step);
      src += P::HB * step;
      dst += P::HB * step;
    }
  };
  const int g0 = (int)blockIdx.y * a.per, g1 = min(g0 + a.per, a.heads + a.kv_heads);
  if (g0 < a.heads) walk(a.q, a.q_out, a.heads, g0, min(g1, a.heads));
  if (g1 > a.heads) walk(a.k, a.k_out, a.kv_heads, max(g0, a.heads) - a.heads, g1 - a.heads);
}

template <int DT, int INTER, int WIDE, class Args>
static cudaError_t launch_rope(Args &a, cudaStream_t st) {
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int64_t threads = a.tokens * RopePiece<DT, INTER, WIDE>::TPR;
  const int64_t blocks = (threads + kRopeThreads - 1) / kRopeThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  // few tokens: the heads are split over CTAs until the GPU is filled once
  const int all = a.heads + a.kv_heads;
  const int64_t want = ((int64_t)sms * 8 + blocks - 1) / blocks;
  a.per = (int)((all + want - 1) / want);
  const int gy = (all + a.per - 1) / a.per;
  if (gy > 65535) return cudaErrorInvalidValue;
  return launch_next(k_rope<DT, INTER, WIDE, Args>, dim3((unsigned)blocks, (unsigned)gy), kRopeThreads, 0, st, a);
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

namespace lkv {

template <class Args>
static cudaError_t launch_rope(Args &a, int32_t dtype, cudaStream_t st) {
  const bool bf = dtype == LKV_DTYPE_BF16, in = a.r.layout == LKV_ROPE_INTERLEAVED;
  // whether the pairs fill whole 16-byte vectors
  const bool wide = a.r.rotary_dim % ((bf ? 8 : 4) * (in ? 1 : 2)) == 0;
  if (bf) return in ? (wide ? launch_rope<1, 1, 1>(a, st) : launch_rope<1, 1, 0>(a, st))
                    : (wide ? launch_rope<1, 0, 1>(a, st) : launch_rope<1, 0, 0>(a, st));
  return in ? (wide ? launch_rope<0, 1, 1>(a, st) : launch_rope<0, 1, 0>(a, st))
            : (wide ? launch_rope<0, 0, 1>(a, st) : launch_rope<0, 0, 0>(a, st));
}

// Both calls: positions [axes][B][n], axis null for one axis.
static lkv_status apply_rope(const char *where, const lkv_rope *rope, const uint8_t *axis, int32_t axes, int32_t dtype,
                             int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t n, const void *q, const void *k,
                             const int32_t *positions, void *q_out, void *k_out, cudaStream_t st) {
  auto no = [&](const char *why) {
    char buf[160];
    std::snprintf(buf, sizeof buf, "%s: %s", where, why);
    return refuse(buf);
  };
  if (!rope) return no("null table");
  if (rope->rotary_dim < 2 || rope->rotary_dim > kHeadDim || rope->rotary_dim % 2 != 0 ||
      (rope->layout != LKV_ROPE_HALF && rope->layout != LKV_ROPE_INTERLEAVED))
    return no("the table was not filled by lkv_rope_init");
  if (axes < 1 || axes > LKV_ROPE_AXES) return no("axes must be 1..4");
  if (axis)
    for (int i = 0; i < rope->rotary_dim / 2; ++i)
      if (axis[i] >= axes) return no("a pair's axis is not one of the axes");
  if (dtype != LKV_DTYPE_FP32 && dtype != LKV_DTYPE_BF16) return no("bad dtype");
  if (batch < 0 || n < 0 || n_heads < 0 || n_kv_heads < 0) return no("negative size");
  if (n_heads > 32768 || n_kv_heads > 32768) return no("at most 32768 heads");
  const int64_t tokens = (int64_t)batch * n;
  if (tokens == 0 || n_heads + n_kv_heads == 0) return LKV_OK;
  if (!positions || (n_heads && (!q || !q_out)) || (n_kv_heads && (!k || !k_out)))
    return no("null tensor");
  if (!aligned(positions, 4) || (n_heads && (!aligned(q, 16) || !aligned(q_out, 16))) ||
      (n_kv_heads && (!aligned(k, 16) || !aligned(k_out, 16))))
    return no("tensors must be 16-byte aligned, positions 4-byte aligned");
  if (tokens > (int64_t(1) << 31)) return no("more than 2^31 tokens");
  const int64_t es = dtype == LKV_DTYPE_BF16 ? 2 : 4;
  const int64_t qb = tokens * n_heads * kHeadDim * es, kb = tokens * n_kv_heads * kHeadDim * es;
  const int64_t pb = tokens * axes * 4;
  if ((q_out != q && overlap(q_out, qb, q, qb)) || (k_out != k && overlap(k_out, kb, k, kb)) ||
      overlap(q_out, qb, k, kb) || overlap(k_out, kb, q, qb) || overlap(q_out, qb, k_out, kb) ||
      overlap(q_out, qb, positions, pb) || overlap(k_out, kb, positions, pb))
    return no("an output overlaps another tensor (in place: the same pointer)");
  RopeAxesArgs a{};
  a.r = *rope;
  a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
  a.positions = positions;
  a.heads = n_heads; a.kv_heads = n_kv_heads; a.n = n;
  a.tokens = tokens;
  cudaError_t e;
  if (axis) {
    a.axes = axes;
    std::memcpy(a.axis, axis, rope->rotary_dim / 2);
    e = launch_rope(a, dtype, st);
  } else {
    e = launch_rope(static_cast<RopeArgs &>(a), dtype, st);
  }
  return e == cudaSuccess ? LKV_OK : cuda_refuse(where, e);
}

}  // namespace lkv

extern "C" lkv_status lkv_rope_apply(const lkv_rope *rope, int32_t dtype, int32_t batch, int32_t n_heads,
                                     int32_t n_kv_heads, int32_t n, const void *q, const void *k,
                                     const int32_t *positions, void *q_out, void *k_out, void *stream) {
  return lkv::apply_rope("lkv_rope_apply", rope, nullptr, 1, dtype, batch, n_heads, n_kv_heads, n, q, k, positions, q_out,
                         k_out, (cudaStream_t)stream);
}

extern "C" lkv_status lkv_rope_apply_axes(const lkv_rope *rope, const uint8_t *axis, int32_t axes, int32_t dtype,
                                          int32_t batch, int32_t n_heads, int32_t n_kv_heads, int32_t n, const void *q,
                                          const void *k, const int32_t *positions, void *q_out, void *k_out, void *stream) {
  if (!axis) return lkv::refuse("lkv_rope_apply_axes: null axes of the pairs");
  return lkv::apply_rope("lkv_rope_apply_axes", rope, axis, axes, dtype, batch, n_heads, n_kv_heads, n, q, k, positions,
                         q_out, k_out, (cudaStream_t)stream);
}
