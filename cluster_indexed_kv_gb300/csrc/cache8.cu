// cache8.cu -- the 8-bit key/value cache: writing, reading back, status.
#include "cache8.cuh"

#include <cuda_fp16.h>

namespace lkv {

constexpr int kCacheThreads = 128;
constexpr int kCacheWarps = kCacheThreads / 32;

const char *check_cache8(const lkv_cache8 *c) {
  if (!c) return "null cache";
  if (c->batch < 1 || c->batch > (1 << 20)) return "batch must be 1..2^20";
  if (c->n_kv_heads < 1 || c->n_kv_heads > 4096) return "n_kv_heads must be 1..4096";
  if (c->capacity < kBlock || c->capacity % kBlock != 0 || c->capacity > (1 << 30))
    return "capacity must be a multiple of 16, 16..2^30";
  if (c->dtype != LKV_DTYPE_FP32 && c->dtype != LKV_DTYPE_BF16) return "bad dtype";
  if (c->code != LKV_CODE_INT8 && c->code != LKV_CODE_E4M3) return "unknown code";
  if (!c->k_codes || !c->v_codes || !c->k_scale || !c->v_scale || !c->k_tail || !c->v_tail || !c->lengths || !c->ticket)
    return "null array of the cache";
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_tail, 16) || !aligned(c->v_tail, 16) ||
      !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) || !aligned(c->lengths, 4) || !aligned(c->ticket, 4))
    return "the cache's codes and tails must be 16-byte aligned, its other arrays 4-byte aligned";
  return nullptr;
}

struct Extent { const void *at; int64_t bytes; };
constexpr int kArrays = 8;
static void extents(const lkv_cache8 *c, Extent (&e)[kArrays]) {
  const int64_t slices = (int64_t)c->batch * c->n_kv_heads, es = c->dtype == LKV_DTYPE_BF16 ? 2 : 4;
  const int64_t codes = slices * c->capacity * kHeadDim, scales = slices * (c->capacity / kBlock) * 4;
  const int64_t tail = slices * kBlock * kHeadDim * es;
  e[0] = {c->k_codes, codes}; e[1] = {c->v_codes, codes};
  e[2] = {c->k_scale, scales}; e[3] = {c->v_scale, scales};
  e[4] = {c->k_tail, tail}; e[5] = {c->v_tail, tail};
  e[6] = {c->lengths, (int64_t)c->batch * 4}; e[7] = {c->ticket, ((int64_t)c->batch + 1) * 4};
}

bool overlaps_cache8(const lkv_cache8 *c, const void *p, int64_t bytes) {
  Extent e[kArrays];
  extents(c, e);
  for (const Extent &x : e)
    if (overlap(p, bytes, x.at, x.bytes)) return true;
  return false;
}

// Whether two of the cache's own arrays share memory.
static bool arrays_overlap(const lkv_cache8 *c) {
  Extent e[kArrays];
  extents(c, e);
  for (int i = 0; i < kArrays; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(e[i].at, e[i].bytes, e[j].at, e[j].bytes)) return true;
  return false;
}

// ---------------------------------------------------------------- write

// The sign of top * a - half * amax. bf16 values: both products are exact
// (8-bit by 9-bit significands). fp32 values: the products are taken with
// their rounding errors (24-bit by 9-bit significands: an error has at most 9
// bits and the difference of two at most 11, so the sum has the exact sign).
// fp64 would do too, at a sixty-fourth of the rate; bf16 inputs sit exactly
// halfway often enough (one value in 600) for that to show.
template <int DT>
__device__ __forceinline__ float halfway_sign(float top, float a, float half, float amax) {
  const float p = top * a;
  if (DT == 1) return __fmaf_rn(-half, amax, p);
  const float r = half * amax;
  return (p - r) + (__fmaf_rn(top, a, -p) - __fmaf_rn(half, amax, -r));
}

template <int DT>
__device__ __forceinline__ uint32_t int8_exact(float x, float inv, float amax) {
  const float a = fabsf(x);
  const float m = rintf(__fmaf_rn(a, inv, -0.5f));  // the halfway point is m + 1/2
  const float d = halfway_sign<DT>(254.f, a, 2.f * m + 1.f, amax);
  const int k = (int)m, up = d > 0.f || (d == 0.f && (k & 1));
  return (uint32_t)(x < 0.f ? -(k + up) : k + up);
}

template <int DT>
__device__ __forceinline__ float e4m3_exact(float x, float inv, float amax) {
  const float a = fabsf(x), q = a * inv;
  // step of the code's binade: 2^(e - 3), 2^-9 below 2^-6
  const uint32_t step = q < 0x1p-6f ? (127u - 9u) << 23 : (__float_as_uint(q) & 0x7f800000u) - (3u << 23);
  const float m = rintf(__fmaf_rn(q, __uint_as_float((254u << 23) - step), -0.5f));
  const float d = halfway_sign<DT>(448.f, a, (m + 0.5f) * __uint_as_float(step), amax);
  const bool up = d > 0.f || (d == 0.f && ((int)m & 1));
  return copysignf((up ? m + 1.f : m) * __uint_as_float(step), x);
}

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ uint32_t pack_low_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

// The codes of x[0..3] in a block of largest magnitude amax, decided exactly;
// inv is 127 / amax or 448 / amax, rounded.
template <int DT, int CODE>
__device__ __noinline__ uint32_t settle4(float x0, float x1, float x2, float x3, float inv, float amax) {
  if constexpr (CODE == LKV_CODE_INT8)
    return pack_low_bytes(int8_exact<DT>(x0, inv, amax), int8_exact<DT>(x1, inv, amax), int8_exact<DT>(x2, inv, amax),
                          int8_exact<DT>(x3, inv, amax));
  else
    return e4m3x2(e4m3_exact<DT>(x0, inv, amax), e4m3_exact<DT>(x1, inv, amax)) |
           (e4m3x2(e4m3_exact<DT>(x2, inv, amax), e4m3_exact<DT>(x3, inv, amax)) << 16);
}

// The same for magnitudes far from 1, scaled by a power of two (exactly, but
// for values whose code is 0): no product overflows or loses bits.
template <int DT, int CODE>
__device__ __noinline__ uint32_t settle4_scaled(float x0, float x1, float x2, float x3, float amax) {
  const float f = amax < 1.f ? 0x1p100f : 0x1p-60f;
  return settle4<DT, CODE>(x0 * f, x1 * f, x2 * f, x3 * f, __fdiv_rn(CODE == LKV_CODE_INT8 ? 127.f : 448.f, amax * f), amax * f);
}

// Codes of N values, four in a word; inv is 127 / amax or 448 / amax, rounded.
// x * inv is off by at most 2 units in its last place; where that could change
// a code the lane decides exactly, as it does everywhere in blocks far from 1.
template <int DT, int CODE, int N>
__device__ __forceinline__ void codes(const float (&x)[N], float inv, float amax, bool far_from_one, uint32_t (&out)[N / 4]) {
  bool settle = false;
  constexpr float kMagic = 12582912.f;  // 1.5 * 2^23: a sum's low bits are the rounded integer
  if constexpr (CODE == LKV_CODE_INT8 && DT == 1) {
    // the remainder 127 x - k amax is exact (16 bits each): halfway or wrong if
    // it is amax / 2 or more
    float top = 0.f;
    float s[N], r[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      s[e] = __fmaf_rn(x[e], inv, kMagic);
      r[e] = __fmaf_rn(kMagic - s[e], amax, 127.f * x[e]);
      top = fmaxf(top, fabsf(r[e]));
    }
    if (2.f * top >= amax) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const bool odd = __float_as_uint(s[e]) & 1u;
        if (2.f * fabsf(r[e]) > amax || (2.f * fabsf(r[e]) == amax && odd)) s[e] += copysignf(1.f, r[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < N / 4; ++e)
      out[e] = pack_low_bytes(__float_as_uint(s[4 * e]), __float_as_uint(s[4 * e + 1]), __float_as_uint(s[4 * e + 2]), __float_as_uint(s[4 * e + 3]));
  } else if constexpr (CODE == LKV_CODE_INT8) {
    float far = 0.f;
    uint32_t r[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float s = __fmaf_rn(x[e], inv, kMagic);
      r[e] = __float_as_uint(s);
      far = fmaxf(far, fabsf(__fmaf_rn(x[e], inv, kMagic - s)));
    }
#pragma unroll
    for (int e = 0; e < N / 4; ++e) out[e] = pack_low_bytes(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
    settle = far > 0.5f - 0x1p-14f;  // |x * inv| < 128 is off by less than 2^-15
  } else {
    uint32_t near = 0xffffffffu, small = 0xffffffffu;
#pragma unroll
    for (int e = 0; e < N / 4; ++e) {
      float q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        q[k] = x[4 * e + k] * inv;
        const uint32_t u = __float_as_uint(q[k]) & 0x7fffffffu;
        near = min(near, (uint32_t)abs((int)(u & 0xfffffu) - 0x80000));  // the 20 bits behind a code
        small = min(small, u - 1u);                                      // zero wraps to the top
      }
      out[e] = e4m3x2(q[0], q[1]) | (e4m3x2(q[2], q[3]) << 16);
    }
    settle = near <= 8u || small < 0x3c800000u;  // below 2^-6 the codes are evenly spaced: settled exactly too
  }
  if (far_from_one) {
#pragma unroll
    for (int e = 0; e < N / 4; ++e) out[e] = settle4_scaled<DT, CODE>(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3], amax);
  } else if (settle) {
#pragma unroll
    for (int e = 0; e < N / 4; ++e) out[e] = settle4<DT, CODE>(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3], inv, amax);
  }
}

// One block of one (sequence, KV head) of K or V: the rows of a block from
// the tail and the new rows, codes and scale where the block is full, and the
// new rows of the last block into the tail.
template <int DT, int CODE>
struct BlockWriter {
  static constexpr int E = DT == 1 ? 8 : 4;         // values of a 16-byte load
  static constexpr int LPR = kHeadDim / E;          // lanes of a row
  static constexpr int RPL = 32 / LPR;              // rows of a load
  static constexpr int NL = kBlock / RPL;           // loads of a block
  const uint4 *src;      // new rows of the slice
  uint4 *tail;           // the slice's tail
  uint8_t *codes_at;     // the slice's codes
  float *scale;          // the slice's scales
  int32_t *anomalies;
  int start, end, lane;

  // largest |x| of two bf16 or one fp32, as bits that order like the values
  static __device__ __forceinline__ uint32_t mag(uint32_t w) {
    return DT == 1 ? w & 0x7fff7fffu : w & 0x7fffffffu;
  }
  static __device__ __forceinline__ uint32_t top(uint32_t a, uint32_t b) {
    return DT == 1 ? __vmaxu2(a, b) : max(a, b);
  }

  static __device__ __forceinline__ float amax_of(const uint4 (&w)[NL]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NL; ++i)
      m = top(m, top(top(mag(w[i].x), mag(w[i].y)), top(mag(w[i].z), mag(w[i].w))));
    if (DT == 1) m = max(m << 16, m & 0xffff0000u);
    return __uint_as_float(__reduce_max_sync(0xffffffffu, m));
  }

  // NaN to 0, infinities to the largest finite value
  static __device__ __forceinline__ uint32_t finite(uint32_t w) {
    if (DT == 1) {
      uint32_t lo = w & 0xffffu, hi = w >> 16;
      if ((lo & 0x7fffu) >= 0x7f80u) lo = (lo & 0x7fffu) > 0x7f80u ? 0u : (lo & 0x8000u) | 0x7f7fu;
      if ((hi & 0x7fffu) >= 0x7f80u) hi = (hi & 0x7fffu) > 0x7f80u ? 0u : (hi & 0x8000u) | 0x7f7fu;
      return lo | (hi << 16);
    }
    if ((w & 0x7fffffffu) < 0x7f800000u) return w;
    return (w & 0x7fffffffu) > 0x7f800000u ? 0u : (w & 0x80000000u) | 0x7f7fffffu;
  }

  __device__ __forceinline__ void put(const uint4 (&w)[NL], int64_t block, float inv, float amax, bool far_from_one) const {
    uint8_t *to = codes_at + (block * kBlock + lane / LPR) * kHeadDim + (lane % LPR) * E;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      float x[E];
      uint32_t c[E / 4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (DT == 1) {
          x[2 * e] = __uint_as_float(u[e] << 16);
          x[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
        } else {
          x[e] = __uint_as_float(u[e]);
        }
      }
      codes<DT, CODE>(x, inv, amax, far_from_one, c);
      if constexpr (DT == 1) *(uint2 *)(to + i * RPL * kHeadDim) = make_uint2(c[0], c[1]);
      else *(uint32_t *)(to + i * RPL * kHeadDim) = c[0];
    }
  }

  __device__ __forceinline__ void block(int j) const {
    uint4 w[NL];
    const int p0 = j * kBlock, sub = lane / LPR, chunk = lane % LPR;
    if (p0 >= start && p0 + kBlock <= end) {  // all new
      const uint4 *from = src + (int64_t)(p0 - start) * LPR + lane;
#pragma unroll
      for (int i = 0; i < NL; ++i) w[i] = __ldcs(from + i * 32);
    } else {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int r = i * RPL + sub, pos = p0 + r;
        w[i] = make_uint4(0, 0, 0, 0);
        if (pos < start) w[i] = tail[r * LPR + chunk];
        else if (pos < end) w[i] = __ldcs(src + (int64_t)(pos - start) * LPR + chunk);
      }
    }
    float amax = amax_of(w);
    if (!(amax <= 0x1.fffffep127f)) {  // an infinity or a NaN
#pragma unroll
      for (int i = 0; i < NL; ++i)
        w[i] = make_uint4(finite(w[i].x), finite(w[i].y), finite(w[i].z), finite(w[i].w));
      amax = amax_of(w);
      if (lane == 0) atomicOr(anomalies, kAnomNotFinite);
    }
    constexpr float kTop = CODE == LKV_CODE_INT8 ? 127.f : 448.f;
    if (p0 + kBlock <= end) {
      if (amax > 0.f) {
        put(w, j, __fdiv_rn(kTop, amax), amax, amax < 0x1p-60f || amax > 0x1p100f);
      } else {
        uint4 *to = (uint4 *)(codes_at + (int64_t)j * kBlock * kHeadDim);
#pragma unroll
        for (int i = 0; i < kBlock * kHeadDim / 512; ++i) to[i * 32 + lane] = make_uint4(0, 0, 0, 0);
      }
      if (lane == 0) scale[j] = __fdiv_rn(amax, kTop);
    }
    __syncwarp();  // every lane has read the tail
    if (p0 + kBlock >= end) {
#pragma unroll
      for (int i = 0; i < NL; ++i) {
        const int r = i * RPL + sub, pos = p0 + r;
        if (pos >= start && pos < end) tail[r * LPR + chunk] = w[i];
      }
    }
  }
};

struct WriteArgs {
  lkv_cache8 c;
  const void *k, *v;
  const int32_t *start, *counts;
  int32_t n;
  int32_t per;        // blocks that a warp takes
  int32_t chunks;     // warps of a (sequence, KV head) and tensor
  int64_t tasks;
};

// A warp takes a run of blocks of one (sequence, KV head) of K or V: a block
// is 16 rows in registers (4 KB of bf16), its largest magnitude one warp
// reduction, its codes one store. Reading, writing and the arithmetic of
// different warps overlap; nothing passes through shared memory.
//
// The tail is read by the first block and written by the last one, so where
// the first block starts in the tail, its warp takes the last block too.
// The last warp of a sequence to finish sets the length (every warp has
// read it by then).
//
// Bound: bytes (2 or 4 in, 1 out a value). On a GB300, 8 x 32K tokens of 8 KV
// heads, bf16 to int8: 273 us, 87% of the measured copy rate; one token of 32
// sequences 4.3 us.
template <int DT, int CODE>
__global__ void __launch_bounds__(kCacheThreads, DT == 1 ? 6 : 3) k_cache8_write(const __grid_constant__ WriteArgs a) {
  wait_prerequisites();
  launch_dependents();
  const int64_t task = (int64_t)blockIdx.x * kCacheWarps + threadIdx.x / 32;
  if (task >= a.tasks) return;
  const lkv_cache8 &c = a.c;
  const int ch = (int)(task % a.chunks);
  const int64_t rest = task / a.chunks;
  const int kv = (int)(rest & 1);
  const int64_t slice = rest >> 1;
  const int b = (int)(slice / c.n_kv_heads);
  const int len = __ldcg(c.lengths + b);
  const int start = a.start ? a.start[b] : len;
  const int cnt = a.counts ? a.counts[b] : a.n;
  int anomaly = 0;
  if (len < 0 || len > c.capacity || cnt < 0 || cnt > a.n) anomaly = kAnomRange;
  else if (cnt > 0) {
    const bool fits = start >= 0 && start <= len && (start % kBlock == 0 || start / kBlock == (len - 1) / kBlock);
    if (!fits) anomaly = kAnomRange;
    else if (cnt > c.capacity - start) anomaly = kAnomCapacity;
  }
  const int end = anomaly ? 0 : start + cnt;
  if (!anomaly && cnt > 0) {
    BlockWriter<DT, CODE> w;
    const int64_t es = DT == 1 ? 2 : 4;
    w.src = (const uint4 *)((const char *)(kv ? a.v : a.k) + slice * a.n * kHeadDim * es);
    w.tail = (uint4 *)((char *)(kv ? c.v_tail : c.k_tail) + slice * kBlock * kHeadDim * es);
    w.codes_at = (uint8_t *)(kv ? c.v_codes : c.k_codes) + slice * c.capacity * kHeadDim;
    w.scale = (kv ? c.v_scale : c.k_scale) + slice * (c.capacity / kBlock);
    w.anomalies = c.ticket + c.batch;
    w.start = start;
    w.end = end;
    w.lane = threadIdx.x & 31;
    const int first = start / kBlock, last = (end - 1) / kBlock;
    const bool both = start % kBlock != 0 && last != first;
    const int j0 = first + ch * a.per, j1 = min(j0 + a.per, last + 1);
    for (int j = j0; j < j1; ++j)
      if (!(both && j == last)) w.block(j);
    if (both && ch == 0) w.block(last);
  }
  __syncwarp();
  // The lengths have been read (they decided the run) when the arrival is
  // issued; the rows need no fence, since only later launches read them.
  if ((threadIdx.x & 31) == 0) {
    const int all = 2 * c.n_kv_heads * a.chunks;
    if (atomicAdd(c.ticket + b, 1) == all - 1) {
      c.ticket[b] = 0;
      if (anomaly) atomicOr(c.ticket + c.batch, anomaly);
      else if (cnt > 0) c.lengths[b] = end;
    }
  }
}

// ---------------------------------------------------------------- read

struct ReadArgs {
  lkv_cache8 c;
  const int32_t *first;
  void *k_out, *v_out;
  int32_t n;
  int32_t groups;     // warps of a (sequence, KV head) and tensor: 16 rows each
  int64_t tasks;
};

template <int CODE>
__device__ __forceinline__ void decode4(uint32_t w, float (&x)[4]) {
  if constexpr (CODE == LKV_CODE_INT8) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = (float)(int8_t)(w >> (8 * e));
  } else {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    const float2 a = __half22float2(*(__half2 *)&lo), b = __half22float2(*(__half2 *)&hi);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  }
}

// A warp takes 16 rows, all its loads first: codes (8 or 4 bytes a lane) and
// the rows' scales, then a product in fp32 a value, rounded to the type. Bound: bytes (1 in, 2
// or 4 out a value). On a GB300, 128K tokens of 8 KV heads to bf16: 115 us, the
// measured copy rate; 777 rows of 2 sequences 4.8 us.
template <int DT, int CODE>
__global__ void __launch_bounds__(kCacheThreads) k_cache8_read(const __grid_constant__ ReadArgs a) {
  constexpr int E = DT == 1 ? 8 : 4, LPR = kHeadDim / E, RPL = 32 / LPR, NL = kBlock / RPL;
  wait_prerequisites();
  const int64_t task = (int64_t)blockIdx.x * kCacheWarps + threadIdx.x / 32;
  if (task >= a.tasks) return;
  const lkv_cache8 &c = a.c;
  const int lane = threadIdx.x & 31, sub = lane / LPR, chunk = lane % LPR;
  const int r0 = (int)(task % a.groups) * kBlock;
  const int64_t rest = task / a.groups;
  const int kv = (int)(rest & 1);
  const int64_t slice = rest >> 1;
  const int b = (int)(slice / c.n_kv_heads);
  const int len = min(max(c.lengths[b], 0), c.capacity), full = len / kBlock * kBlock;
  const int64_t p0 = (int64_t)(a.first ? a.first[b] : 0) + r0;
  const uint8_t *codes = (const uint8_t *)(kv ? c.v_codes : c.k_codes) + slice * c.capacity * kHeadDim;
  const float *scale = (kv ? c.v_scale : c.k_scale) + slice * (c.capacity / kBlock);
  const uint4 *tail = (const uint4 *)((const char *)(kv ? c.v_tail : c.k_tail) + slice * kBlock * kHeadDim * (DT == 1 ? 2 : 4));
  uint4 *out = (uint4 *)((char *)(kv ? a.v_out : a.k_out) + slice * a.n * kHeadDim * (DT == 1 ? 2 : 4));
  uint2 w[NL];
  float s[NL];
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int64_t pos = p0 + i * RPL + sub;
    w[i] = make_uint2(0, 0);
    s[i] = 0.f;
    if (pos >= 0 && pos < full && r0 + i * RPL + sub < a.n) {
      const uint8_t *p = codes + pos * kHeadDim + chunk * E;
      if constexpr (DT == 1) w[i] = __ldcs((const uint2 *)p);
      else w[i].x = __ldcs((const uint32_t *)p);
      s[i] = scale[pos / kBlock];
    }
  }
#pragma unroll
  for (int i = 0; i < NL; ++i) {
    const int r = r0 + i * RPL + sub;
    const int64_t pos = p0 + i * RPL + sub;
    if (r >= a.n) continue;
    uint4 o;
    if (pos >= full && pos < len) {
      o = tail[(int)(pos % kBlock) * LPR + chunk];
    } else {
      float x[4], y[4];
      decode4<CODE>(w[i].x, x);
      if constexpr (DT == 1) {
        decode4<CODE>(w[i].y, y);
        o = make_uint4(pack_bf16(x[0] * s[i], x[1] * s[i]), pack_bf16(x[2] * s[i], x[3] * s[i]),
                       pack_bf16(y[0] * s[i], y[1] * s[i]), pack_bf16(y[2] * s[i], y[3] * s[i]));
      } else {
        o = make_uint4(__float_as_uint(x[0] * s[i]), __float_as_uint(x[1] * s[i]), __float_as_uint(x[2] * s[i]),
                       __float_as_uint(x[3] * s[i]));
      }
    }
    __stcs(out + (int64_t)r * LPR + chunk, o);
  }
}

}  // namespace lkv

extern "C" lkv_status lkv_cache8_write(const lkv_cache8 *c, const void *k, const void *v, int32_t n,
                                       const int32_t *start, const int32_t *counts, void *stream) {
  using namespace lkv;
  if (const char *m = check_cache8(c)) {
    char buf[160];
    std::snprintf(buf, sizeof buf, "lkv_cache8_write: %s", m);
    return refuse(buf);
  }
  if (n < 0) return refuse("lkv_cache8_write: n must be >= 0");
  if (n == 0) return LKV_OK;
  if (!k || !v) return refuse("lkv_cache8_write: null keys or values");
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(start, 4) || !aligned(counts, 4))
    return refuse("lkv_cache8_write: keys and values must be 16-byte aligned, start and counts 4-byte aligned");
  if (arrays_overlap(c)) return refuse("lkv_cache8_write: two of the cache's arrays overlap");
  const int64_t slices = (int64_t)c->batch * c->n_kv_heads;
  const int64_t bytes = slices * n * kHeadDim * (c->dtype == LKV_DTYPE_BF16 ? 2 : 4), ib = (int64_t)c->batch * 4;
  if (overlaps_cache8(c, k, bytes) || overlaps_cache8(c, v, bytes) || overlaps_cache8(c, start, ib) ||
      overlaps_cache8(c, counts, ib))
    return refuse("lkv_cache8_write: an input overlaps the cache's arrays");
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_refuse("lkv_cache8_write", e);
  WriteArgs a{};
  a.c = *c;
  a.k = k; a.v = v; a.start = start; a.counts = counts;
  a.n = n;
  // n rows from any start touch at most this many blocks
  const int64_t touch = ((int64_t)n + 2 * kBlock - 2) / kBlock;
  // runs of blocks, so that fewer warps meet at a sequence's ticket, but
  // only as long as the GPU stays full (32 warps an SM)
  const int64_t per = 2 * slices * touch / ((int64_t)sms * 32 * 4);
  a.per = (int32_t)(per < 1 ? 1 : per > 8 ? 8 : per);
  a.chunks = (int32_t)((touch + a.per - 1) / a.per);
  if (2 * (int64_t)c->n_kv_heads * a.chunks > 0x7fffffff) return refuse("lkv_cache8_write: too many rows");
  a.tasks = 2 * slices * a.chunks;
  const int64_t blocks = (a.tasks + kCacheWarps - 1) / kCacheWarps;
  if (blocks > 0x7fffffff) return refuse("lkv_cache8_write: too many rows");
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf = c->dtype == LKV_DTYPE_BF16, i8 = c->code == LKV_CODE_INT8;
  if (bf && i8) e = launch_next(k_cache8_write<1, LKV_CODE_INT8>, dim3((unsigned)blocks), kCacheThreads, 0, st, a);
  else if (bf) e = launch_next(k_cache8_write<1, LKV_CODE_E4M3>, dim3((unsigned)blocks), kCacheThreads, 0, st, a);
  else if (i8) e = launch_next(k_cache8_write<0, LKV_CODE_INT8>, dim3((unsigned)blocks), kCacheThreads, 0, st, a);
  else e = launch_next(k_cache8_write<0, LKV_CODE_E4M3>, dim3((unsigned)blocks), kCacheThreads, 0, st, a);
  return e == cudaSuccess ? LKV_OK : cuda_refuse("lkv_cache8_write", e);
}

extern "C" lkv_status lkv_cache8_read(const lkv_cache8 *c, const int32_t *first, int32_t n, void *k_out, void *v_out,
                                      void *stream) {
  using namespace lkv;
  if (const char *m = check_cache8(c)) {
    char buf[160];
    std::snprintf(buf, sizeof buf, "lkv_cache8_read: %s", m);
    return refuse(buf);
  }
  if (n < 0) return refuse("lkv_cache8_read: n must be >= 0");
  if (n == 0) return LKV_OK;
  if (!k_out || !v_out) return refuse("lkv_cache8_read: null output");
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(first, 4))
    return refuse("lkv_cache8_read: outputs must be 16-byte aligned, first 4-byte aligned");
  const int64_t slices = (int64_t)c->batch * c->n_kv_heads;
  const int64_t bytes = slices * n * kHeadDim * (c->dtype == LKV_DTYPE_BF16 ? 2 : 4), ib = (int64_t)c->batch * 4;
  if (overlaps_cache8(c, k_out, bytes) || overlaps_cache8(c, v_out, bytes) || overlap(k_out, bytes, v_out, bytes) ||
      overlap(first, ib, k_out, bytes) || overlap(first, ib, v_out, bytes))
    return refuse("lkv_cache8_read: an output overlaps the cache's arrays or another tensor");
  ReadArgs a{};
  a.c = *c;
  a.first = first;
  a.k_out = k_out; a.v_out = v_out;
  a.n = n;
  a.groups = (int32_t)(((int64_t)n + kBlock - 1) / kBlock);
  a.tasks = 2 * slices * a.groups;
  const int64_t blocks = (a.tasks + kCacheWarps - 1) / kCacheWarps;
  if (blocks > 0x7fffffff) return refuse("lkv_cache8_read: too many rows");
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  const bool bf = c->dtype == LKV_DTYPE_BF16, i8 = c->code == LKV_CODE_INT8;
  if (bf && i8) e = launch_next(k_cache8_read<1, LKV_CODE_INT8>, dim3((unsigned)blocks), kCacheThreads, 0, st, a);
  else if (bf) e = launch_next(k_cache8_read<1, LKV_CODE_E4M3>, dim3((unsigned)blocks), kCacheThreads, 0, st, a);
  else if (i8) e = launch_next(k_cache8_read<0, LKV_CODE_INT8>, dim3((unsigned)blocks), kCacheThreads, 0, st, a);
  else e = launch_next(k_cache8_read<0, LKV_CODE_E4M3>, dim3((unsigned)blocks), kCacheThreads, 0, st, a);
  return e == cudaSuccess ? LKV_OK : cuda_refuse("lkv_cache8_read", e);
}

extern "C" lkv_status lkv_cache8_status(const lkv_cache8 *c, void *stream) {
  using namespace lkv;
  if (const char *m = check_cache8(c)) {
    char buf[160];
    std::snprintf(buf, sizeof buf, "lkv_cache8_status: %s", m);
    return refuse(buf);
  }
  cudaStream_t st = (cudaStream_t)stream;
  int32_t bits = 0, *at = c->ticket + c->batch;
  cudaError_t e = cudaMemcpyAsync(&bits, at, sizeof bits, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  if (e == cudaSuccess && bits) e = cudaMemsetAsync(at, 0, sizeof bits, st);
  if (e == cudaSuccess && bits) e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_refuse("lkv_cache8_status", e);
  if (bits & kAnomTimeout) {
    set_unbound_error("lkv_cache8: a device-side wait of an attention gave up; its output is not complete");
    return LKV_ETIMEOUT;
  }
  if (bits & kAnomCapacity) {
    set_unbound_error("lkv_cache8: a write went past the capacity; that sequence was left as it was");
    return LKV_ECAPACITY;
  }
  if (bits & kAnomRange)
    return refuse("lkv_cache8: a write's start or count was out of range; that sequence was left as it was");
  if (bits & kAnomNotFinite) return refuse("lkv_cache8: a NaN or an infinity was written");
  return LKV_OK;
}
