// attend8.cu -- causal attention over the 8-bit cache (lkv_cache8_attend).
#include "cache8.cuh"

#include <cuda_fp16.h>

namespace lkv {

constexpr int kAtThreads = 128;
constexpr int kAtWarps = kAtThreads / 32;
constexpr int kAtMaxCluster = 16;
constexpr float kLog2e = 1.4426950408889634f;

struct AttendArgs {
  lkv_cache8 c;
  const void *q;
  void *out;
  const int32_t *counts;
  int32_t n, group, window, sinks;
  int32_t row_tiles;
  float scale_log2;   // scale * log2(e)
};

// c += a * b, fp16 operands, fp32 accumulators
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *(const uint32_t *)&h; }

// 2^e as a float, e clamped to the normal range
__device__ __forceinline__ float pow2f(int e) {
  return __uint_as_float((uint32_t)(min(max(e, -126), 127) + 127) << 23);
}

// x (fp32) as an fp16 value and an fp16 remainder
__device__ __forceinline__ void split_h2(float x, float y, uint32_t &hi, uint32_t &lo) {
  const __half2 h = __floats2half2_rn(x, y);
  const float2 f = __half22float2(h);
  hi = h2_bits(h);
  lo = h2_bits(__floats2half2_rn(x - f.x, y - f.y));
}

// The two fp16 pairs of the four codes in w (exact in fp16).
template <int CODE>
__device__ __forceinline__ void codes_row(uint32_t w, uint32_t &p01, uint32_t &p23) {
  if constexpr (CODE == LKV_CODE_INT8) {
    const uint32_t u = w ^ 0x80808080u;  // x + 128; 0x6400 | u is 1024 + u in fp16
    const __half2 off = __float2half2_rn(1152.f);
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    p01 = h2_bits(__hsub2(*(const __half2 *)&a, off));
    p23 = h2_bits(__hsub2(*(const __half2 *)&b, off));
  } else {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(p01), "=r"(p23) : "r"(w));
  }
}

// Bytes 2 h and 2 h + 1 of two tokens' words as two fp16 pairs across the tokens.
template <int CODE>
__device__ __forceinline__ void codes_across(uint32_t wa, uint32_t wb, int h, uint32_t &even, uint32_t &odd) {
  if constexpr (CODE == LKV_CODE_INT8) {
    const uint32_t u = __byte_perm(wa, wb, h ? 0x7632 : 0x5410) ^ 0x80808080u;
    const __half2 off = __float2half2_rn(1152.f);
    const uint32_t a = __byte_perm(u, 0x64646464u, 0x4240), b = __byte_perm(u, 0x64646464u, 0x4341);
    even = h2_bits(__hsub2(*(const __half2 *)&a, off));
    odd = h2_bits(__hsub2(*(const __half2 *)&b, off));
  } else {
    const uint32_t u = __byte_perm(wa, wb, h ? 0x7362 : 0x5140);
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(even), "=r"(odd) : "r"(u));
  }
}

// The attention of RT = 8 NT rows (a row is one query head of one token; the
// rows of a KV head are ordered token-major) over a share of the visible
// blocks of one (sequence, KV head).
//
// A warp takes one block of 16 tokens at a time. Scores are mma.sync
// m16n8k16 products with the rows as M (fp16; rows 8..15 hold the remainders
// of fp32 queries, or a second 8 rows) and 8 tokens as N; the contraction's
// order over d is free, so a lane's K operands are 16-byte runs of a token's
// row, straight from global memory. P V takes 16 values of d as M, the 16
// tokens as K and 8 rows as N: the score accumulators are its B operand as
// they stand, and a lane's V operands are again 16-byte runs of four tokens.
// 8-bit codes are exact in fp16. The queries are scaled by a power of two
// into fp16's range, scores get the block's K scale in fp32, and each block's
// P V partial gets its V scale in fp32 when it is added.
//
// Softmax in base 2 with a reference per row that only moves when a score
// passes it by 2^8: the weights lie below 2^(8 + kPShift) <= 2^15, fp16's
// range, and small ones keep 2^-30 of the reference. For fp32 outputs the
// weights carry an fp16 remainder too (one more product a block).
//
// The shares of a tile of rows are the CTAs of one cluster. Each CTA merges
// its warps in shared memory, then every CTA of the cluster merges a part of
// the outputs over distributed shared memory: one launch, no workspace, no
// atomics, the same result each time.
constexpr float kPShift = 6.f;
constexpr float kSlack = 8.f;

template <int NT>
struct AtSmem {
  static constexpr int RT = 8 * NT;
  static constexpr int RS = 20;               // floats between rows (bank spread)
  static constexpr int IS = RT * RS + 8;      // floats between the 8 d-pair planes
  float o[kAtWarps][8 * IS];
  float part[RT][kHeadDim];                   // the CTA's merged partial
  float m[kAtWarps][RT], l[kAtWarps][RT];
  float f[kAtWarps][RT];
  float pm[RT], pl[RT];
};

template <int DT, int CODE, int NT>
struct Warp {
  static constexpr int RT = 8 * NT;
  static constexpr bool SPLIT = DT == 0;      // fp32: operands with remainders
  static constexpr int QL = SPLIT && NT == 2 ? 2 : 1;
  uint32_t qa[QL][8][4];      // A fragments of the queries for the 8 steps over d
  float rc[NT];               // row g (+8): query scale * scale * log2(e)
  int pos[NT];                // its position, -1 for none
  float mref[NT], l[NT];
  float o[NT][8][4];
  int lane, g, t;
  int pmin, pmax, window, sinks;

  // Scores of the block, masked, turned into weights; the reference moves if needed.
  __device__ __forceinline__ void weights(float (&s)[2][4], float ks, int block, uint32_t (&ph)[NT][2], uint32_t (&pl)[NT][2]) {
    const int p0 = block * kBlock;
    float x[NT][4];
    bool jump = false;
    const bool all = p0 + kBlock - 1 <= pmin &&
                     (window == 0 || p0 > pmax - window || p0 + kBlock <= sinks);
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const float f = rc[r] * ks;
      const bool rem = SPLIT && NT == 1;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = e >> 1, col = e & 1;
        float v = s[j][2 * r + col];
        if (rem) v += s[j][2 + col];
        v *= f;
        if (!all) {
          const int tok = p0 + 8 * j + 2 * t + col;
          if (!(tok <= pos[r] && (window == 0 || tok > pos[r] - window || tok < sinks))) v = -INFINITY;
        }
        x[r][e] = v;
        jump |= v > mref[r] + kSlack;
      }
    }
    if (__any_sync(0xffffffffu, jump)) {
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        float m = fmaxf(fmaxf(x[r][0], x[r][1]), fmaxf(x[r][2], x[r][3]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        const float now = fmaxf(mref[r], m);
        const float k = now == -INFINITY ? 1.f : exp2f(mref[r] - now);
        mref[r] = now;
        l[r] *= k;
        // accumulator columns are rows 2 t and 2 t + 1
        const float ka = __shfl_sync(0xffffffffu, k, 8 * t), kb = __shfl_sync(0xffffffffu, k, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[r][i][0] *= ka; o[r][i][1] *= kb; o[r][i][2] *= ka; o[r][i][3] *= kb;
        }
      }
    }
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      const float ref = mref[r] == -INFINITY ? 0.f : mref[r] - kPShift;
      float p[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[e] = exp2f(x[r][e] - ref);
        l[r] += p[e];
      }
      if (SPLIT) {
        split_h2(p[0], p[1], ph[r][0], pl[r][0]);
        split_h2(p[2], p[3], ph[r][1], pl[r][1]);
      } else {
        ph[r][0] = h2_bits(__floats2half2_rn(p[0], p[1]));
        ph[r][1] = h2_bits(__floats2half2_rn(p[2], p[3]));
      }
    }
  }

  // One quantised block: k[2][2] are the lane's K runs (tokens g and 8 + g,
  // d 16 t.. and 64 + 16 t..), v[4] its V runs (tokens 2 t, 2 t + 1, 8 + 2 t,
  // 9 + 2 t, d 16 g..).
  __device__ __forceinline__ void step(const uint4 (&k)[2][2], const uint4 (&v)[4], float ks, float vs, int block) {
    float s[2][4] = {};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t w = e == 0 ? k[j][c].x : e == 1 ? k[j][c].y : e == 2 ? k[j][c].z : k[j][c].w;
          uint32_t b0, b1;
          codes_row<CODE>(w, b0, b1);
          mma16816(s[j], qa[0][4 * c + e], b0, b1);
          if (QL == 2) mma16816(s[j], qa[QL - 1][4 * c + e], b0, b1);
        }
      }
    }
    uint32_t ph[NT][2], pl[NT][2];
    weights(s, ks, block, ph, pl);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = e == 0 ? v[j].x : e == 1 ? v[j].y : e == 2 ? v[j].z : v[j].w;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[4];
        codes_across<CODE>(w[0], w[1], h, a[0], a[1]);
        codes_across<CODE>(w[2], w[3], h, a[2], a[3]);
        accumulate(a, ph, pl, vs, 2 * e + h);
      }
    }
  }

  __device__ __forceinline__ void accumulate(const uint32_t (&a)[4], const uint32_t (&ph)[NT][2], const uint32_t (&pl)[NT][2],
                                             float vs, int i) {
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      float c[4] = {};
      mma16816(c, a, ph[r][0], ph[r][1]);
      if (SPLIT) mma16816(c, a, pl[r][0], pl[r][1]);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[r][i][e] += vs * c[e];
    }
  }

  // Four consecutive values of a tail row; zeros for rows that are not there.
  __device__ __forceinline__ float4 tail4(const void *tail, int row, int d, int rows) const {
    if (row >= rows) return make_float4(0.f, 0.f, 0.f, 0.f);
    if (DT == 1) {
      const uint2 w = *(const uint2 *)((const uint16_t *)tail + row * kHeadDim + d);
      return make_float4(__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u), __uint_as_float(w.y << 16),
                         __uint_as_float(w.y & 0xffff0000u));
    }
    return *(const float4 *)((const float *)tail + row * kHeadDim + d);
  }

  // A power of two that brings the tail's largest magnitude below 1.
  __device__ __forceinline__ int tail_exp(const void *tail, int rows) const {
    float m = 0.f;
    for (int row = 0; row < rows; ++row) {
      const float4 x = tail4(tail, row, 4 * lane, rows);
      m = fmaxf(m, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
    return min(max((int)(top >> 23) - 126, -100), 126);
  }

  // The last, partial block, from the tails in full precision: the same
  // products on fp16 values and (fp32 tails) their remainders.
  __device__ __noinline__ void tail_step(const void *kt, const void *vt, int rows, int block) {
    const int ke = tail_exp(kt, rows), ve = tail_exp(vt, rows);
    const float kf = pow2f(-ke), vf = pow2f(-ve);
    float s[2][4] = {};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 x = tail4(kt, 8 * j + g, 64 * c + 16 * t + 4 * e, rows);
          uint32_t h0, h1, l0, l1;
          split_h2(x.x * kf, x.y * kf, h0, l0);
          split_h2(x.z * kf, x.w * kf, h1, l1);
#pragma unroll
          for (int z = 0; z < QL; ++z) {
            mma16816(s[j], qa[z][4 * c + e], h0, h1);
            if (SPLIT) mma16816(s[j], qa[z][4 * c + e], l0, l1);
          }
        }
      }
    }
    uint32_t ph[NT][2], pl[NT][2];
    weights(s, pow2f(ke), block, ph, pl);
    const int tok[4] = {2 * t, 2 * t + 1, 8 + 2 * t, 9 + 2 * t};
    const float back = pow2f(ve);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = tail4(vt, tok[j], 16 * g + 4 * e, rows);
        x[j].x *= vf; x[j].y *= vf; x[j].z *= vf; x[j].w *= vf;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[4], b[4];
        split_h2(h ? x[0].z : x[0].x, h ? x[1].z : x[1].x, a[0], b[0]);
        split_h2(h ? x[0].w : x[0].y, h ? x[1].w : x[1].y, a[1], b[1]);
        split_h2(h ? x[2].z : x[2].x, h ? x[3].z : x[3].x, a[2], b[2]);
        split_h2(h ? x[2].w : x[2].y, h ? x[3].w : x[3].y, a[3], b[3]);
        accumulate(a, ph, pl, back, 2 * e + h);
        if (SPLIT) accumulate(b, ph, pl, back, 2 * e + h);
      }
    }
  }
};

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive;\n\tbarrier.cluster.wait;" ::: "memory");
}
// float at p's place in the shared memory of CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer_addr(const void *p, uint32_t rank) {
  uint32_t a = (uint32_t)__cvta_generic_to_shared(p), r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(rank));
  return r;
}
__device__ __forceinline__ float peer_f(const void *p, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(peer_addr(p, rank)));
  return v;
}
__device__ __forceinline__ float2 peer_f2(const void *p, uint32_t rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(peer_addr(p, rank)));
  return v;
}

// 2^(m - top), 0 for a share that saw nothing
__device__ __forceinline__ float share(float m, float top) { return m == -INFINITY ? 0.f : exp2f(m - top); }

template <int DT, int CODE, int NT>
__global__ void __launch_bounds__(kAtThreads) k_attend8(const __grid_constant__ AttendArgs a) {
  extern __shared__ __align__(16) unsigned char raw[];
  AtSmem<NT> &sm = *(AtSmem<NT> *)raw;
  constexpr int RT = 8 * NT;
  using W = Warp<DT, CODE, NT>;
  const lkv_cache8 &c = a.c;
  const int parts = (int)cluster_size(), part = (int)cluster_rank();
  const int wid = threadIdx.x >> 5;
  const int64_t tile = blockIdx.x / parts;
  const int64_t S = (int64_t)c.batch * c.n_kv_heads;
  const int64_t slice = tile % S;
  const int rt = a.row_tiles - 1 - (int)(tile / S);  // the rows with most to see come first
  const int b = (int)(slice / c.n_kv_heads), h = (int)(slice % c.n_kv_heads);
  const int len = min(max(c.lengths[b], 0), c.capacity);
  const int cnt = a.counts ? min(max(a.counts[b], 0), a.n) : a.n;
  const int R = a.n * a.group, r0 = rt * RT;

  W w;
  w.lane = threadIdx.x & 31;
  w.g = w.lane >> 2;
  w.t = w.lane & 3;
  w.window = a.window;
  w.sinks = a.sinks;
  const int imin = r0 / a.group, imax = min((min(r0 + RT, R) - 1) / a.group, cnt - 1);
  w.pmin = len - cnt + imin;
  w.pmax = imin <= imax ? len - cnt + imax : -1;

  // the visible blocks: the first `sb` (sinks), then lo..hi
  const int lo = a.window > 0 ? max(0, w.pmin - a.window + 1) / kBlock : 0;
  const int hi = w.pmax >= 0 ? w.pmax / kBlock : -1;
  const int sb = a.window > 0 && hi >= 0 ? min((min(a.sinks, len) + kBlock - 1) / kBlock, lo) : 0;
  const int nb = hi >= 0 ? sb + hi - lo + 1 : 0;
  const int64_t es = DT == 1 ? 2 : 4;

#pragma unroll
  for (int r = 0; r < NT; ++r) {
    w.mref[r] = -INFINITY;
    w.l[r] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) w.o[r][i][e] = 0.f;
  }
  // queries: row g (and g + 8), the 32 values of d that go with the lane's K runs
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    const int row = r0 + 8 * r + w.g;
    const int i = row / a.group;
    const bool valid = row < R && i < cnt;
    w.pos[r] = valid ? len - cnt + i : -1;
    float x[32];
    const char *p = (const char *)a.q +
                    (((int64_t)(b * (int64_t)c.n_kv_heads + h) * a.group + (valid ? row % a.group : 0)) * a.n + (valid ? i : 0)) * kHeadDim * es;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float4 v = valid ? w.tail4(p, 0, 64 * (u >> 2) + 16 * w.t + 4 * (u & 3), 1) : make_float4(0.f, 0.f, 0.f, 0.f);
      x[4 * u] = v.x; x[4 * u + 1] = v.y; x[4 * u + 2] = v.z; x[4 * u + 3] = v.w;
    }
    float m = 0.f;
#pragma unroll
    for (int u = 0; u < 32; ++u) m = fmaxf(m, fabsf(x[u]));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const int e = min(max((int)(__float_as_uint(m) >> 23) - 126, -100), 126);
    const float f = pow2f(-e);
    w.rc[r] = pow2f(e) * a.scale_log2;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      uint32_t h0, h1, l0, l1;
      split_h2(x[4 * u] * f, x[4 * u + 1] * f, h0, l0);
      split_h2(x[4 * u + 2] * f, x[4 * u + 3] * f, h1, l1);
      w.qa[0][u][r] = h0;
      w.qa[0][u][2 + r] = h1;
      if (W::SPLIT && NT == 1) { w.qa[0][u][1] = l0; w.qa[0][u][3] = l1; }
      if (!W::SPLIT && NT == 1) { w.qa[0][u][1] = 0; w.qa[0][u][3] = 0; }
      if (W::QL == 2) { w.qa[W::QL - 1][u][r] = l0; w.qa[W::QL - 1][u][2 + r] = l1; }
    }
  }

  const uint8_t *kc = (const uint8_t *)c.k_codes + slice * c.capacity * kHeadDim;
  const uint8_t *vc = (const uint8_t *)c.v_codes + slice * c.capacity * kHeadDim;
  const float *ksc = c.k_scale + slice * (c.capacity / kBlock), *vsc = c.v_scale + slice * (c.capacity / kBlock);
  const int full = len / kBlock;   // blocks before it are quantised
  const int b0 = (int)((int64_t)nb * part / parts), b1 = (int)((int64_t)nb * (part + 1) / parts);
  const bool tail = nb > 0 && hi >= full && b1 == nb && b1 > b0;  // the share's last block is the partial one
  const int b2 = tail ? b1 - 1 : b1;
  auto block_of = [&](int u) { return u < sb ? u : u - sb + lo; };

  struct Frag { uint4 k[2][2], v[4]; };
  auto load = [&](Frag &f, int u) {
    const int64_t at = (int64_t)block_of(u) * kBlock * kHeadDim;
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int cc = 0; cc < 2; ++cc)
        f.k[j][cc] = __ldg((const uint4 *)(kc + at + (8 * j + w.g) * kHeadDim + 64 * cc + 16 * w.t));
    const int tok[4] = {2 * w.t, 2 * w.t + 1, 8 + 2 * w.t, 9 + 2 * w.t};
#pragma unroll
    for (int j = 0; j < 4; ++j) f.v[j] = __ldg((const uint4 *)(vc + at + tok[j] * kHeadDim + 16 * w.g));
  };
  Frag x, y;
  float ks = 0.f, vs = 0.f;
  int u = b0 + wid, k = 0;
  if (u < b2) load(x, u);
  auto one = [&](Frag &cur, Frag &next) {
    if ((k & 31) == 0) {  // the scales of the warp's next 32 blocks
      const int mine = u + w.lane * kAtWarps;
      if (mine < b2) {
        ks = ksc[block_of(mine)];
        vs = vsc[block_of(mine)];
      }
    }
    if (u + kAtWarps < b2) load(next, u + kAtWarps);
    w.step(cur.k, cur.v, __shfl_sync(0xffffffffu, ks, k & 31), __shfl_sync(0xffffffffu, vs, k & 31), block_of(u));
    u += kAtWarps;
    ++k;
  };
  while (u < b2) {
    one(x, y);
    if (u >= b2) break;
    one(y, x);
  }
  if (tail && wid == kAtWarps - 1) {
    W z = w;  // a copy: w itself stays in registers
    z.tail_step((const char *)c.k_tail + slice * kBlock * kHeadDim * es, (const char *)c.v_tail + slice * kBlock * kHeadDim * es,
                len - full * kBlock, full);
    w = z;
  }

  // the warps' partials
#pragma unroll
  for (int r = 0; r < NT; ++r) {
    float l = w.l[r];
    l += __shfl_xor_sync(0xffffffffu, l, 1);
    l += __shfl_xor_sync(0xffffffffu, l, 2);
    if (w.t == 0) {
      sm.m[wid][8 * r + w.g] = w.mref[r];
      sm.l[wid][8 * r + w.g] = l;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        *(float2 *)&sm.o[wid][i * AtSmem<NT>::IS + (8 * r + 2 * w.t + e) * AtSmem<NT>::RS + 2 * w.g] =
            make_float2(w.o[r][i][e], w.o[r][i][2 + e]);
  }
  __syncthreads();
  if (threadIdx.x < RT) {
    const int row = threadIdx.x;
    float top = -INFINITY, l = 0.f;
#pragma unroll
    for (int j = 0; j < kAtWarps; ++j) top = fmaxf(top, sm.m[j][row]);
#pragma unroll
    for (int j = 0; j < kAtWarps; ++j) {
      const float f = share(sm.m[j][row], top);
      sm.f[j][row] = f;
      l += f * sm.l[j][row];
    }
    sm.pm[row] = top;
    sm.pl[row] = l;
  }
  __syncthreads();
  auto finish = [&](int row, int d, float2 o, float l) {
    const int rr = r0 + row, i = rr / a.group;
    if (rr >= R) return;
    if (i >= cnt || l == 0.f) o = make_float2(0.f, 0.f);
    else { o.x = o.x / l; o.y = o.y / l; }
    const int64_t at = (((int64_t)(b * (int64_t)c.n_kv_heads + h) * a.group + rr % a.group) * a.n + i) * kHeadDim + d;
    if (DT == 1) *(uint32_t *)((uint16_t *)a.out + at) = pack_bf16(o.x, o.y);
    else *(float2 *)((float *)a.out + at) = o;
  };
  for (int it = threadIdx.x; it < RT * 64; it += kAtThreads) {
    const int row = it >> 6, p = it & 63;  // values 2 p, 2 p + 1: plane p % 8 of group p / 8
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kAtWarps; ++j) {
      const float2 x2 = *(const float2 *)&sm.o[j][(p & 7) * AtSmem<NT>::IS + row * AtSmem<NT>::RS + 2 * (p >> 3)];
      const float f = sm.f[j][row];
      s.x += f * x2.x;
      s.y += f * x2.y;
    }
    if (parts == 1) finish(row, 2 * p, s, sm.pl[row]);
    else *(float2 *)&sm.part[row][2 * p] = s;
  }
  if (parts == 1) return;
  cluster_barrier();
  for (int it = threadIdx.x + part * kAtThreads; it < RT * 64; it += parts * kAtThreads) {
    const int row = it >> 6, p = it & 63;
    float m[kAtMaxCluster], top = -INFINITY, l = 0.f;
#pragma unroll
    for (int j = 0; j < kAtMaxCluster; ++j) {
      if (j >= parts) break;
      m[j] = peer_f(&sm.pm[row], j);
      top = fmaxf(top, m[j]);
    }
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < kAtMaxCluster; ++j) {
      if (j >= parts) break;
      const float f = share(m[j], top);
      const float2 x2 = peer_f2(&sm.part[row][2 * p], j);
      l += f * peer_f(&sm.pl[row], j);
      s.x += f * x2.x;
      s.y += f * x2.y;
    }
    finish(row, 2 * p, s, l);
  }
  cluster_barrier();  // no CTA leaves while another reads its shared memory
}

template <int DT, int CODE, int NT>
static cudaError_t launch_attend(const AttendArgs &a, int64_t tiles, int cluster, cudaStream_t st) {
  auto *fn = k_attend8<DT, CODE, NT>;
  const int smem = (int)sizeof(AtSmem<NT>);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && cluster > 8) e = cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * cluster));
  cfg.blockDim = dim3(kAtThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fn, a);
}

template <int DT, int CODE>
static cudaError_t launch_attend(const AttendArgs &a, int nt, int64_t tiles, int cluster, cudaStream_t st) {
  return nt == 1 ? launch_attend<DT, CODE, 1>(a, tiles, cluster, st) : launch_attend<DT, CODE, 2>(a, tiles, cluster, st);
}

// What the arguments of an attention call have to be, apart from the tensors.
static const char *check_attend(const lkv_cache8 *c, int32_t group, int32_t n, int32_t window, int32_t sinks, int32_t max_len) {
  if (const char *m = check_cache8(c)) return m;
  if (group < 1 || group > 128) return "group must be 1..128";
  if (n < 0 || n > (1 << 24)) return "n must be 0..2^24";
  if (window < 0 || sinks < 0 || max_len < 0) return "window, sinks and max_len must be >= 0";
  return nullptr;
}

}  // namespace lkv

extern "C" lkv_status lkv_cache8_attend_workspace(const lkv_cache8 *c, int32_t group, int32_t n, int32_t window,
                                                  int32_t sinks, int32_t max_len, int64_t *bytes) {
  using namespace lkv;
  if (const char *m = check_attend(c, group, n, window, sinks, max_len)) {
    char buf[160];
    std::snprintf(buf, sizeof buf, "lkv_cache8_attend_workspace: %s", m);
    return refuse(buf);
  }
  if (!bytes) return refuse("lkv_cache8_attend_workspace: null result");
  *bytes = 0;
  return LKV_OK;
}

extern "C" lkv_status lkv_cache8_attend(const lkv_cache8 *c, const void *q, int32_t group, int32_t n,
                                        const int32_t *counts, float scale, int32_t window, int32_t sinks,
                                        int32_t max_len, void *out, void *workspace, int64_t workspace_bytes,
                                        void *stream) {
  using namespace lkv;
  if (const char *m = check_attend(c, group, n, window, sinks, max_len)) {
    char buf[160];
    std::snprintf(buf, sizeof buf, "lkv_cache8_attend: %s", m);
    return refuse(buf);
  }
  if (!(scale - scale == 0.f)) return refuse("lkv_cache8_attend: scale is not finite");
  if (n == 0) return LKV_OK;
  if (!q || !out) return refuse("lkv_cache8_attend: null queries or output");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(counts, 4))
    return refuse("lkv_cache8_attend: queries and output must be 16-byte aligned, counts 4-byte aligned");
  const int64_t S = (int64_t)c->batch * c->n_kv_heads, R = (int64_t)n * group;
  const int64_t bytes = S * R * kHeadDim * (c->dtype == LKV_DTYPE_BF16 ? 2 : 4);
  if (overlaps_cache8(c, out, bytes) || overlap(out, bytes, q, bytes) || overlap(out, bytes, counts, (int64_t)c->batch * 4))
    return refuse("lkv_cache8_attend: the output overlaps the cache or an input");
  (void)workspace;
  (void)workspace_bytes;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_refuse("lkv_cache8_attend", e);
  if (R > 0x7fffffff - 16) return refuse("lkv_cache8_attend: too many rows");
  AttendArgs a{};
  a.c = *c;
  a.q = q;
  a.out = out;
  a.counts = counts;
  a.n = n;
  a.group = group;
  a.window = window >= c->capacity ? 0 : window;  // a window that reaches everything is none
  a.sinks = sinks < c->capacity ? sinks : c->capacity;
  a.scale_log2 = scale * kLog2e;
  const int nt = R <= 8 ? 1 : 2;
  a.row_tiles = (int32_t)((R + 8 * nt - 1) / (8 * nt));
  const int64_t tiles = S * a.row_tiles;
  // blocks that a tile's rows may see, at most
  int64_t most = max_len > 0 && max_len < c->capacity ? max_len : c->capacity;
  if (a.window > 0) {
    const int64_t seen = (int64_t)a.window + a.sinks + (8 * nt + group - 1) / group;
    if (seen < most) most = seen;
  }
  const int64_t blocks = (most + kBlock - 1) / kBlock + 1;
  int cluster = 1;
  while (cluster < kAtMaxCluster && tiles * cluster < (int64_t)sms * 3 && blocks >= (int64_t)2 * cluster * kAtWarps * 4)
    cluster *= 2;
  if (tiles * cluster > 0x7fffffff) return refuse("lkv_cache8_attend: too many rows");
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf = c->dtype == LKV_DTYPE_BF16, i8 = c->code == LKV_CODE_INT8;
  if (bf) e = i8 ? launch_attend<1, LKV_CODE_INT8>(a, nt, tiles, cluster, st) : launch_attend<1, LKV_CODE_E4M3>(a, nt, tiles, cluster, st);
  else e = i8 ? launch_attend<0, LKV_CODE_INT8>(a, nt, tiles, cluster, st) : launch_attend<0, LKV_CODE_E4M3>(a, nt, tiles, cluster, st);
  return e == cudaSuccess ? LKV_OK : cuda_refuse("lkv_cache8_attend", e);
}
