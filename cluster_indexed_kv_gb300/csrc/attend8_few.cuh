// attend8_few.cuh -- attention of few rows over the 8-bit cache: the kernel of
// lkv_cache8_attend's decode steps and of lkv_cache8_attend_shared.
#pragma once

#include <type_traits>

#include "attend8_shared.cuh"

namespace lkv {

constexpr int kAtWarps = 6;
constexpr int kAtThreads = 32 * kAtWarps;
constexpr int kAtMaxCluster = 8;
constexpr int kTailTurns = 4;       // turns that the partial block takes as long as (10,000 clocks, a turn 2500)
constexpr int kCodeBytes = kBlock * kHeadDim;      // one block of K or V
constexpr int kTurnBytes = 2 * 2 * kCodeBytes;     // two blocks of both
constexpr int kRingBytes = kAtWarps * 2 * kTurnBytes;

// c += a * b, fp16 operands, fp32 accumulators
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// c = a * b
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// c += a * b, bf16 operands, fp32 accumulators
__device__ __forceinline__ void mma16816_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x and y (fp32) as three bf16 parts each: 24 bits, whatever their size
__device__ __forceinline__ void split_bf16(float x, float y, uint32_t &p0, uint32_t &p1, uint32_t &p2) {
  p0 = pack_bf16(x, y);
  x -= __uint_as_float(p0 << 16);
  y -= __uint_as_float(p0 & 0xffff0000u);
  p1 = pack_bf16(x, y);
  p2 = pack_bf16(x - __uint_as_float(p1 << 16), y - __uint_as_float(p1 & 0xffff0000u));
}

// A warp's part of a tile's attention (see k_attend8).
template <int DT, int CODE, int NT>
struct Warp {
  static constexpr int RT = 8 * NT;
  static constexpr bool SPLIT = DT == 0;      // fp32: operands with remainders
  static constexpr int QL = SPLIT && NT == 2 ? 2 : 1;
  static constexpr int PW = SPLIT ? 4 : 2;    // words of a lane's four weights: fp32, or fp16 pairs
  uint32_t qa[QL][8][4];      // A fragments of the queries for the 8 steps over d
  float rc[NT];               // row g (+8): query scale * scale * log2(e)
  int pos[NT];                // its position, -1 for none
  float ref[NT], l[NT];
  bool seen[NT];              // the row has a reference (rows that are not there have one from the start)
  float limit;                // a y above it moves a reference
  int unit;                   // V scales count in units of 2^unit
  float o[NT][8][4];
  int lane, g, t;
  int tk, cg;                 // the lane's token of 8 and its V chunk of 8 (see step)
  int koff, voff;
  int window, sinks;
  int open0, open1;           // blocks [open0, open1) are visible to every row as a whole

  // V scales up to 2^(e + 1) are to come: o counts in units of 2^(ref + unit), l
  // in units of 2^ref. Weights carry the scales, so those of all scales known
  // so far shrink as the unit grows: the references go down by as much, which
  // leaves y and o as they are, as far as l (2^100, with room for weights over
  // the smallest scales) allows; o takes the rest. Without that, tokens beside
  // a block of far larger values lost their weights. Rows that are not there
  // keep their reference: their y follows no score.
  __device__ __forceinline__ void raise_unit(int e) {
    if (e <= unit) return;
    const int by = unit == kNoUnit ? 0 : e - unit;
    unit = e;
    if (by == 0) return;
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      float m = l[r];
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
      const int room = 226 - (int)(__float_as_uint(m) >> 23);  // l < 2^(e - 126) of its exponent field e
      const int down = pos[r] < 0 ? 0 : max(0, min(by, room));
      ref[r] -= (float)down;
      l[r] *= pow2f(down);
      const float k = exp2f((float)(down - by));
      const float ka = __shfl_sync(0xffffffffu, k, 8 * t), kb = __shfl_sync(0xffffffffu, k, 8 * t + 4);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        o[r][i][0] *= ka; o[r][i][1] *= kb; o[r][i][2] *= ka; o[r][i][3] *= kb;
      }
    }
  }

  // Scores of NB blocks, masked, turned into weights; the reference moves if
  // needed. ks: the blocks' K scales, lu: log2 of their V scales, iu: 1 / those.
  template <int NB>
  __device__ __forceinline__ void weights(float (&s)[NB][2][4], const float (&ks)[NB], const float (&lu)[NB], const float (&iu)[NB],
                                          const int (&block)[NB], uint32_t (&pw)[NB][NT][PW]) {
    float y[NB][NT][4];
    float far = -INFINITY;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        const float f = rc[r] * ks[n], at = lu[n] - ref[r];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = e >> 1, col = e & 1;
          float v = s[n][j][2 * r + col];
          if (SPLIT && NT == 1) v += s[n][j][2 + col];
          y[n][r][e] = __fmaf_rn(v, f, at);
        }
      }
      if (block[n] < open0 || block[n] >= open1) {  // not every token is visible to every row
#pragma unroll
        for (int r = 0; r < NT; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = block[n] * kBlock + 8 * (e >> 1) + t + 4 * (e & 1);
            if (!(tok <= pos[r] && (window == 0 || tok > pos[r] - window || tok < sinks))) y[n][r][e] = -INFINITY;
          }
      }
#pragma unroll
      for (int r = 0; r < NT; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) far = fmaxf(far, y[n][r][e]);
    }
    if (__any_sync(0xffffffffu, far > limit)) {
      limit = kPShift + kSlack;
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        // the reference is the exponent of weight 1: it goes kPShift below the
        // row's largest y, anywhere the first time and only up from there
        float m = -INFINITY;
#pragma unroll
        for (int n = 0; n < NB; ++n) m = fmaxf(fmaxf(m, fmaxf(y[n][r][0], y[n][r][1])), fmaxf(y[n][r][2], y[n][r][3]));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        float by = m - kPShift;
        if (seen[r] ? by < 0.f : m == -INFINITY) by = 0.f;
        const float k = seen[r] ? exp2f(-by) : 1.f;
        seen[r] |= m > -INFINITY;
        if (!seen[r]) limit = -INFINITY;
        ref[r] += by;
        l[r] *= k;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) y[n][r][e] -= by;
        // accumulator columns are rows 2 t and 2 t + 1
        const float ka = __shfl_sync(0xffffffffu, k, 8 * t), kb = __shfl_sync(0xffffffffu, k, 8 * t + 4);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[r][i][0] *= ka; o[r][i][1] *= kb; o[r][i][2] *= ka; o[r][i][3] *= kb;
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int r = 0; r < NT; ++r) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = ex2(y[n][r][e]);
        l[r] = __fmaf_rn((p[0] + p[1]) + (p[2] + p[3]), iu[n], l[r]);
#pragma unroll
        for (int e = 0; e < PW; ++e)
          pw[n][r][e] = SPLIT ? __float_as_uint(p[e]) : h2_bits(__floats2half2_rn(p[2 * (e & 1)], p[2 * (e & 1) + 1]));
      }
  }

  // NB quantised blocks from the ring (K then V of each, as the copies lay
  // them down: the 16-byte chunk j of row r at j ^ (r & 7)). The lane's K are
  // tokens (g / 2) + 4 (g & 1) and that + 8, d 16 t.. and 64 + 16 t..; its V
  // tokens t, t + 4, t + 8, t + 12, d 16 cg..: of every 8 lanes that a
  // 16-byte load serves together, no two meet in a bank. NB blocks together
  // give their chains of products and their softmax to one another to hide
  // behind.
  template <int NB>
  __device__ __forceinline__ void step(const unsigned char *ring, const float (&ks)[NB], const float (&lu)[NB], const float (&iu)[NB],
                                       const int (&block)[NB]) {
    float s[NB][2][4];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int n = 0; n < NB; ++n) {
        const uint4 k0 = *(const uint4 *)(ring + n * 2 * kCodeBytes + (koff ^ (64 * c)));
        const uint4 k1 = *(const uint4 *)(ring + n * 2 * kCodeBytes + 1024 + (koff ^ (64 * c)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 &k = j ? k1 : k0;
            uint32_t b0, b1;
            codes_row<CODE>(e == 0 ? k.x : e == 1 ? k.y : e == 2 ? k.z : k.w, b0, b1);
            if (c == 0 && e == 0) mma16816_first(s[n][j], qa[0][0], b0, b1);
            else mma16816(s[n][j], qa[0][4 * c + e], b0, b1);
            if (QL == 2) mma16816(s[n][j], qa[QL - 1][4 * c + e], b0, b1);
          }
        }
      }
    }
    uint32_t pw[NB][NT][PW];
    weights<NB>(s, ks, lu, iu, block, pw);
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      Weights wn(pw[n]);
      uint4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        v[j] = *(const uint4 *)(ring + (2 * n + 1) * kCodeBytes + (j >> 1) * 1024 + (j & 1) * 512 + (voff ^ (64 * (j & 1))));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = e == 0 ? v[j].x : e == 1 ? v[j].y : e == 2 ? v[j].z : v[j].w;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t a[4];
          codes_across<CODE, SPLIT>(w[0], w[1], h, a[0], a[1]);
          codes_across<CODE, SPLIT>(w[2], w[3], h, a[2], a[3]);
          accumulate(a, wn, 2 * e + h, SPLIT ? 3 : 1);
        }
      }
    }
  }

  // The weights of a block as operands of P V: fp16 for bf16 caches (off by 2^-11
  // of themselves, or 2^-25 where they are small), in one product; three bf16
  // parts for fp32 ones, which keep 24 bits of weights of any size.
  struct Weights {
    uint32_t b[SPLIT ? 3 : 1][NT][2];
    __device__ __forceinline__ explicit Weights(const uint32_t (&w)[NT][PW]) {
#pragma unroll
      for (int r = 0; r < NT; ++r) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          if constexpr (SPLIT)
            split_bf16(__uint_as_float(w[r][2 * e]), __uint_as_float(w[r][2 * e + 1]), b[0][r][e], b[1][r][e], b[2][r][e]);
          else
            b[0][r][e] = w[r][e];
        }
      }
    }
  };

  // o += values * weights, with the first `parts` parts of the weights
  __device__ __forceinline__ void accumulate(const uint32_t (&a)[4], const Weights &w, int i, int parts) {
#pragma unroll
    for (int r = 0; r < NT; ++r) {
#pragma unroll
      for (int z = 0; z < parts; ++z) {
        if constexpr (SPLIT) mma16816_bf16(o[r][i], a, w.b[z][r][0], w.b[z][r][1]);
        else mma16816(o[r][i], a, w.b[z][r][0], w.b[z][r][1]);
      }
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

  static __device__ __forceinline__ int below(uint32_t bits) { return min(max((int)(bits >> 23) - 126, -100), 126); }

  // The last, partial block, from the tails: the same products, scores on fp16
  // values and (fp32 tails) their remainders, in units of the largest one; P V
  // on fp16 values in such units, or (fp32) on three bf16 parts of them.
  __device__ __noinline__ void tail_step(const void *kt, const void *vt, int rows, int block) {
    // powers of two that bring the tails' largest magnitudes below 1; what is
    // read again below comes from L1
    float mk = 0.f, mv = 0.f;
#pragma unroll
    for (int row = 0; row < kBlock; ++row) {
      const float4 x = tail4(kt, row, 4 * lane, rows), y = tail4(vt, row, 4 * lane, rows);
      mk = fmaxf(mk, fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w))));
      mv = fmaxf(mv, fmaxf(fmaxf(fabsf(y.x), fabsf(y.y)), fmaxf(fabsf(y.z), fabsf(y.w))));
    }
    const int ke = below(__reduce_max_sync(0xffffffffu, __float_as_uint(mk)));
    const int ve = max(below(__reduce_max_sync(0xffffffffu, __float_as_uint(mv))), unit - kUnitSpan);
    raise_unit(ve);
    const float kf = pow2f(-ke), vf = pow2f(-ve);
    float s[1][2][4] = {};
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float4 x = tail4(kt, 8 * j + tk, 64 * c + 16 * t + 4 * e, rows);
          uint32_t h0, h1, l0, l1;
          split_h2(x.x * kf, x.y * kf, h0, l0);
          split_h2(x.z * kf, x.w * kf, h1, l1);
#pragma unroll
          for (int z = 0; z < QL; ++z) {
            mma16816(s[0][j], qa[z][4 * c + e], h0, h1);
            if (SPLIT) mma16816(s[0][j], qa[z][4 * c + e], l0, l1);
          }
        }
      }
    }
    uint32_t pw[1][NT][PW];
    const float ks[1] = {pow2f(ke)}, lu[1] = {(float)(ve - unit)}, iu[1] = {pow2f(unit - ve)};
    const int at[1] = {block};
    weights<1>(s, ks, lu, iu, at, pw);
    const Weights w0(pw[0]);
    const int tok[4] = {t, t + 4, t + 8, t + 12};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float4 x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = tail4(vt, tok[j], 16 * cg + 4 * e, rows);
        x[j].x *= vf; x[j].y *= vf; x[j].z *= vf; x[j].w *= vf;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t a[3][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // d (+ 1) of tokens t and t + 4, then of t + 8 and t + 12
          const float4 &y0 = x[j & 2], &y1 = x[(j & 2) + 1];
          const float f0 = h ? (j & 1 ? y0.w : y0.z) : (j & 1 ? y0.y : y0.x), f1 = h ? (j & 1 ? y1.w : y1.z) : (j & 1 ? y1.y : y1.x);
          if constexpr (SPLIT) split_bf16(f0, f1, a[0][j], a[1][j], a[2][j]);
          else a[0][j] = h2_bits(__floats2half2_rn(f0, f1));
        }
        accumulate(a[0], w0, 2 * e + h, SPLIT ? 3 : 1);
        if constexpr (SPLIT) {  // parts together below 2^-24 of a product are left out
          accumulate(a[1], w0, 2 * e + h, 2);
          accumulate(a[2], w0, 2 * e + h, 1);
        }
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

template <int NT>
struct AtSmem {
  static constexpr int RT = 8 * NT;
  static constexpr int RS = 20;               // floats between rows (bank spread)
  static constexpr int IS = RT * RS + 8;      // floats between the 8 d-pair planes
  static constexpr int kSlot = RT * kHeadDim + 3 * RT;  // floats of a partial in the workspace
  float o[kAtWarps][8 * IS];
  float part[RT][kHeadDim];                   // the CTA's merged partial
  float m[kAtWarps][RT], t[kAtWarps][RT];     // exponents of the units of o and of l
  float l[kAtWarps][RT], f[kAtWarps][RT];
  float pm[RT], pt[RT], pl[RT];
};

// Values d, d + 1 of a row of the output: o / l * 2^e.
template <int DT>
__device__ __forceinline__ void put_out(const AttendArgs &a, int64_t slice, int cnt, int rr, int d, float2 o, float l, float e) {
  const int i = rr / a.group;
  if (rr >= a.n * a.group) return;
  if (i >= cnt || l == 0.f) {
    o = make_float2(0.f, 0.f);
  } else {
    const float unit = exp2f(e);
    o.x = o.x / l * unit;
    o.y = o.y / l * unit;
  }
  const int64_t at = ((slice * a.group + rr % a.group) * a.n + i) * kHeadDim + d;
  if (DT == 1) *(uint32_t *)((uint16_t *)a.out + at) = pack_bf16(o.x, o.y);
  else *(float2 *)((float *)a.out + at) = o;
}

// What k_attend8 is part of: lkv_cache8_attend (kAlone), or attention behind
// shared prefixes: the prefixes' part (kPrefix, always streamed, its results
// parts for the join) or the sequences' own tokens (kOwn, in clusters, joined
// with their prefix's parts).
enum { kAlone = 0, kPrefix = 1, kOwn = 2 };
template <int MODE>
using ArgsOf = std::conditional_t<MODE == kAlone, AttendArgs, SharedArgs>;
template <int MODE>
__device__ __forceinline__ const lkv_cache8 &keys_of(const ArgsOf<MODE> &a) {
  if constexpr (MODE == kPrefix) return a.p;
  else return a.c;
}

// What the prefix adds to a sequence's rows.
template <int RT>
struct PrefixSum {
  float o[RT][kHeadDim];             // in units of 2^m
  float m[RT], t[RT], l[RT];         // l in units of 2^t
};

// Row `row` of the sequence's (slice: sequence and KV head): the sum of its
// prefix's parts, by a warp, into r of z: a lane takes four values of d, and
// a part's exponents and total. As many parts are on their way together as
// registers hold: in fours, a step of 32 samples of 32K tokens took 1.8 us longer.
constexpr int kSumAtOnce = 16;
template <int RT>
__device__ __forceinline__ void sum_prefix(const SharedArgs &a, int64_t slice, int row, PrefixSum<RT> &z, int r, int lane) {
  const int b = (int)((uint32_t)slice / (uint32_t)a.c.n_kv_heads), h = (int)((uint32_t)slice % (uint32_t)a.c.n_kv_heads);
  const int per = a.n * a.group, rows = a.part_rows;
  const int4 sq = row < per ? a.seq[b] : make_int4(-1, 0, 0, 0);
  float top = -INFINITY, topt = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (sq.x >= 0) {
    const int64_t pr = (int64_t)sq.y * per + row, rt = quotient(pr, rows);
    const int tile = sq.x + (int)rt * a.c.n_kv_heads + h, rr = (int)(pr - rt * rows);
    const int2 who = a.tile[tile];
    const float *const part = a.parts + ((int64_t)who.x + tile) * part_floats(rows);
    auto at = [&](int j) { return part + (int64_t)j * part_floats(rows); };
    for (int j0 = 0; j0 < who.y; j0 += 32) {  // 32 parts: a lane's own one's exponents, and values of kSumAtOnce at a time
      const int some = min(32, who.y - j0);
      float4 x[kSumAtOnce];
      auto load = [&](int k0) {
#pragma unroll
        for (int k = 0; k < kSumAtOnce; ++k) {
          x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k0 + k < some) x[k] = *(const float4 *)(at(j0 + k0 + k) + part_place(rr, 4 * lane));
        }
      };
      load(0);
      float m = -INFINITY, t = -INFINITY, mine = 0.f;
      if (lane < some) {
        const float *p = at(j0 + lane) + rows * kHeadDim + rr;
        m = p[0];
        t = p[rows];
        mine = p[2 * rows];
      }
      float above = fmaxf(top, m), abovet = fmaxf(topt, t);
#pragma unroll
      for (int d = 16; d; d /= 2) {
        above = fmaxf(above, __shfl_xor_sync(0xffffffffu, above, d));
        abovet = fmaxf(abovet, __shfl_xor_sync(0xffffffffu, abovet, d));
      }
      const float k = share(top, above), f = share(m, above);
      o.x = k == 0.f ? 0.f : k * o.x;
      o.y = k == 0.f ? 0.f : k * o.y;
      o.z = k == 0.f ? 0.f : k * o.z;
      o.w = k == 0.f ? 0.f : k * o.w;
      l = share(topt, abovet) * l + share(t, abovet) * mine;
      top = above;
      topt = abovet;
#pragma unroll 1
      for (int k0 = 0; k0 < some; k0 += kSumAtOnce) {
        if (k0) load(k0);
#pragma unroll
        for (int k = 0; k < kSumAtOnce; ++k) {
          const float g = __shfl_sync(0xffffffffu, f, (k0 + k) & 31);
          if (k0 + k < some && g != 0.f) {  // a part that saw nothing holds anything
            o.x += g * x[k].x;
            o.y += g * x[k].y;
            o.z += g * x[k].z;
            o.w += g * x[k].w;
          }
        }
      }
    }
#pragma unroll
    for (int d = 16; d; d /= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
  }
  *(float4 *)&z.o[r][4 * lane] = o;
  if (lane == 0) {
    z.m[r] = top;
    z.t[r] = topt;
    z.l[r] = l;
  }
}

// A row's own result (o in units of 2^m, l of 2^t) and its prefix's, values d and d + 1.
template <int RT>
__device__ __forceinline__ void add_prefix(const PrefixSum<RT> &z, int r, int d, float2 &o, float &l, float &m, float &t) {
  const float top = fmaxf(m, z.m[r]), topt = fmaxf(t, z.t[r]), f = share(m, top), g = share(z.m[r], top);
  o.x = (f == 0.f ? 0.f : f * o.x) + (g == 0.f ? 0.f : g * z.o[r][d]);
  o.y = (f == 0.f ? 0.f : f * o.y) + (g == 0.f ? 0.f : g * z.o[r][d + 1]);
  l = share(t, topt) * l + share(z.t[r], topt) * z.l[r];
  m = top;
  t = topt;
}

// The attention of RT = 8 NT rows (a row is one query head of one token; the
// rows of a KV head are ordered token-major) over the visible blocks of one
// (sequence, KV head): a tile.
//
// A warp takes two blocks of 16 tokens a turn, which one of its lanes has
// copied into its own ring by TMA a turn ahead. Scores are mma.sync m16n8k16
// products with the rows as M (fp16; rows 8..15 hold the remainders of fp32
// queries, or a second 8 rows) and 8 tokens as N; the contraction's order
// over d is free, so a lane's K operands are 16-byte runs of a token's row.
// P V takes 16 values of d as M, the 16 tokens as K and 8 rows as N: the
// score accumulators are its B operand as they stand, and a lane's V operands
// are again 16-byte runs of four tokens. 8-bit codes are exact in fp16. The
// queries are scaled by a power of two into fp16's range, and scores get the
// block's K scale in fp32.
//
// Softmax in base 2. The weights carry the block's V scale u as well: with
// y = score + log2(u), w = 2^(y - reference), out = sum w code / sum w / u, so
// P V accumulates in the tensor cores' registers as it is. Scales count in
// units of the largest one that the warp has met (u <= 2), whatever the
// values' magnitude. The reference of a row only moves when a y passes it by
// 2^8: the weights lie below 2^(8 + kPShift), fp16's range, and small ones
// are off by 2^-25, 2^-31 of the largest one or less: tokens that weigh less than
// 2^-22 of it count with fewer bits than bf16 has.
// For fp32 caches they are three bf16 parts (three products a block in place of
// two on fp16 and a remainder, which lost weights below 2^-25 altogether).
//
// Small calls: a tile's blocks are shared by the CTAs of one cluster. Each CTA
// merges its warps in shared memory, then every CTA of the cluster merges a
// part of the outputs over distributed shared memory: one launch, no
// workspace. Streamed: the blocks of all tiles in a row are shared evenly by
// as many CTAs as the GPU holds, whatever the sequences' lengths; a tile that
// several CTAs share goes to the workspace in parts, and k_attend8_merge joins
// them. No atomics in either: the same result each time.
//
// Bound by the codes' bytes. On a GB300, 4 query heads, bf16: 64 slices of 33,000 tokens 89 us, 89%
// of the measured copy rate; 8 of 131,579 tokens 53 us, 75% (the merge is a
// second kernel behind the first); 256 slices of a window of 1024 tokens 19.5 us,
// 51% (one warp's partial block, and launch, lengths, queries and merges in
// turn, as for one slice of 2048 tokens: 9 us). fp32 caches are bound by their
// products: 64 slices of 33,000 tokens 116 us, 8 of 131,579 tokens 66 us, one
// of 2048 tokens 9.6 us.
//
// Behind prefixes: 4 samples of a 2048-token prompt (8 KV heads, 16 rows of each)
// 17 us, 6 samples of 8191 tokens in fp32 34 us (a tile of 16 rows a CTA: 4 turns,
// the partial block as long as 4 more). The own tokens need nothing of the kernel
// before this one but its word for what came before both, and its parts are read
// last: 21 and 44 us with its end awaited first (the word costs 0.7 us).
template <int DT, int CODE, int NT, int MODE>
__global__ void __launch_bounds__(kAtThreads, NT == 1 || DT == 1 ? 2 : 1)
    k_attend8(const __grid_constant__ ArgsOf<MODE> a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full_bar[kAtWarps][2];
  __shared__ std::conditional_t<MODE == kAlone, Stream, int> stream;
  constexpr int RT = 8 * NT;
  using W = Warp<DT, CODE, NT>;
  using Sm = AtSmem<NT>;
  const lkv_cache8 &c = keys_of<MODE>(a);
  unsigned char *const area = raw + ((1024u - (smem_at(raw) & 1023u)) & 1023u);
  Sm &sm = *(Sm *)area;
  const int wid = threadIdx.x >> 5;
  unsigned char *const ring = area + wid * 2 * kTurnBytes;
  uint64_t *const bar = full_bar[wid];
  const bool streamed = MODE == kAlone ? a.streamed : MODE == kPrefix;
  const int parts = streamed ? 1 : (int)cluster_size(), part = streamed ? 0 : (int)cluster_rank();
  const int G = MODE == kPrefix ? c.batch : c.batch * a.row_tiles;
  // the prefixes' tables lie behind what the rings and merges use
  [[maybe_unused]] __shared__ __align__(16) std::conditional_t<MODE == kOwn, PrefixSum<RT>, int> prefix;
  [[maybe_unused]] __shared__ uint64_t vouched_s[kAtWarps];  // what each warp's reads go by (see vouch)
  constexpr int kUsed = (int)sizeof(Sm) > kRingBytes ? (int)sizeof(Sm) : kRingBytes;
  static_assert(kUsed % 8 == 0, "the tables begin with 8-byte words");
  [[maybe_unused]] auto pre = [&] {
    if constexpr (MODE == kPrefix) return Prefixes<false>(a, area + kUsed);
    else return 0;
  }();

  W w;
  w.lane = threadIdx.x & 31;
  w.g = w.lane >> 2;
  w.t = w.lane & 3;
  w.tk = (w.g >> 1) | ((w.g & 1) << 2);
  w.cg = w.tk;
  w.koff = w.tk * kHeadDim + ((w.t ^ w.tk) << 4);
  w.voff = w.t * kHeadDim + ((w.t ^ w.cg) << 4);
  w.window = a.window;
  w.sinks = a.sinks;
  if (w.lane == 0) {
    bar_init(&bar[0], 1);
    bar_init(&bar[1], 1);
    bar_init_fence();
    if (wid == 0) {
      tma_prefetch(&kmap);
      tma_prefetch(&vmap);
    }
  }
  // Own tokens behind prefixes: the kernel before this one has waited for all
  // before it and vouches for that; what it writes is read, and waited for, last.
  if constexpr (MODE == kOwn) {
    if (w.lane == 0) vouched_s[wid] = vouched(a);
  } else {
    wait_prerequisites();
  }
  __syncwarp();
  if constexpr (MODE == kPrefix) launch_vouched(a);
  else if (streamed) launch_dependents();
  uint32_t phase = 0;      // parities of the two barriers
  bool dead = false;       // a copy did not arrive in time: the warp takes no more
  const int64_t es = DT == 1 ? 2 : 4;

  int64_t x0 = 0, x1 = 1;  // streamed: the CTA's share of the row of blocks
  if constexpr (MODE == kAlone) {
    if (streamed) {
      stream.fill(a, RT, 1, 0);
      stream.share(G, x0, x1);
    }
  } else if constexpr (MODE == kPrefix) {
    pre.fill(a);
    pre.share(a, x0, x1);
  }
  for (int64_t x = x0; x < x1;) {
    Tile tile;
    int64_t slice;
    int rt, b0, b1;
    [[maybe_unused]] Prefixes<false>::Piece piece{};
    if constexpr (MODE == kPrefix) {
      piece = pre.piece(a, x, x1);
      if (threadIdx.x == 0 && piece.u0 == 0) pre.announce(a, piece, x);
      rt = piece.rt;
      slice = (int64_t)piece.list * c.n_kv_heads + piece.h;
      tile.len = pre.len(piece.list);
      tile.lo = tile.sb = tile.cnt = 0;
      tile.hi = (tile.len - 1) / kBlock;
      tile.nb = tile.hi + 1;
      tile.pmin = tile.pmax = tile.len - 1;
      b0 = max(piece.u0 - pre.start, 0);
      b1 = max(piece.u1 - pre.start, 0);
      x += piece.u1 - piece.u0;
    } else if (MODE == kAlone && streamed) {
      if constexpr (MODE == kAlone) {
      const int gi = stream.group(x, G), nb = stream.nu[gi];
      const int64_t off = x - stream.at[gi];
      const int h = (int)(off / nb), b = gi % c.batch;
      rt = gi / c.batch;
      slice = (int64_t)b * c.n_kv_heads + h;
      tile = Tile(a, b, rt, RT);
      b0 = (int)(off % nb);
      b1 = (int)min((int64_t)nb, b0 + (x1 - x));
      x += b1 - b0;
      }
    } else {
      const uint32_t id = blockIdx.x / (uint32_t)parts, S = (uint32_t)c.batch * c.n_kv_heads;  // the grid is below 2^31
      slice = id % S;
      rt = a.row_tiles - 1 - (int)(id / S);  // the rows with most to see come first
      tile = Tile(a, (int)((id % S) / c.n_kv_heads), rt, RT);
      b0 = (int)((uint32_t)tile.nb * part / parts);  // at most 8 x 2^26
      b1 = (int)((uint32_t)tile.nb * (part + 1) / parts);
      x = x1;
    }
    const int r0 = rt * RT, full = tile.len / kBlock;  // blocks before `full` are quantised
    const bool tail = tile.nb > 0 && tile.hi >= full && b1 == tile.nb && b1 > b0;  // the share ends in the partial one
    const int b2 = dead ? b0 : tail ? b1 - 1 : b1;

    // The warp's turn i: units unit_at(i) and the next. The turns go round the
    // warps, kTailTurns rounds without the last warp, which takes the partial
    // block.
    const int late = tail ? kTailTurns : 0;
    auto unit_at = [&](int i) { return b0 + 2 * (i * kAtWarps + wid + (wid == kAtWarps - 1 ? late * (kAtWarps - 1) : -min(i, late))); };
    auto issue = [&](int i) {
      const int u = unit_at(i);
      if (u < b2 && w.lane == 0) {
        unsigned char *to = ring + (i & 1) * kTurnBytes;
        uint64_t *on = &bar[i & 1];
        const bool two = u + 1 < b2;
        bar_expect(on, two ? kTurnBytes : kTurnBytes / 2);
        const int k0 = tile.block(u) * kBlock;
        tma_3d(to, &kmap, 0, k0, (int)slice, on);
        tma_3d(to + kCodeBytes, &vmap, 0, k0, (int)slice, on);
        if (two) {
          const int k1 = tile.block(u + 1) * kBlock;
          tma_3d(to + 2 * kCodeBytes, &kmap, 0, k1, (int)slice, on);
          tma_3d(to + 3 * kCodeBytes, &vmap, 0, k1, (int)slice, on);
        }
      }
    };
    issue(0);
    issue(1);
    const char *const kt = (const char *)c.k_tail + slice * kBlock * kHeadDim * es, *const vt = (const char *)c.v_tail + slice * kBlock * kHeadDim * es;
    if (tail && wid == kAtWarps - 1)
      for (int64_t at = 128 * w.lane; at < kBlock * kHeadDim * es; at += 32 * 128) {
        asm volatile("prefetch.global.L2 [%0];" ::"l"(kt + at));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(vt + at));
      }

    const float *ksc = c.k_scale + slice * (c.capacity / kBlock), *vsc = c.v_scale + slice * (c.capacity / kBlock);
    // the scales of the warp's turns, 16 turns ahead
    float ks_next = 0.f, vs_next = 0.f;
    auto scales = [&](int i) {
      const int mine = unit_at(i + (w.lane >> 1)) + (w.lane & 1);
      vs_next = 0.f;
      if (mine < b2) {
        ks_next = ksc[tile.block(mine)];
        vs_next = vsc[tile.block(mine)];
      }
    };
    scales(0);
    w.open0 = a.window > 0 ? max(0, tile.pmax - a.window + kBlock) / kBlock : 0;
    w.open1 = (tile.pmin + 1) / kBlock;
    [[maybe_unused]] int pmin = tile.pmin;
    w.limit = -INFINITY;
    w.unit = kNoUnit;
    // queries: row g (and g + 8), the 32 values of d that go with the lane's K runs
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      w.ref[r] = 0.f;
      w.l[r] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) w.o[r][i][e] = 0.f;
      const int row = r0 + 8 * r + w.g;
      const int i = row / a.group;
      bool valid = row < a.n * a.group && i < tile.cnt;
      w.pos[r] = valid ? tile.len - tile.cnt + i : -1;
      int64_t q_row = (slice * a.group + (valid ? row % a.group : 0)) * a.n + (valid ? i : 0);
      if constexpr (MODE == kPrefix) {
        const ListRow pr = list_row(a, pre, piece.list, piece.h, tile.len, (int64_t)rt * RT + 8 * r + w.g);
        valid = pr.at >= 0;
        w.pos[r] = pr.pos;
        q_row = max(pr.at, (int64_t)0);
        if (valid) pmin = min(pmin, pr.pos);
      }
      w.seen[r] = !valid;
      float x[32];
      const char *p = (const char *)a.q + q_row * kHeadDim * es;
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

    if constexpr (MODE == kPrefix) w.open1 = (__reduce_min_sync(0xffffffffu, pmin) + 1) / kBlock;

    float ks = 0.f, vs = 1.f, lu = 0.f;
    int i = 0;
    for (int u = unit_at(0); u < b2; u = unit_at(++i)) {
      if ((i & 15) == 0) {
        ks = ks_next;
        vs = vs_next;
        scales(i + 16);
        const float top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(vs)));
        if (top > 0.f) w.raise_unit(min(max((int)(__float_as_uint(top) >> 23) - 127, -126), 126));
        vs = fmaxf(vs * pow2f(-w.unit), pow2f(-kUnitSpan));  // a scale of 0 too: its codes stand for zeros, whatever they are
        lu = log2f(vs);
        vs = 1.f / vs;
      }
      if (!__all_sync(0xffffffffu, bar_wait(&bar[i & 1], (phase >> (i & 1)) & 1))) {
        dead = true;
        break;
      }
      phase ^= 1u << (i & 1);
      const int s0 = (2 * i) & 31, s1 = s0 + 1;
      const float k0 = __shfl_sync(0xffffffffu, ks, s0), k1 = __shfl_sync(0xffffffffu, ks, s1);
      const float l0 = __shfl_sync(0xffffffffu, lu, s0), l1 = __shfl_sync(0xffffffffu, lu, s1);
      const float i0 = __shfl_sync(0xffffffffu, vs, s0), i1 = __shfl_sync(0xffffffffu, vs, s1);
      const unsigned char *turn = ring + (i & 1) * kTurnBytes;
      if (u + 1 < b2) {
        const float kk[2] = {k0, k1}, ll[2] = {l0, l1}, ii[2] = {i0, i1};
        const int bb[2] = {tile.block(u), tile.block(u + 1)};
        w.template step<2>(turn, kk, ll, ii, bb);
      } else {
        const float kk[1] = {k0}, ll[1] = {l0}, ii[1] = {i0};
        const int bb[1] = {tile.block(u)};
        w.template step<1>(turn, kk, ll, ii, bb);
      }
      __syncwarp();
      issue(i + 2);
    }
    if (dead && b2 > b0) {
      if (w.lane == 0) atomicOr(a.c.ticket + a.c.batch, kAnomTimeout);
      // copies still in flight land before the ring is used again
      for (int j = 0; j < 2; ++j)
        if (unit_at(i + j) < b2) bar_wait(&bar[(i + j) & 1], (phase >> ((i + j) & 1)) & 1);
    }
    if (tail && wid == kAtWarps - 1) {
      W z = w;  // a copy: w itself stays in registers
      z.tail_step(kt, vt, tile.len - full * kBlock, full);
      w = z;
    }

    __syncthreads();  // the rings are free: the warps' partials go over them
#pragma unroll
    for (int r = 0; r < NT; ++r) {
      float l = w.l[r];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      if (w.t == 0) {
        sm.m[wid][8 * r + w.g] = w.seen[r] && w.unit != kNoUnit ? w.ref[r] + (float)w.unit : -INFINITY;
        sm.t[wid][8 * r + w.g] = w.seen[r] ? w.ref[r] : -INFINITY;
        sm.l[wid][8 * r + w.g] = l;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          *(float2 *)&sm.o[wid][i * Sm::IS + (8 * r + 2 * w.t + e) * Sm::RS + 2 * w.cg] = make_float2(w.o[r][i][e], w.o[r][i][2 + e]);
    }
    if constexpr (MODE == kOwn) {  // a CTA of a cluster takes the rows that it will write
      wait_prerequisites();
      const uint64_t now = vouched_now(a);
      for (int row = part + parts * wid; row < RT; row += parts * kAtWarps) sum_prefix(a, slice, r0 + row, prefix, row, w.lane);
      if (__syncthreads_or(vouched_s[wid] != now)) {  // copies go over what was just written here
        if (w.lane == 0) vouched_s[wid] = now;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
        x = x0;
        continue;
      }
    } else {
      __syncthreads();
    }
    if (threadIdx.x < RT) {
      const int row = threadIdx.x;
      float top = -INFINITY, topt = -INFINITY, l = 0.f;
#pragma unroll
      for (int j = 0; j < kAtWarps; ++j) {
        top = fmaxf(top, sm.m[j][row]);
        topt = fmaxf(topt, sm.t[j][row]);
      }
#pragma unroll
      for (int j = 0; j < kAtWarps; ++j) {
        sm.f[j][row] = share(sm.m[j][row], top);
        l += share(sm.t[j][row], topt) * sm.l[j][row];
      }
      sm.pm[row] = top;
      sm.pt[row] = topt;
      sm.pl[row] = l;
    }
    __syncthreads();
    const bool whole = MODE == kPrefix ? false : streamed ? b0 == 0 && b1 == tile.nb : parts == 1;
    float *slot = nullptr;
    if constexpr (MODE == kPrefix) slot = a.parts + ((int64_t)blockIdx.x + piece.tile) * part_floats(RT);
    else if (streamed && !whole) slot = a.ws + (2 * (int64_t)blockIdx.x + (x - (b1 - b0) == x0 ? 0 : 1)) * Sm::kSlot;
    for (int it = threadIdx.x; it < RT * 64; it += kAtThreads) {
      const int row = it >> 6, p = it & 63;  // values 2 p, 2 p + 1: plane p % 8 of chunk p / 8
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kAtWarps; ++j) {
        const float2 x2 = *(const float2 *)&sm.o[j][(p & 7) * Sm::IS + row * Sm::RS + 2 * (p >> 3)];
        const float f = sm.f[j][row];
        s.x += f * x2.x;
        s.y += f * x2.y;
      }
      if constexpr (MODE == kPrefix) {
        *(float2 *)(slot + part_place(row, 2 * p) + 2 * (p & 1)) = s;
      } else if (whole) {
        float m = sm.pm[row], t = sm.pt[row], l = sm.pl[row];
        if constexpr (MODE == kOwn) add_prefix(prefix, row, 2 * p, s, l, m, t);
        put_out<DT>(a, slice, tile.cnt, r0 + row, 2 * p, s, l, m - t);
      } else {
        *(float2 *)(slot ? slot + row * kHeadDim + 2 * p : &sm.part[row][2 * p]) = s;
      }
    }
    if (slot && threadIdx.x < RT) {
      slot[RT * kHeadDim + threadIdx.x] = sm.pm[threadIdx.x];
      slot[RT * kHeadDim + RT + threadIdx.x] = sm.pt[threadIdx.x];
      slot[RT * kHeadDim + 2 * RT + threadIdx.x] = sm.pl[threadIdx.x];
    }
    if (streamed) {
      if (x < x1) {  // the next tile's copies go over what was just read and written here
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
      }
      continue;
    }
    if (whole) return;
    cluster_barrier();
    const int step = MODE == kOwn ? kAtThreads : parts * kAtThreads;
    for (int it = threadIdx.x + (MODE == kOwn ? 0 : part * kAtThreads);; it += step) {
      const int row = MODE == kOwn ? (it >> 6) * parts + part : it >> 6, p = it & 63;
      if (row >= RT) break;
      float m[kAtMaxCluster], mt[kAtMaxCluster], top = -INFINITY, topt = -INFINITY, l = 0.f;
#pragma unroll
      for (int j = 0; j < kAtMaxCluster; ++j) {
        if (j >= parts) break;
        m[j] = peer_f(&sm.pm[row], j);
        mt[j] = peer_f(&sm.pt[row], j);
        top = fmaxf(top, m[j]);
        topt = fmaxf(topt, mt[j]);
      }
      float2 s = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kAtMaxCluster; ++j) {
        if (j >= parts) break;
        const float f = share(m[j], top);
        const float2 x2 = peer_f2(&sm.part[row][2 * p], j);
        l += share(mt[j], topt) * peer_f(&sm.pl[row], j);
        s.x += f * x2.x;
        s.y += f * x2.y;
      }
      if constexpr (MODE == kOwn) add_prefix(prefix, row, 2 * p, s, l, top, topt);
      put_out<DT>(a, slice, tile.cnt, r0 + row, 2 * p, s, l, top - topt);
    }
    cluster_barrier();  // no CTA leaves while another reads its shared memory
  }
  if constexpr (MODE == kPrefix) {
    if (a.late && blockIdx.x == 0 && threadIdx.x == 0) vouch(a);
  }
}

}  // namespace lkv
