// attend8.cu -- causal attention over the 8-bit cache (lkv_cache8_attend).
#include "attend8.cuh"

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
template <int DT, int CODE, int NT>
__global__ void __launch_bounds__(kAtThreads, NT == 1 || DT == 1 ? 2 : 1)
    k_attend8(const __grid_constant__ AttendArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) uint64_t full_bar[kAtWarps][2];
  __shared__ Stream stream;
  constexpr int RT = 8 * NT;
  using W = Warp<DT, CODE, NT>;
  using Sm = AtSmem<NT>;
  const lkv_cache8 &c = a.c;
  unsigned char *const area = raw + ((1024u - (smem_at(raw) & 1023u)) & 1023u);
  Sm &sm = *(Sm *)area;
  const int wid = threadIdx.x >> 5;
  unsigned char *const ring = area + wid * 2 * kTurnBytes;
  uint64_t *const bar = full_bar[wid];
  const int parts = a.streamed ? 1 : (int)cluster_size(), part = a.streamed ? 0 : (int)cluster_rank();
  const int G = c.batch * a.row_tiles;

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
  __syncwarp();
  wait_prerequisites();
  if (a.streamed) launch_dependents();
  uint32_t phase = 0;      // parities of the two barriers
  bool dead = false;       // a copy did not arrive in time: the warp takes no more
  const int64_t es = DT == 1 ? 2 : 4;

  int64_t x0 = 0, x1 = 1;  // streamed: the CTA's share of the row of blocks
  if (a.streamed) {
    stream.fill(a, RT, 1, 0);
    stream.share(G, x0, x1);
  }
  for (int64_t x = x0; x < x1;) {
    Tile tile;
    int64_t slice;
    int rt, b0, b1;
    if (a.streamed) {
      const int gi = stream.group(x, G), nb = stream.nu[gi];
      const int64_t off = x - stream.at[gi];
      const int h = (int)(off / nb), b = gi % c.batch;
      rt = gi / c.batch;
      slice = (int64_t)b * c.n_kv_heads + h;
      tile = Tile(a, b, rt, RT);
      b0 = (int)(off % nb);
      b1 = (int)min((int64_t)nb, b0 + (x1 - x));
      x += b1 - b0;
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
      const bool valid = row < a.n * a.group && i < tile.cnt;
      w.pos[r] = valid ? tile.len - tile.cnt + i : -1;
      w.seen[r] = !valid;
      float x[32];
      const char *p = (const char *)a.q + ((slice * a.group + (valid ? row % a.group : 0)) * a.n + (valid ? i : 0)) * kHeadDim * es;
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
      if (w.lane == 0) atomicOr(c.ticket + c.batch, kAnomTimeout);
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
    __syncthreads();
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
    const bool whole = a.streamed ? b0 == 0 && b1 == tile.nb : parts == 1;
    float *const slot = a.streamed && !whole ? a.ws + (2 * (int64_t)blockIdx.x + (x - (b1 - b0) == x0 ? 0 : 1)) * Sm::kSlot : nullptr;
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
      if (whole) put_out<DT>(a, slice, tile.cnt, r0 + row, 2 * p, s, sm.pl[row], sm.pm[row] - sm.pt[row]);
      else *(float2 *)(slot ? slot + row * kHeadDim + 2 * p : &sm.part[row][2 * p]) = s;
    }
    if (slot && threadIdx.x < RT) {
      slot[RT * kHeadDim + threadIdx.x] = sm.pm[threadIdx.x];
      slot[RT * kHeadDim + RT + threadIdx.x] = sm.pt[threadIdx.x];
      slot[RT * kHeadDim + 2 * RT + threadIdx.x] = sm.pl[threadIdx.x];
    }
    if (a.streamed) {
      if (x < x1) {  // the next tile's copies go over what was just read and written here
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncthreads();
      }
      continue;
    }
    if (whole) return;
    cluster_barrier();
    for (int it = threadIdx.x + part * kAtThreads; it < RT * 64; it += parts * kAtThreads) {
      const int row = it >> 6, p = it & 63;
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
      put_out<DT>(a, slice, tile.cnt, r0 + row, 2 * p, s, l, top - topt);
    }
    cluster_barrier();  // no CTA leaves while another reads its shared memory
  }
}

// Joins the parts of the tiles that several CTAs of a streamed launch share,
// and zeroes tiles that see nothing. One CTA a row of a tile: every part's
// factor first, then a thread sums a pair of values over each eighth part and
// the eight sums are added in order.
constexpr int kMergeThreads = 512;
constexpr int kMergeGroups = kMergeThreads / 64;
constexpr int kMergeEarly = 4;  // parts that a thread loads while the factors are made
static_assert(kAtGroups <= kMergeThreads, "a thread checks one (sequence, row tile)");
constexpr int kMaxCtas = 1024;

template <int DT, int NT>
__global__ void __launch_bounds__(kMergeThreads, 3) k_attend8_merge(const __grid_constant__ AttendArgs a, int ctas) {
  __shared__ Stream stream;
  constexpr int RT = 8 * NT, kSlot = AtSmem<NT>::kSlot;
  __shared__ float factor[kMaxCtas];
  __shared__ float2 sums[kMergeGroups][64];
  __shared__ float total_l, unit;
  __shared__ int range[3];
  const int G = a.c.batch * a.row_tiles, row = blockIdx.y;
  const int gi = blockIdx.x / a.c.n_kv_heads, h = blockIdx.x % a.c.n_kv_heads;
  const int b = gi % a.c.batch, rt = gi / a.c.batch;
  const int64_t slice = (int64_t)b * a.c.n_kv_heads + h;
  const int p = threadIdx.x & 63, grp = threadIdx.x >> 6;
  auto slot = [&](int j) { return a.ws + (2 * (int64_t)(range[0] + j) + (j == 0 ? range[2] : 0)) * kSlot; };
  auto part_at = [&](int j) { return *(const float2 *)(slot(j) + row * kHeadDim + 2 * p); };
  float2 early[kMergeEarly];
  int np;
  // Which CTAs share the tile follows from the lengths and counts. They are
  // read ahead of the wait, where nothing vouches for them yet, and again
  // behind it: if they were others then, the second turn has them right.
  // (Reading them behind the wait alone: 1 to 1.5 us a call.)
  for (int turn = 0;; ++turn) {
    stream.fill(a, RT, 1, 0);
    if (threadIdx.x == 0) {
      const int nb = stream.nu[gi];
      const int64_t total = stream.at[G], P = min((int64_t)ctas, total), p0 = stream.at[gi] + (int64_t)h * nb;
      range[0] = range[1] = range[2] = 0;
      if (nb > 0) {  // CTAs range[0].. share the tile; the first one's part is its second if it began before
        range[0] = stream.owner(p0, total, P);
        range[1] = stream.owner(p0 + nb - 1, total, P) - range[0] + 1;
        range[2] = total * range[0] / P < p0;
      }
    }
    __syncthreads();
    if (turn == 0) wait_prerequisites();  // by every CTA: this kernel's end stands for the first one's
    np = range[1];
    const bool others = threadIdx.x < G && stream.nu[threadIdx.x] != Tile(a, threadIdx.x % a.c.batch, threadIdx.x / a.c.batch, RT).nb;
#pragma unroll
    for (int k = 0; k < kMergeEarly; ++k)
      early[k] = np > 1 && grp + k * kMergeGroups < np ? part_at(grp + k * kMergeGroups) : make_float2(0.f, 0.f);
    if (threadIdx.x < 32 && np != 1) {
      const int lane = threadIdx.x;
      float top = -INFINITY, topt = -INFINITY, l = 0.f;
      for (int j = lane; j < np; j += 32) {
        top = fmaxf(top, slot(j)[RT * kHeadDim + row]);
        topt = fmaxf(topt, slot(j)[RT * kHeadDim + RT + row]);
      }
#pragma unroll
      for (int d = 16; d; d /= 2) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        topt = fmaxf(topt, __shfl_xor_sync(0xffffffffu, topt, d));
      }
      for (int j = lane; j < np; j += 32) {
        factor[j] = share(slot(j)[RT * kHeadDim + row], top);
        l += share(slot(j)[RT * kHeadDim + RT + row], topt) * slot(j)[RT * kHeadDim + 2 * RT + row];
      }
#pragma unroll
      for (int d = 16; d; d /= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
      if (lane == 0) {
        total_l = l;
        unit = top - topt;
      }
    }
    if (!__syncthreads_or(others) || turn == 1) break;
  }
  if (np == 1 || rt * RT + row >= a.n * a.group) return;  // one CTA had it all, or the row is none
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kMergeEarly; ++k) {
    if (grp + k * kMergeGroups < np) {
      const float f = factor[grp + k * kMergeGroups];
      s.x += f * early[k].x;
      s.y += f * early[k].y;
    }
  }
#pragma unroll 4
  for (int j = grp + kMergeEarly * kMergeGroups; j < np; j += kMergeGroups) {
    const float2 x2 = part_at(j);
    const float f = factor[j];
    s.x += f * x2.x;
    s.y += f * x2.y;
  }
  sums[grp][p] = s;
  __syncthreads();
  if (grp) return;
#pragma unroll
  for (int j = 1; j < kMergeGroups; ++j) {
    s.x += sums[j][p].x;
    s.y += sums[j][p].y;
  }
  const int cnt = a.counts ? min(max(a.counts[b], 0), a.n) : a.n;
  put_out<DT>(a, slice, cnt, rt * RT + row, 2 * p, s, total_l, unit);
}

// How a call is split.
struct AttendPlan {
  int nt, row_tiles, cluster;
  int ctas;  // of a streamed launch, 0 if it is none
  bool rows; // the kernel for many rows
  int64_t tiles;
};

static const char *plan_attend(const lkv_cache8 *c, int32_t group, int32_t n, int32_t window, int32_t sinks, int32_t max_len, int sms,
                               AttendPlan *p) {
  const int64_t R = (int64_t)n * group, S = (int64_t)c->batch * c->n_kv_heads;
  if (R > 0x7fffffff - 256) return "too many rows";
  p->nt = R <= 8 ? 1 : 2;
  p->row_tiles = (int)((R + 8 * p->nt - 1) / (8 * p->nt));
  p->tiles = S * p->row_tiles;
  // tokens that a tile of `rows` rows may see, at most
  auto most = [&](int rows) {
    const int64_t len = max_len > 0 && max_len < c->capacity ? max_len : c->capacity;
    const int64_t seen = (int64_t)window + (sinks < c->capacity ? sinks : c->capacity) + (rows + group - 1) / group;
    return window > 0 && seen < len ? seen : len;
  };
  // Many rows go to the tensor memory's kernel where it is faster: its time
  // against this kernel's, in its steps, of which this one takes 0.4 for 16 rows
  // x 128 tokens on every SM and 3 to start. On a GB300, int8, 4 query heads,
  // this kernel's and its time: 64 slices of 32K tokens, 16 tokens each 363 and
  // 277 us; 8 slices, 16 tokens 58 and 73 us, 32 tokens 101 and 72; 8 slices of
  // 4096 tokens, 64 tokens 33 and 42 us; 64 slices of 256 tokens, 64 tokens 39
  // and 29 us.
  p->rows = false;
  p->ctas = 0;
  if (c->dtype == LKV_DTYPE_BF16) {
    const int64_t steps = (most(kRowsTile) + kRowsStep - 1) / kRowsStep + (window > 0);
    const double time = rows_plan(*c, R, window > 0 ? 0 : n, steps, sms, &p->ctas);
    p->rows = 0.4 * (double)(S * ((R + 15) / 16)) * steps / sms > time - 3;
    if (p->rows) return nullptr;
    p->ctas = 0;
  }
  const int64_t blocks = (most(8 * p->nt) + kBlock - 1) / kBlock + 1;
  int64_t slots = (int64_t)sms * (c->dtype == LKV_DTYPE_FP32 && p->nt == 2 ? 1 : 2);  // CTAs that the GPU holds
  if (slots > kMaxCtas) slots = kMaxCtas;
  int64_t cluster = slots / p->tiles, most_cluster = blocks / (2 * kAtWarps);  // a turn for every warp
  if (cluster > most_cluster) cluster = most_cluster;
  p->cluster = (int)(cluster < 1 ? 1 : cluster > kAtMaxCluster ? kAtMaxCluster : cluster);
  // Streamed where whole tiles would leave over two fifths of the GPU idle (in
  // their last wave) and are long enough to pay for the second kernel. On a
  // GB300, int8 and 4 query heads: 8 KV heads of 131,579 tokens 131 us as 64
  // CTAs in clusters, 53 us streamed; 2 of 8,000 tokens 14.4 and 10.1 us; 160
  // of 33,000 tokens 306 and 220 us; but 64 of 33,000 tokens (256 CTAs in
  // clusters) 89 and 105 us.
  const int64_t ctas = p->tiles * p->cluster, last = ctas <= slots ? ctas : ctas % slots;
  if (ctas < 3 * slots && last > 0 && last * 5 < slots * 3 && blocks >= 24 * p->cluster &&
      (int64_t)c->batch * p->row_tiles <= kAtGroups) {
    // at least 16 blocks for each CTA; few tiles: a whole number of CTAs each,
    // so that none begins two, and not the last ones (parts cost merging). With
    // 24, 27, 29 and 32 of 32 CTAs, us: 8 slices of 131,579 tokens 56.9, 52.8,
    // 53.0, 53.6; 16 of 60,000 51.8, 48.9, 48.5, 48.8; 4 of 65,000 22.0, 19.8,
    // 20.2, 20.0; one of 131,000 20.8, 20.1, 20.8, 20.9.
    int64_t most_ctas = p->tiles * blocks / 16;
    if (most_ctas < p->tiles) most_ctas = p->tiles;
    const int64_t full = slots * 27 / 32 < most_ctas ? slots * 27 / 32 : most_ctas;
    p->ctas = (int)(p->tiles * 4 <= full ? full / p->tiles * p->tiles : slots < most_ctas ? slots : most_ctas);
    p->cluster = 1;
  }
  if (p->tiles * p->cluster > 0x7fffffff) return "too many rows";
  return nullptr;
}

template <int DT, int CODE, int NT>
static cudaError_t launch_attend(const AttendArgs &a, const AttendPlan &p, const CUtensorMap &km, const CUtensorMap &vm, cudaStream_t st) {
  auto *fn = k_attend8<DT, CODE, NT>;
  constexpr int smem = 1024 + ((int)sizeof(AtSmem<NT>) > kRingBytes ? (int)sizeof(AtSmem<NT>) : kRingBytes);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(p.ctas ? p.ctas : p.tiles * p.cluster));
  cfg.blockDim = dim3(kAtThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = p.cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = p.ctas ? 1 : 2;
  e = cudaLaunchKernelEx(&cfg, fn, a, km, vm);
  if (e != cudaSuccess || !p.ctas) return e;
  cfg.gridDim = dim3((unsigned)p.tiles, 8 * NT);
  cfg.blockDim = dim3(kMergeThreads);
  cfg.dynamicSmemBytes = 0;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_attend8_merge<DT, NT>, a, p.ctas);
}

template <int DT, int CODE>
static cudaError_t launch_attend(const AttendArgs &a, const AttendPlan &p, const CUtensorMap &km, const CUtensorMap &vm, cudaStream_t st) {
  return p.nt == 1 ? launch_attend<DT, CODE, 1>(a, p, km, vm, st) : launch_attend<DT, CODE, 2>(a, p, km, vm, st);
}

// What the arguments of an attention call have to be, apart from the tensors.
static const char *check_attend(const lkv_cache8 *c, int32_t group, int32_t n, int32_t window, int32_t sinks, int32_t max_len) {
  if (const char *m = check_cache8(c)) return m;
  if (group < 1 || group > 128) return "group must be 1..128";
  if (n < 0 || n > (1 << 24)) return "n must be 0..2^24";
  if (window < 0 || sinks < 0 || max_len < 0) return "window, sinks and max_len must be >= 0";
  return nullptr;
}

static lkv_status refuse_in(const char *where, const char *why) {
  char buf[192];
  std::snprintf(buf, sizeof buf, "%s: %s", where, why);
  return refuse(buf);
}

static int64_t plan_bytes(const AttendPlan &p) {
  return p.rows ? rows_bytes(p.ctas) : p.ctas ? (int64_t)p.ctas * 2 * (p.nt == 1 ? AtSmem<1>::kSlot : AtSmem<2>::kSlot) * 4 : 0;
}

}  // namespace lkv

extern "C" lkv_status lkv_cache8_attend_workspace(const lkv_cache8 *c, int32_t group, int32_t n, int32_t window,
                                                  int32_t sinks, int32_t max_len, int64_t *bytes) {
  using namespace lkv;
  if (const char *m = check_attend(c, group, n, window, sinks, max_len)) return refuse_in("lkv_cache8_attend_workspace", m);
  if (!bytes) return refuse("lkv_cache8_attend_workspace: null result");
  *bytes = 0;
  if (n == 0) return LKV_OK;
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_refuse("lkv_cache8_attend_workspace", e);
  AttendPlan p;
  if (const char *m = plan_attend(c, group, n, window, sinks, max_len, sms, &p)) return refuse_in("lkv_cache8_attend_workspace", m);
  *bytes = plan_bytes(p);
  return LKV_OK;
}

extern "C" lkv_status lkv_cache8_attend(const lkv_cache8 *c, const void *q, int32_t group, int32_t n,
                                        const int32_t *counts, float scale, int32_t window, int32_t sinks,
                                        int32_t max_len, void *out, void *workspace, int64_t workspace_bytes,
                                        void *stream) {
  using namespace lkv;
  if (const char *m = check_attend(c, group, n, window, sinks, max_len)) return refuse_in("lkv_cache8_attend", m);
  const float scale_log2 = scale * kLog2e;
  if (!(scale_log2 - scale_log2 == 0.f)) return refuse("lkv_cache8_attend: scale, or its product with log2(e), is not finite");
  if (n == 0) return LKV_OK;
  if (!q || !out) return refuse("lkv_cache8_attend: null queries or output");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(counts, 4) || !aligned(workspace, 16))
    return refuse("lkv_cache8_attend: queries, output and workspace must be 16-byte aligned, counts 4-byte aligned");
  const int64_t S = (int64_t)c->batch * c->n_kv_heads;
  const int64_t bytes = S * group * n * kHeadDim * (c->dtype == LKV_DTYPE_BF16 ? 2 : 4), ib = (int64_t)c->batch * 4;
  if (overlaps_cache8(c, out, bytes) || overlap(out, bytes, q, bytes) || overlap(out, bytes, counts, ib))
    return refuse("lkv_cache8_attend: the output overlaps the cache or an input");
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_refuse("lkv_cache8_attend", e);
  AttendPlan p;
  if (const char *m = plan_attend(c, group, n, window, sinks, max_len, sms, &p)) return refuse_in("lkv_cache8_attend", m);
  const int64_t need = plan_bytes(p);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return refuse("lkv_cache8_attend: the workspace is smaller than lkv_cache8_attend_workspace says");
    if (overlaps_cache8(c, workspace, need) || overlap(workspace, need, q, bytes) || overlap(workspace, need, out, bytes) ||
        overlap(workspace, need, counts, ib))
      return refuse("lkv_cache8_attend: the workspace overlaps another tensor");
  }
  AttendArgs a{};
  a.c = *c;
  a.q = q;
  a.out = out;
  a.counts = counts;
  a.n = n;
  a.group = group;
  a.window = window >= c->capacity ? 0 : window;  // a window that reaches everything is none
  a.sinks = sinks < c->capacity ? sinks : c->capacity;
  a.scale_log2 = scale_log2;
  a.row_tiles = p.rows ? 0 : p.row_tiles;
  a.streamed = p.ctas > 0;
  a.ws = (float *)workspace;
  if (p.rows) {
    e = launch_attend_rows(a, p.ctas, (cudaStream_t)stream);
    return e == cudaSuccess ? LKV_OK : cuda_refuse("lkv_cache8_attend", e);
  }
  CUtensorMap km, vm;
  if (!codes_map(&km, c->k_codes, c->capacity, S, kBlock) || !codes_map(&vm, c->v_codes, c->capacity, S, kBlock)) {
    set_unbound_error("lkv_cache8_attend: the driver refused a tensor map of the codes");
    return LKV_ECUDA;
  }
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf = c->dtype == LKV_DTYPE_BF16, i8 = c->code == LKV_CODE_INT8;
  if (bf) e = i8 ? launch_attend<1, LKV_CODE_INT8>(a, p, km, vm, st) : launch_attend<1, LKV_CODE_E4M3>(a, p, km, vm, st);
  else e = i8 ? launch_attend<0, LKV_CODE_INT8>(a, p, km, vm, st) : launch_attend<0, LKV_CODE_E4M3>(a, p, km, vm, st);
  return e == cudaSuccess ? LKV_OK : cuda_refuse("lkv_cache8_attend", e);
}
