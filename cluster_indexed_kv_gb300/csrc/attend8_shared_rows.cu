// attend8_shared_rows.cu -- attention behind shared prefixes on tcgen05, for bf16
// caches: the prefixes' part, and for many rows a sequence the own tokens' too.
#include "attend8_rows.cuh"
#include "attend8_shared.cuh"
#include "tma.cuh"

namespace lkv {

// A CTA takes pieces of 128-row tiles (attend8_shared.cuh), 128 tokens (8 blocks,
// a step) at a time. With one row tile, steps take the place that row tiles have
// in attend8_rows.cu: even and odd steps have four softmax warps each, a
// reference, a total and an accumulator of their own, and while one half weighs
// its step the tensor cores work for the other.
//   - Four warps turn K's codes into fp16 tiles (exact), four V's, both as they
//     lie in the cache, a row a token (128-byte swizzle); the next step's codes are
//     in registers meanwhile. The product with V takes its tile with d along the
//     rows, so nothing is transposed (which took half of a step's work).
//   - One warp issues: S = Q K^T, and O += P V with P in tensor memory over S.
//   - One warp reads the blocks' scales, four steps ahead.
//   - Weights, references and units are those of attend8_rows.cu. At a piece's end
//     the halves are added, row by row, and one copy takes the part to memory.
// Tensor memory: S and O of both halves, all 512 columns.
//
// Bound, a step of 128 rows: products 1024 clocks; shared memory 1280 (Q, K and V
// read by the products, K and V written), 1540 with the codes that pass through the
// same memory on their way in; bytes 1390 at the measured copy rate. It takes 2130
// (8 x 256 tokens behind 16K) to 2400 (a step of 16 or 32 samples): the chain of a
// half, weights 2850 and then P V and the next S 1000 to 1400, is two steps long,
// and the producers work 1500 to 1800 of the time. With 54 steps a CTA (32 samples
// with 4 new tokens each behind 32K, profiled): tensor pipe 39% active, issue slots
// 50%, LSU data pipe 47%. Beside the steps a piece costs its beginning (5000
// clocks: tables, rows, queries, each a round trip or two) and its end (3000 to
// 4000). On a GB300, 8 KV heads, 4 query heads: 32 samples of a 32K prompt, 14 steps a
// CTA, 30 us; 8 x 256 tokens behind 16K 535 us, 1.03 PFLOP/s, 52% of the measured
// bf16 rate. Measured before, the latter: K, V and scales by the same four warps
// 2870 us; warps with one role each 751; V as it lies and a whole warp along with
// the issuing lane 637 (a lane on its own took 1900 clocks a step to issue); 7
// steps counted for a tile's beginning, 535. Slower: the scores of 64 tokens at a
// time, over columns that the other half's weights do not need (the wait for S
// goes, but Q is read twice: a call 599 against 570); rows that fill half a tile
// twice in it, each time for half of a step's tokens (half the weights a warp, but
// the products' queue grows as long; 3% faster there, 4% slower elsewhere); every
// warp finding its pieces by itself (registers: 680 against 637).
constexpr uint32_t kShSmem = 5 * kRwTile + 1024;  // Q, K: 2, V: 2
static_assert(kSharedRows == kRwRows && kSharedStep == kRwTok, "a tile is one of tensor memory's");

// Warps: softmax of the even steps and of the odd ones, producers of K and of V,
// and a fifth group with the issuing warp and the one that reads scales. The
// launch's registers (96 a thread) are shared out anew: 136, 80 and 48 a thread
// of these, 480 a lane of an SM's quarter in all.
constexpr int kShSoft = 8, kShK = 8, kShV = 12, kShIssuer = 16, kShScales = 17, kShThreads = 20 * 32;
template <int N>
__device__ __forceinline__ void registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// Products with shared-memory operands by the low words of their descriptors
// (the address in 16-byte units): K-major as rw_desc, and V as it lies in the
// cache, d along a row of 64 (128-byte swizzle), 8 tokens 1 KB and the other 64
// values of d kRwHalf apart.
constexpr uint32_t kShHi = (1024u >> 4) | (1u << 14) | (2u << 29);
constexpr uint32_t kShIdescV = kRwIdesc | (1u << 16);
__device__ __forceinline__ void mma_ss2(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n .reg .b64 x, y;\n setp.ne.b32 p, %5, 0;\n mov.b64 x, {%1, %3};\n mov.b64 y, {%2, %3};\n"
               " tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n}"
               ::"r"(d), "r"(a | (1u << 16)), "r"(b | (1u << 16)), "r"(kShHi), "r"(kRwIdesc), "r"(acc));
}
__device__ __forceinline__ void mma_ts2(uint32_t d, uint32_t a, uint32_t b, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n .reg .b64 y;\n setp.ne.b32 p, %5, 0;\n mov.b64 y, {%2, %3};\n"
               " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %4, p;\n}"
               ::"r"(d), "r"(a), "r"(b | ((kRwHalf >> 4) << 16)), "r"(kShHi), "r"(kShIdescV), "r"(acc));
}
__device__ __forceinline__ void group_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

// What a CTA is at.
struct SharedPiece {
  Prefixes<true>::Piece p;
  int64_t x, end;             // of the row of units: where the CTA is, and its end
  const uint8_t *codes[2];    // the list's cache: K's and V's codes, scales and tails of the KV head
  const float *scale[2];
  const uint16_t *tail[2];
  int len;
  int go;                     // whether there is a piece
  int dead;                   // a wait in an earlier one has given up: this one has no steps, but tiles and parts are told of
  int once;                   // whether its tokens are read for this row tile alone
  int last;                   // the last token that a row sees
  uint32_t top, tail_top[2];  // largest V scale of the piece's blocks, largest magnitudes of the tails (bits)
  int64_t at[kRwRows];        // the rows' queries, -1 for none
  int pos[kRwRows];           // the last token that a row sees
  float rc[kRwRows];          // query unit * scale * log2(e)
  float ref[2][kRwRows], l[2][kRwRows];  // references and totals of the even and odd steps
};

// A piece's steps and units, as every warp forms them.
struct Steps {
  int s0, s1, nb, full, tail_rows;
  bool tail;  // the partial block is among them, as the last
  __device__ __forceinline__ explicit Steps(const SharedPiece &p) {
    nb = (p.len + kBlock - 1) / kBlock;
    full = p.len / kBlock;
    tail_rows = p.len - full * kBlock;
    // steps behind the last token that a row sees are nobody's
    s0 = max(p.p.u0 - kSharedStart, 0);
    s1 = p.dead ? s0 : max(min(p.p.u1 - kSharedStart, (p.last + kRwTok) / kRwTok), s0);
    tail = s1 > s0 && full < nb && s1 * kRwBlocks >= nb;
  }
};
// V scales count in units of 2^unit; tails in units of 2^ke and 2^ve.
struct Units {
  int ke, ve, unit;
  __device__ __forceinline__ Units(const SharedPiece &p, bool tail) {
    ke = exponent_of(p.tail_top[0]);
    ve = exponent_of(p.tail_top[1]);
    unit = max(max((int)(p.top >> 23) - 127, -126), tail ? ve : -126);
  }
};

// What both halves of the softmax have of a row goes into the piece's part: each
// half's threads bring 64 of the values of d into `stage`, from where one copy
// takes them; the rows' exponents and totals go straight to the part.
__device__ __forceinline__ void store_part(const SharedArgs &a, const SharedPiece &z, int steps, int done, int unit, uint32_t tmem, float *stage) {
  const int w = threadIdx.x >> 7, r = threadIdx.x & 127;
  const bool valid = z.at[r] >= 0, has0 = steps > 1 || (done & 1) == 0, has1 = steps > 1 || (done & 1) == 1;
  const float m0 = valid && has0 ? z.ref[0][r] : -INFINITY, m1 = valid && has1 ? z.ref[1][r] : -INFINITY;
  const float top = fmaxf(m0, m1), f0 = share(m0, top), f1 = share(m1, top);
  const uint32_t o0 = tmem + ((uint32_t)(r & 96) << 16) + 256 + 64 * w, o1 = o0 + 128;
  if (__any_sync(0xffffffffu, valid)) {
#pragma unroll 1
    for (int d = 0; d < 64; d += 16) {
      uint32_t u[16], v[16];
      if (has0) tmem_ld16(o0 + d, u);
      if (has1) tmem_ld16(o1 + d, v);
      if (has0) tmem_wait16(u);
      if (has1) tmem_wait16(v);
      float o[16];
#pragma unroll
      for (int e = 0; e < 16; ++e)
        o[e] = (has0 && f0 != 0.f ? f0 * __uint_as_float(u[e]) : 0.f) + (has1 && f1 != 0.f ? f1 * __uint_as_float(v[e]) : 0.f);
#pragma unroll
      for (int e = 0; e < 16; e += 4) *(float4 *)(stage + part_place(r, 64 * w + d + e)) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  group_sync(1, 32 * kShSoft);
  float *const part = a.parts + ((int64_t)blockIdx.x + z.p.tile) * part_floats(kRwRows);
  if (threadIdx.x == 0) {
    bulk_store(part, stage, kRwRows * kHeadDim * 4);
    bulk_commit();
  }
  if (w == 0) {
    float *const p = part + kRwRows * kHeadDim + r;
    p[0] = top == -INFINITY ? top : top + (float)unit;
    p[kRwRows] = top;
    p[2 * kRwRows] = valid ? (has0 ? f0 * z.l[0][r] : 0.f) + (has1 ? f1 * z.l[1][r] : 0.f) : 0.f;
  }
}

template <int CODE>
__global__ void __launch_bounds__(kShThreads, 1) k_shared_rows(const __grid_constant__ SharedArgs a) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) RowsSync sy;
  __shared__ __align__(8) uint64_t scempty[4];
  __shared__ float4 scales[4][kRwBlocks];  // a block's K scale, log2 and reciprocal of its V scale's share of the unit, first token
  __shared__ uint32_t tmem_s;
  __shared__ volatile int abort_s;
  __shared__ __align__(16) uint16_t tails[2][kBlock * kHeadDim];  // K's and V's partial block, zeros behind its rows
  __shared__ SharedPiece seg;
  const uint32_t base = (smem_at(raw) + 1023u) & ~1023u;
  unsigned char *const area = raw + (base - smem_at(raw));
  const uint32_t q_at = base, k_at = base + kRwTile, v_at = base + 3 * kRwTile;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;  // the warp: uniform for the compiler too
  Prefixes<true> pre(a, area + 5 * kRwTile);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&sy.kfull[i], 4);
      bar_init(&sy.kempty[i], 1);
      bar_init(&sy.vfull[i], 4);
      bar_init(&sy.vempty[i], 1);
      bar_init(&sy.sfull[i], 1);
      bar_init(&sy.pfull[i][0], 4);
      bar_init(&sy.pfull[i][1], 4);
      bar_init(&sy.odone[i][0], 1);
      bar_init(&sy.odone[i][1], 1);
    }
    for (int i = 0; i < 4; ++i) {
      bar_init(&sy.scfull[i], 1);
      bar_init(&scempty[i], 1);
    }
    bar_init(&sy.drained, 1);
    bar_init_fence();
    abort_s = 0;
  }
  if (warp == kShIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(&tmem_s)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  wait_prerequisites();
  launch_vouched(a);
  pre.fill(a);
  if (threadIdx.x == 32 * kShK) pre.share(a, seg.x, seg.end);
  tmem_before();
  __syncthreads();
  tmem_after();
  const uint32_t tmem = tmem_s;
  int done = 0;  // steps of earlier pieces: the barriers' phases go on

  // Every warp passes the same four barriers a piece: (1) the piece before is
  // done with, (2) the piece is named, (3) its rows are, (4) queries, units and
  // tails are in place. Then each has its part of the steps.
  if (warp < kShSoft) {
    // ---------------------------------------------------------------- softmax
    registers_up<136>();
    // Four warps take the even steps, four the odd ones; both hold all rows,
    // each with a reference, a total and an accumulator of its own.
    const int w = warp >> 2, row = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_at = tmem + lanes + w * 128, o_at = tmem + lanes + 256 + w * 128;
    while (true) {
      __syncthreads();
      __syncthreads();
      if (!seg.go) break;
      if (w == 0) {
        const ListRow x = list_row(a, pre, seg.p.list, seg.p.h, seg.len, (int64_t)seg.p.rt * kRwRows + row);
        seg.at[row] = x.at;
        seg.pos[row] = x.pos;
        const int top = __reduce_max_sync(0xffffffffu, x.at < 0 ? -1 : x.pos);
        if (lane == 0 && top >= 0) atomicMax(&seg.last, top);
      }
      __syncthreads();
      {
        // queries as fp16 in units of a power of two into the swizzled tile, 16 lanes a row, 16 rows a warp
        const int half = lane >> 4, run = lane & 15;
        uint4 q[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int64_t at = seg.at[warp * 16 + 2 * k + half];
          q[k] = at >= 0 ? *(const uint4 *)((const uint16_t *)a.q + at * kHeadDim + 8 * run) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int rr = warp * 16 + 2 * k + half;
          uint32_t m = __vmaxu2(__vmaxu2(q[k].x & 0x7fff7fffu, q[k].y & 0x7fff7fffu), __vmaxu2(q[k].z & 0x7fff7fffu, q[k].w & 0x7fff7fffu));
#pragma unroll
          for (int d = 8; d > 0; d /= 2) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
          const int e = exponent_of(max(m << 16, m & 0xffff0000u));
          const float f = pow2f(-e);
          if (run == 0) seg.rc[rr] = pow2f(e) * a.scale_log2;
          const uint32_t x[4] = {q[k].x, q[k].y, q[k].z, q[k].w};
          uint32_t h[4];
#pragma unroll
          for (int v = 0; v < 4; ++v)
            h[v] = h2_bits(__floats2half2_rn(__uint_as_float(x[v] << 16) * f, __uint_as_float(x[v] & 0xffff0000u) * f));
          unsigned char *to = area + (run >> 3) * kRwHalf + rr * 128;
          *(uint4 *)(to + (((run & 7) ^ (rr & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      }
      // the producers write where the part before is copied from
      if (threadIdx.x == 0) bulk_wait_read<0>();
      __syncthreads();
      const bool valid = seg.at[row] >= 0, any = __any_sync(0xffffffffu, valid);
      const int pos = valid ? seg.pos[row] : -1;
      const float rc = seg.rc[row];
      const int last_open = (int)__reduce_min_sync(0xffffffffu, (uint32_t)(valid ? pos + 1 : 0x7fffffff)) - kBlock;  // first token of the last whole block
      const int end = done + Steps(seg).s1 - Steps(seg).s0;
      float ref = 0.f, l = 0.f, limit = valid ? -1.f : INFINITY;  // limit: of a block's sum of weights
      bool seen = !valid;
      bool ok = true;
      int g = done + ((done ^ w) & 1);
      if (!any) {  // no row of this warp's is there
        for (; ok && g < end; g += 2) {
          ok = rows_wait_warp(&sy.sfull[w], (g >> 1) & 1, &abort_s, a.limit_ns);
          if (ok && lane == 0) {
            bar_arrive(&sy.pfull[w][0]);
            bar_arrive(&sy.pfull[w][1]);
          }
        }
      }
#pragma unroll 1
      for (; ok && g < end; g += 2) {
        ok = rows_wait_warp(&sy.scfull[g & 3], (g >> 2) & 1, &abort_s, a.limit_ns);
        if (!ok) break;
        const float4 *const sc = scales[g & 3];
        const bool open = __float_as_int(sc[kRwBlocks - 1].w) <= last_open;
        ok = rows_wait_warp(&sy.sfull[w], (g >> 1) & 1, &abort_s, a.limit_ns);
        if (!ok) break;
        tmem_after();
        float sum = 0.f;
        uint32_t x[32];
        tmem_ld32(s_at, x);
        // four blocks at a time, two by two: scores become weights, over the
        // columns of blocks that have been read
#pragma unroll 1
        for (int b = 0; b < kRwBlocks; b += 4) {
          uint32_t p[32];
          float t[4];
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const float4 sc0 = sc[b + 2 * v], sc1 = sc[b + 2 * v + 1];
            float y[32];
            tmem_wait32(x);
            {
              const float f0 = rc * sc0.x, at0 = sc0.y - ref, f1 = rc * sc1.x, at1 = sc1.y - ref;
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float f = e < 16 ? f0 : f1, at = e < 16 ? at0 : at1;
                const float2 z = fma_2(make_float2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), make_float2(f, f), make_float2(at, at));
                y[e] = z.x;
                y[e + 1] = z.y;
              }
            }
            if (v == 0 || b + 4 < kRwBlocks) tmem_ld32(s_at + 16 * (b + 2 * v + 2), x);
            if (!open) {
              const int see0 = pos - __float_as_int(sc0.w), see1 = pos - __float_as_int(sc1.w);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if ((e & 15) > (e < 16 ? see0 : see1)) y[e] = -INFINITY;
            }
#pragma unroll
            for (int e = 0; e < 32; ++e) y[e] = ex2(y[e]);
            float2 z[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              z[k] = make_float2(y[8 * k], y[8 * k + 1]);
#pragma unroll
              for (int e = 2; e < 8; e += 2) z[k] = add_2(z[k], make_float2(y[8 * k + e], y[8 * k + e + 1]));
#pragma unroll
              for (int e = 0; e < 4; ++e) p[16 * v + 4 * k + e] = h2_bits(__floats2half2_rn(y[8 * k + 2 * e], y[8 * k + 2 * e + 1]));
            }
            z[0] = add_2(z[0], z[1]);
            z[2] = add_2(z[2], z[3]);
            t[2 * v] = z[0].x + z[0].y;
            t[2 * v + 1] = z[2].x + z[2].y;
          }
          // a weight is at most its block's sum: below the limit none leaves fp16's range
          if (__any_sync(0xffffffffu, !(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) <= limit))) {
            tmem_wait32(x);  // the scores on their way, before registers change hands
            const RowState z = move_reference(RowState{ref, l, sum, limit, seen}, s_at, o_at, sc, rc, open, pos, 0, 0, b,
                                              g - done >= 2 || b > 0, b > 0 ? &sy.odone[w][0] : nullptr, (g >> 1) & 1, &abort_s);
            ref = z.ref;
            l = z.l;
            sum = z.sum;
            limit = z.limit;
            seen = z.seen;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) sum = __fmaf_rn(t[k], sc[b + k].z, sum);
            tmem_st32(s_at + 8 * b, p);
          }
          tmem_wait_st();
          tmem_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&sy.pfull[w][b >> 2]);
        }
        l += sum;
      }
      // the last step's product, if there was one
      if (ok && any && end - done > ((done ^ w) & 1)) ok = rows_wait_warp(&sy.odone[w][1], ((g - 2) >> 1) & 1, &abort_s, a.limit_ns);
      // (a row whose scores are all NaN has no reference, but l and O, which are NaN, count)
      seg.ref[w][row] = seen ? ref : -INFINITY;
      seg.l[w][row] = l;
      tmem_before();
      group_sync(1, 32 * kShSoft);
      tmem_after();
      {
        const Steps st(seg);
        if (st.s1 > st.s0) {
          store_part(a, seg, st.s1 - st.s0, done, Units(seg, st.tail).unit, tmem, (float *)(area + kRwTile));
        } else if (w == 0) {
          float *const p = a.parts + ((int64_t)blockIdx.x + seg.p.tile) * part_floats(kRwRows) + kRwRows * kHeadDim + row;
          p[0] = p[kRwRows] = -INFINITY;
          p[2 * kRwRows] = 0.f;
        }
        done += st.s1 - st.s0;
      }
    }
    if (threadIdx.x == 0) {
      bulk_wait_all();
      if (a.late && blockIdx.x == 0) vouch(a);
    }
    tmem_before();
    __syncthreads();
  } else if (warp < kShIssuer) {
    // ---------------------------------------------------------------- producers
    registers_down<80>();
    const int pw = warp & 3, kv = warp >= kShV;  // K's, and V's
    while (true) {
      __syncthreads();
      if (threadIdx.x == 32 * kShK) {
        seg.go = seg.x < seg.end;
        seg.dead = abort_s;
        if (seg.go) {
          const Prefixes<true>::Piece p = pre.piece(a, seg.x, seg.end);
          if (p.u0 == 0) pre.announce(a, p, seg.x);
          seg.p = p;
          auto from = [&](const lkv_cache8 &c, int b) {
            const int64_t slice = (int64_t)b * c.n_kv_heads + p.h, codes = slice * c.capacity * kHeadDim, tail = slice * kBlock * kHeadDim;
            seg.codes[0] = (const uint8_t *)c.k_codes + codes;
            seg.codes[1] = (const uint8_t *)c.v_codes + codes;
            seg.scale[0] = c.k_scale + slice * (c.capacity / kBlock);
            seg.scale[1] = c.v_scale + slice * (c.capacity / kBlock);
            seg.tail[0] = (const uint16_t *)c.k_tail + tail;
            seg.tail[1] = (const uint16_t *)c.v_tail + tail;
          };
          if (p.list < a.p.batch) from(a.p, p.list);
          else from(a.c, p.list - a.p.batch);
          seg.len = pre.len(p.list);
          seg.once = pre.tiles[p.list + 1] - pre.tiles[p.list] == a.c.n_kv_heads;
          seg.x += p.u1 - p.u0;
          seg.top = seg.tail_top[0] = seg.tail_top[1] = 0;
          seg.last = -1;
        }
      }
      __syncthreads();
      if (!seg.go) break;
      __syncthreads();
      const Steps z(seg);
      const int s0 = z.s0, s1 = z.s1;
      uint4 cr[8];
      const uint8_t *const codes = seg.codes[kv] + (32 * pw + (lane >> 3)) * kHeadDim + 16 * (lane & 7);
      // 4 whole rows a load, 16 codes a lane: a load takes a pass for each 128-byte
      // line. What is read for one row tile alone passes by the caches (16 samples
      // of 131K tokens 97 -> 88 us), what others read too stays (8 x 256
      // tokens behind 16K, 64 row tiles a KV head: 582 us where it does not, 570).
      const bool once = seg.once;
      auto load = [&](int j) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const int b = j * kRwBlocks + 2 * pw + (t >> 2);
          const uint4 *p = (const uint4 *)(codes + ((int64_t)j * kRwTok + 4 * t) * kHeadDim);
          cr[t] = make_uint4(0, 0, 0, 0);
          if (b < z.full) cr[t] = once ? __ldcs(p) : *p;
        }
      };
      if (s1 > s0) load(s0);
      {
        // the unit of the V scales, and the tails with their largest values
        const int t = threadIdx.x - 32 * kShK, stride = 32 * (kShIssuer - kShK);
        const float *const vsc = seg.scale[1];
        uint32_t top = 0;
#pragma unroll 4
        for (int u = s0 * kRwBlocks + t; u < min(s1 * kRwBlocks, z.full); u += stride) top = max(top, __float_as_uint(vsc[u]));
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0 && top) atomicMax(&seg.top, top);
        if (z.tail) {
          constexpr int kRun = kBlock * kHeadDim / 8;  // 16-byte runs of a tail: as many as there are threads here
          static_assert(kRun == 32 * (kShIssuer - kShK), "each takes a run of both");
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint4 x = make_uint4(0, 0, 0, 0);
            if (t / 16 < z.tail_rows) x = *(const uint4 *)(seg.tail[k] + t * 8);
            *(uint4 *)(tails[k] + t * 8) = x;
            uint32_t m = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
            m = __reduce_max_sync(0xffffffffu, max(m << 16, m & 0xffff0000u));
            if (lane == 0) atomicMax(&seg.tail_top[k], m);
          }
        }
      }
      __syncthreads();
      const Units un(seg, z.tail);
      const float tf = pow2f(kv ? -max(un.ve, un.unit - kUnitSpan) : -un.ke);
      const int tail_at = (z.nb - 1) % kRwBlocks * kBlock;
      for (int g = done; g < done + s1 - s0; ++g) {
        const int j = g - done + s0, st = g & 1;
        const bool ends = z.tail && (j + 1) * kRwBlocks >= z.nb;  // the step's last block is the partial one
        if (!rows_wait_warp(kv ? &sy.vempty[st] : &sy.kempty[st], ((g >> 1) & 1) ^ 1, &abort_s, a.limit_ns)) break;
        unsigned char *const to_tile = area + (1 + 2 * kv + st) * kRwTile;
        const int half = (lane >> 2) & 1, run = lane & 3;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          // a run's 16-byte chunks go to places 2 run and 2 run + 1, the second
          // half's in the other order: 8 lanes fill 8 places of a row at a time
          const int r = 32 * pw + 4 * t + (lane >> 3);
          const uint4 c = half ? make_uint4(cr[t].z, cr[t].w, cr[t].x, cr[t].y) : cr[t];
          uint32_t x[8];
          codes_row<CODE>(c.x, x[0], x[1]);
          codes_row<CODE>(c.y, x[2], x[3]);
          codes_row<CODE>(c.z, x[4], x[5]);
          codes_row<CODE>(c.w, x[6], x[7]);
          unsigned char *to = to_tile + half * kRwHalf + r * 128;
          *(uint4 *)(to + (((2 * run + half) ^ (r & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
          *(uint4 *)(to + (((2 * run + 1 - half) ^ (r & 7)) << 4)) = make_uint4(x[4], x[5], x[6], x[7]);
        }
        if (j + 1 < s1) load(j + 1);
        if (ends) {
          __syncwarp();  // over the zeros of the rows' own warp
          if (pw == tail_at / 32) {
#pragma unroll 1
            for (int r = 0; r < z.tail_rows; ++r) {
              const int at = tail_at + r, d = 4 * lane;
              const uint2 x = *(const uint2 *)(tails[kv] + r * kHeadDim + d);
              const uint32_t h0 = h2_bits(__floats2half2_rn(__uint_as_float(x.x << 16) * tf, __uint_as_float(x.x & 0xffff0000u) * tf));
              const uint32_t h1 = h2_bits(__floats2half2_rn(__uint_as_float(x.y << 16) * tf, __uint_as_float(x.y & 0xffff0000u) * tf));
              *(uint2 *)(to_tile + (d >> 6) * kRwHalf + at * 128 + ((((d & 63) >> 3) ^ (at & 7)) << 4) + (d & 7) * 2) = make_uint2(h0, h1);
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(kv ? &sy.vfull[st] : &sy.kfull[st]);
      }
      done += s1 - s0;
    }
    __syncthreads();
  } else {
    registers_down<48>();
    while (true) {
      __syncthreads();
      __syncthreads();
      if (!seg.go) break;
      __syncthreads();
      __syncthreads();
      const Steps z(seg);
      const int end = done + z.s1 - z.s0;
      if (warp == kShIssuer) {
        // -------------------------------------------------------------- products
        // The whole warp goes along, one lane issues: descriptors and addresses stay
        // in uniform registers.
        const int first = __shfl_sync(0xffffffffu, done, 0), stop = __shfl_sync(0xffffffffu, min(end, a.hold), 0);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint32_t q_lo = q_at >> 4, k_lo = k_at >> 4, v_lo = v_at >> 4;
        const bool one = elect_one();
        tmem_after();
        auto qk = [&](int g) {
          const int w = g & 1;
          if (!rows_wait_warp(&sy.kfull[w], (g >> 1) & 1, &abort_s, a.limit_ns)) return false;
          tmem_after();
          if (one) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t at = ((k >> 2) * kRwHalf + (k & 3) * 32) >> 4;
              mma_ss2(tm + w * 128, q_lo + at, k_lo + w * (kRwTile >> 4) + at, k > 0);
            }
            mma_commit(&sy.sfull[w]);
            mma_commit(&sy.kempty[w]);
          }
          __syncwarp();
          return true;
        };
        // O += P V of a step's first and then second 64 tokens, each as soon as its weights are there
        auto pv = [&](int g) {
          const int w = g & 1;
          if (!rows_wait_warp(&sy.vfull[w], (g >> 1) & 1, &abort_s, a.limit_ns)) return false;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!rows_wait_warp(&sy.pfull[w][h], (g >> 1) & 1, &abort_s, a.limit_ns)) return false;
            tmem_after();
            if (one) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts2(tm + 256 + w * 128, tm + w * 128 + 32 * h + 8 * k, v_lo + w * (kRwTile >> 4) + (4 * h + k) * (16 * 128 >> 4),
                        g - first >= 2 || h > 0 || k > 0);
              mma_commit(&sy.odone[w][h]);
              if (h) {
                mma_commit(&sy.vempty[w]);
                mma_commit(&scempty[g & 3]);
              }
            }
            __syncwarp();
          }
          return true;
        };
        bool ok = first >= stop || (qk(first) && (stop - first < 2 || qk(first + 1)));
        for (int g = first; ok && g < stop; ++g) ok = pv(g) && (g + 2 >= stop || qk(g + 2));
      } else if (warp == kShScales) {
        // -------------------------------------------------------------- scales
        const Units un(seg, z.tail);
        const float *const ksc = seg.scale[0], *const vsc = seg.scale[1];
        // four steps' blocks at a time, a lane each, read four steps ahead
        float k = 0.f, v = 0.f;
        auto load = [&](int g) {
          const int b = (g - done + z.s0) * kRwBlocks + lane;
          if (b < z.full) {
            k = ksc[b];
            v = vsc[b];
          }
        };
        load(done);
        bool ok = true;
        for (int g = done; ok && g < end; g += 4) {
          const int b = (g - done + z.s0) * kRwBlocks + lane;
          float4 s = make_float4(0.f, 0.f, 1.f, __int_as_float(kNoToken));
          if (b < z.nb) {
            const float kk = b < z.full ? k : pow2f(un.ke);
            const float vv = b < z.full ? fmaxf(v * pow2f(-un.unit), pow2f(-kUnitSpan)) : pow2f(max(un.ve, un.unit - kUnitSpan) - un.unit);
            s = make_float4(kk, log2f(vv), 1.f / vv, __int_as_float(b * kBlock));
          }
          load(g + 4);
#pragma unroll 1
          for (int i = g; ok && i < min(g + 4, end); ++i) {
            ok = rows_wait_warp(&scempty[i & 3], ((i >> 2) & 1) ^ 1, &abort_s, a.limit_ns);
            if (!ok) break;
            if (lane / kRwBlocks == i - g) scales[i & 3][lane % kRwBlocks] = s;
            __syncwarp();
            if (lane == 0) bar_arrive(&sy.scfull[i & 3]);
          }
        }
      }
      done = end;
    }
    __syncthreads();
    tmem_after();
    if (warp == kShIssuer) {
      if (elect_one()) {  // every product (of this lane, as elected before) has completed before the tensor memory is freed
        mma_commit(&sy.drained);
        bar_wait(&sy.drained, 0);
        if (abort_s) atomicOr(a.c.ticket + a.c.batch, kAnomTimeout);
      }
      __syncwarp();
      tmem_after();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_s), "r"(512) : "memory");
    }
  }
}

// Joins the parts of every row, of its prefix and of its own tokens: a warp a
// row, a lane four values of d. Where the parts of both lie is read at once, and
// then kJoinAtOnce parts at a time. Bound by round trips: 65,536 rows of 2 to 3
// parts 35 us, 100 MB (a part after another 42 us).
constexpr int kJoinWarps = 8, kJoinAtOnce = 4;
__global__ void __launch_bounds__(32 * kJoinWarps) k_shared_join(const __grid_constant__ SharedArgs a) {
  wait_prerequisites();
  const int lane = threadIdx.x & 31, per = a.n * a.group, d = 4 * lane;
  const uint32_t id = blockIdx.x * kJoinWarps + threadIdx.x / 32;
  const int slice = (int)(id / (uint32_t)per), row = (int)(id % (uint32_t)per);
  if (slice >= a.c.batch * a.c.n_kv_heads) return;
  const int b = (int)((uint32_t)slice / (uint32_t)a.c.n_kv_heads), h = slice - b * a.c.n_kv_heads;
  const int i = (int)((uint32_t)row / (uint32_t)a.group), cnt = a.counts ? min(max(__ldcg(a.counts + b), 0), a.n) : a.n;
  float top = -INFINITY, topt = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (i < cnt) {
    const int4 sq = a.seq[b];
    // the row in the prefix's list, and in its own
    const int64_t there = (int64_t)sq.y * per + row, rt = quotient(there, kSharedRows);
    const int tile0 = sq.x + (int)rt * a.c.n_kv_heads + h, tile1 = sq.z + row / kSharedRows * a.c.n_kv_heads + h;
    const int2 none = make_int2(0, 0), who0 = sq.x >= 0 ? a.tile[tile0] : none, who1 = sq.z >= 0 ? a.tile[tile1] : none;
    const float *const at0 = a.parts + ((int64_t)who0.x + tile0) * part_floats(kSharedRows);
    const float *const at1 = a.parts + ((int64_t)who1.x + tile1 - who0.y) * part_floats(kSharedRows);
    const int r0 = (int)(there - rt * kSharedRows), r1 = row % kSharedRows, n = who0.y + who1.y;
    for (int j0 = 0; j0 < n; j0 += kJoinAtOnce) {
      float4 x[kJoinAtOnce];
      float m[kJoinAtOnce], t[kJoinAtOnce], mine[kJoinAtOnce];
#pragma unroll
      for (int k = 0; k < kJoinAtOnce; ++k) {
        const int j = j0 + k, r = j < who0.y ? r0 : r1;
        const float *part = (j < who0.y ? at0 : at1) + (int64_t)j * part_floats(kSharedRows);
        m[k] = t[k] = -INFINITY;
        mine[k] = 0.f;
        if (j < n) {
          x[k] = *(const float4 *)(part + part_place(r, d));
          const float *p = part + kSharedRows * kHeadDim + r;
          m[k] = p[0];
          t[k] = p[kSharedRows];
          mine[k] = p[2 * kSharedRows];
        }
      }
      float above = top, abovet = topt;
#pragma unroll
      for (int k = 0; k < kJoinAtOnce; ++k) {
        above = fmaxf(above, m[k]);
        abovet = fmaxf(abovet, t[k]);
      }
      const float f = share(top, above);
      o.x = f == 0.f ? 0.f : f * o.x;
      o.y = f == 0.f ? 0.f : f * o.y;
      o.z = f == 0.f ? 0.f : f * o.z;
      o.w = f == 0.f ? 0.f : f * o.w;
      l *= share(topt, abovet);
#pragma unroll
      for (int k = 0; k < kJoinAtOnce; ++k) {
        const float g = share(m[k], above);
        l += share(t[k], abovet) * mine[k];
        if (g != 0.f) {  // a part that saw nothing holds anything
          o.x += g * x[k].x;
          o.y += g * x[k].y;
          o.z += g * x[k].z;
          o.w += g * x[k].w;
        }
      }
      top = above;
      topt = abovet;
    }
  }
  const bool none = l == 0.f;
  const float scale = none ? 0.f : 1.f / l, back = none ? 0.f : exp2f(top - topt);
  uint16_t *out = (uint16_t *)a.out + (((int64_t)slice * a.group + row - i * a.group) * a.n + i) * kHeadDim + d;
  *(uint2 *)out = none ? make_uint2(0, 0) : make_uint2(pack_bf16(o.x * scale * back, o.y * scale * back), pack_bf16(o.z * scale * back, o.w * scale * back));
}

cudaError_t launch_shared_rows(const SharedArgs &a, int ctas, cudaStream_t st) {
  auto *fn = a.c.code == LKV_CODE_INT8 ? k_shared_rows<LKV_CODE_INT8> : k_shared_rows<LKV_CODE_E4M3>;
  const size_t smem = kShSmem + (size_t)Prefixes<true>::bytes(a.c.batch, a.p.batch, a.own_parts);
  static SmemAllowed allowed[2];
  const cudaError_t e = allowed[a.c.code == LKV_CODE_INT8].allow((const void *)fn, (int)(kShSmem + Prefixes<true>::bytes(kSharedMost, kSharedMost, true)));
  return e != cudaSuccess ? e : launch_next(fn, dim3((unsigned)ctas), kShThreads, smem, st, a);
}

cudaError_t launch_shared_join(const SharedArgs &a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.n * a.group * a.c.batch * a.c.n_kv_heads;
  if (rows > 0x7fffffff) return cudaErrorInvalidValue;
  return launch_next(k_shared_join, dim3((unsigned)((rows + kJoinWarps - 1) / kJoinWarps)), 32 * kJoinWarps, 0, st, a);
}

}  // namespace lkv
