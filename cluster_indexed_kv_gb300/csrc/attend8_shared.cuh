// attend8_shared.cuh -- attention behind shared prefixes: what its kernels share.
//
// The rows of all sequences behind one prefix are one list, sequence by
// sequence (in the order of the batch), each token-major as elsewhere; runs of
// part_rows of them are the prefix's row tiles. All tiles' work, prefix by
// prefix, row tile by row tile and KV head by KV head, is one row of units (runs
// of part_blocks blocks of a tile), of which each CTA takes an even share. What
// it makes of a tile is a part: slot (CTA + tile) of the workspace, as each step
// along the row goes to the next CTA, the next tile, or both. Calls of many rows
// a sequence put the sequences' own tokens behind the prefixes in the same row,
// as lists of one sequence each.
#pragma once

#include "attend8.cuh"

namespace lkv {

constexpr int kSharedMost = 1024;  // sequences, and prefixes, that a call takes

struct SharedArgs : AttendArgs {
  lkv_cache8 p;               // the prefixes
  const int32_t *prefix_of;   // null: all of prefix 0
  int32_t part_rows;
  int32_t least_units;        // that a CTA takes, at least
  int32_t own_parts;          // whether the sequences' own tokens are parts too
  int4 *seq;                  // [batch]: the first tile of the sequence's prefix (-1: none), its place behind that prefix, its own first tile (-1: none)
  int2 *tile;                 // [tiles]: a tile's first CTA, and how many it has
  float *parts;
  uint64_t *vouch;            // what the first kernel vouches with, another value each time (see vouch)
  int32_t late;               // it does so at its end (lkv_diag_shared_late)
  int32_t hold;               // the step of each CTA from which on there are no products (lkv_diag_shared_hold)
  uint64_t limit_ns;          // of a wait between a CTA's warps
};

// The second kernel begins while the first still runs, and takes the sequences' own
// tokens meanwhile, which the launches before both have written. What the first
// one's wait (griddepcontrol.wait) promises, it promises the first kernel; so one of
// its threads passes it on, behind that wait: it releases the time at `vouch` (in
// ticks of 32 ns, never the same for two calls, which take microseconds), and
// each warp of the second kernel acquires what stands there ahead of its reads. Behind
// its own wait it looks again: if it is the same, it was this call's, and everything
// before the release was there to be read. If it is not, the tokens are taken again.
__device__ __forceinline__ void vouch(const SharedArgs &a) {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(a.vouch), "l"(t) : "memory");
}
// What stands there, by the lane that also issues the warp's copies.
__device__ __forceinline__ uint64_t vouched(const SharedArgs &a) {
  uint64_t t;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(t) : "l"(a.vouch) : "memory");
  asm volatile("fence.proxy.async.global;" ::: "memory");
  return t;
}
// The same behind the kernel's own wait.
__device__ __forceinline__ uint64_t vouched_now(const SharedArgs &a) {
  uint64_t t;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(t) : "l"(a.vouch));
  return t;
}
// The first kernel's threads, behind their wait: the second may start.
__device__ __forceinline__ void launch_vouched(const SharedArgs &a) {
  if (threadIdx.x == 0) {
    if (blockIdx.x == 0 && !a.late) vouch(a);
    launch_dependents();
  }
}

// A part: the rows of o, then the exponents of the units of o and l, and l of
// each. Four values of d go together, those of row r at place (d / 4) ^ (r % 32):
// a thread a row fills shared memory so without bank conflicts, and a warp still
// reads a row as one run. (As [d / 4][row][4], which a thread a row writes as
// whole runs, joining 8 rows took 10 us.)
__host__ __device__ constexpr int part_floats(int rows) { return rows * (kHeadDim + 3); }
__host__ __device__ __forceinline__ int part_place(int row, int d) { return row * kHeadDim + (((d >> 2) ^ (row & 31)) << 2); }

__device__ __forceinline__ int held(const lkv_cache8 &c, int b) { return min(max(__ldcg(c.lengths + b), 0), c.capacity); }

// a / b, both >= 0, in 32 bits where they fit: most do, and several such
// quotients stand between a CTA and its first copy.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  return ((uint64_t)a | (uint64_t)b) >> 32 ? a / b : (int64_t)((uint32_t)a / (uint32_t)b);
}

// Row tiles of the kernel for many rows of bf16 caches, its units, and the steps'
// time that beginning a tile costs it. With 4, 7, 10 and 14: 8 x 256 tokens behind
// 16K 635, 573, 581 and 596 us; 32 x 5 behind 8K 62, 59, 64 and 73.
constexpr int kSharedRows = 128, kSharedStep = 128, kSharedStart = 7;
// The same for tiles of 16, in blocks, where a CTA may begin a second one. With 0, 16,
// 24 and 30: 5 fp32 samples behind 5 prefixes of 100 to 16000 tokens 76, 51, 44
// and 38 us; 6 behind one of 8191 35.5, 33.4, 32.1 and 31.6.
constexpr int kSharedFewStart = 30;

// The work, in shared memory: list e < G is prefix e's, and list G + b
// sequence b's own. ROWS: for tiles of 128.
template <bool ROWS>
struct Prefixes {
  int64_t *at;       // [lists + 1]: units before each list's tiles
  int *tiles;        // [lists + 1]: tiles before
  int *plen;         // [G]: the prefixes' tokens
  int *pnu;          // [G]: units of one of a prefix's tiles
  int *first;        // [G + 1]: sequences before, in `order`
  int *before;       // [batch]: a sequence's own tokens before its first row
  int *rows;         // [batch]: tokens of its rows that are no padding
  int16_t *order;    // [batch]: sequences, prefix by prefix
  int16_t *of;       // [batch]: the sequence's prefix, -1 for none (or an empty one)
  int *plan;         // start and ctas as below
  int G, lists, run;
  int start;         // units that stand for what beginning a tile costs, where a CTA may have several, before those of its blocks
  int ctas;          // that take part

  static __host__ __device__ int64_t bytes(int batch, int G, bool own) {
    return 12 * (int64_t)(G + (own ? batch : 0) + 2) + 12 * (int64_t)(G + 1) + 12 * (int64_t)batch + 8;
  }
  __device__ Prefixes(const SharedArgs &a, void *area) : G(a.p.batch), lists(a.p.batch + (a.own_parts ? a.c.batch : 0)),
                                                          run(ROWS ? kSharedStep : kBlock), start(ROWS ? kSharedStart : kSharedFewStart), ctas(1) {
    const int B = a.c.batch;
    at = (int64_t *)area;
    tiles = (int *)(at + lists + 1);
    plen = tiles + lists + 1;
    pnu = plen + G;
    first = pnu + G;
    before = first + G + 1;
    rows = before + B;
    order = (int16_t *)(rows + B);
    of = order + B;
    plan = (int *)(of + B);
  }
  // a list's tokens, and the units of one of its tiles
  __device__ __forceinline__ int len(int list) const { return list < G ? plen[list] : before[list - G] + rows[list - G]; }
  __device__ __forceinline__ int units(int tokens) const { return start + (int)((uint32_t)(tokens + run - 1) / (uint32_t)run); }
  __device__ __forceinline__ int nu(int list) const { return list < G ? pnu[list] : units(len(list)); }
  __device__ void fill(const SharedArgs &a) {
    const int B = a.c.batch;
    // everything that is read, at once
    for (int b = threadIdx.x; b < B; b += blockDim.x) {
      const int g = a.prefix_of ? __ldcg(a.prefix_of + b) : 0, mine = held(a.c, b);
      const int cnt = a.counts ? min(max(__ldcg(a.counts + b), 0), a.n) : a.n;
      of[b] = (int16_t)(g >= 0 && g < G ? g : -1);
      before[b] = mine - cnt;
      rows[b] = cnt;
    }
    for (int g = threadIdx.x; g < G; g += blockDim.x) {
      pnu[g] = 0;
      plen[g] = held(a.p, g);
    }
    __syncthreads();
    // (loops are kept short: code that runs once costs its fetching, 10,000 clocks of it when these were unrolled)
    if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      const uint32_t below = (1u << lane) - 1u;
#pragma unroll 1
      for (int turn = 0; turn < 2; ++turn) {  // how many sequences a prefix has, then their places
#pragma unroll 1
        for (int b0 = 0; b0 < B; b0 += 32) {
          const int b = b0 + lane;
          int g = b < B ? of[b] : -1;
          if (g >= 0 && plen[g] == 0) of[b] = g = -1;
          const uint32_t same = __match_any_sync(0xffffffffu, g >= 0 ? g : -2 - lane);
          const int had = g >= 0 ? pnu[g] : 0;
          if (turn && g >= 0) order[had + __popc(same & below)] = (int16_t)b;
          __syncwarp();
          if (g >= 0 && (same & below) == 0) pnu[g] = had + __popc(same);
          __syncwarp();
        }
        if (turn) break;
        int64_t sum = 0;
        int nt = 0, seqs = 0, most = 0;  // tiles, sequences, the largest list's tiles
#pragma unroll 1
        for (int e0 = 0; e0 < lists; e0 += 32) {
          const int e = e0 + lane;
          const int tokens = e < lists ? len(e) : 0, have = e < G ? pnu[e] : tokens > 0;  // and sequences that see them
          const int rt = (int)quotient((int64_t)have * a.n * a.group + a.part_rows - 1, a.part_rows);
          int64_t u = (int64_t)rt * a.c.n_kv_heads * units(tokens);
          int t = rt * a.c.n_kv_heads, s = e < G ? have : 0;
          const int mine = s;
          most = max(most, t);
#pragma unroll 1
          for (int d = 1; d < 32; d *= 2) {
            const int64_t u2 = __shfl_up_sync(0xffffffffu, u, d);
            const int t2 = __shfl_up_sync(0xffffffffu, t, d), s2 = __shfl_up_sync(0xffffffffu, s, d);
            if (lane >= d) {
              u += u2;
              t += t2;
              s += s2;
            }
          }
          if (e < lists) {
            at[e + 1] = sum + u;
            tiles[e + 1] = nt + t;
          }
          if (e < G) {
            first[e + 1] = seqs + s;
            pnu[e] = seqs + s - mine;  // where its sequences begin
          }
          sum += __shfl_sync(0xffffffffu, u, 31);
          nt += __shfl_sync(0xffffffffu, t, 31);
          seqs += __shfl_sync(0xffffffffu, s, 31);
        }
        if constexpr (!ROWS) {
          // a CTA for each tile at least; one list whose tiles can each have CTAs of
          // their own is shared so, and evenly
          int P = (int)min((int64_t)gridDim.x, max((int64_t)nt, quotient(sum - (int64_t)nt * start, a.least_units))), stand = start;
          if (__reduce_max_sync(0xffffffffu, most) == nt && nt > 0) {
            if (P < (int)gridDim.x) P -= P % nt;
            if (P % nt == 0) {
              sum -= (int64_t)nt * start;
              stand = 0;
#pragma unroll 1
              for (int e = lane; e < lists; e += 32)
                if (at[e + 1]) at[e + 1] = sum;
            }
          }
          if (lane == 0) {
            plan[0] = stand;
            plan[1] = P;
          }
        }
        if (lane == 0) at[0] = tiles[0] = first[0] = 0;
        __syncwarp();
      }
    }
    __syncthreads();
    if constexpr (!ROWS) {
      start = plan[0];
      ctas = plan[1];
    } else {
      ctas = (int)min((int64_t)gridDim.x, max((int64_t)1, quotient(at[lists], a.least_units)));
    }
    for (int g = threadIdx.x; g < G; g += blockDim.x) pnu[g] = units(plen[g]);
    if (blockIdx.x == 0) {
      auto own = [&](int b) { return lists > G && tiles[G + b + 1] > tiles[G + b] ? tiles[G + b] : -1; };
      for (int b = threadIdx.x; b < B; b += blockDim.x)
        if (of[b] < 0) a.seq[b] = make_int4(-1, 0, own(b), 0);
      for (int i = threadIdx.x; i < first[G]; i += blockDim.x) {
        const int b = order[i], g = of[b];
        a.seq[b] = make_int4(tiles[g], i - first[g], own(b), 0);
      }
    }
    __syncthreads();
  }
  // this CTA's units
  __device__ __forceinline__ void share(const SharedArgs &a, int64_t &x0, int64_t &x1) const {
    const int64_t total = at[lists], P = ctas;
    x0 = blockIdx.x < P ? quotient(total * blockIdx.x, P) : 0;
    x1 = blockIdx.x < P ? quotient(total * (blockIdx.x + 1), P) : 0;
  }
  // a piece of unit x's tile: up to unit x1 of the row
  struct Piece { int list, h, rt, tile, u0, u1; };  // u0, u1: of its units, the start's among them
  __device__ __forceinline__ Piece piece(const SharedArgs &a, int64_t x, int64_t x1) const {
    int lo = 0, hi = lists;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (at[mid] <= x) lo = mid;
      else hi = mid;
    }
    const int64_t off = x - at[lo];
    const int per = nu(lo), idx = (int)quotient(off, per);
    Piece p;
    p.list = lo;
    p.rt = (int)((uint32_t)idx / (uint32_t)a.c.n_kv_heads);
    p.h = idx - p.rt * a.c.n_kv_heads;
    p.tile = tiles[lo] + idx;
    p.u0 = (int)(off - (int64_t)idx * per);
    p.u1 = (int)min((int64_t)per, p.u0 + (x1 - x));
    return p;
  }
  // the tile that begins at unit x of the row, for whoever joins its parts (one thread of the CTA that has the unit)
  __device__ __forceinline__ void announce(const SharedArgs &a, const Piece &p, int64_t x) const {
    const int64_t P = ctas, last = x + nu(p.list) - 1;
    // the last CTA that begins at or before unit `last`
    a.tile[p.tile] = make_int2((int)blockIdx.x, (int)quotient(P * (last + 1) - 1, at[lists]) - (int)blockIdx.x + 1);
  }
};

// Row r of a list: where its query is (in rows of q, of KV head h) and the last
// of the list's `len` tokens that it sees; at < 0: no row, or padding.
struct ListRow { int64_t at; int pos; };
template <bool ROWS>
__device__ __forceinline__ ListRow list_row(const SharedArgs &a, const Prefixes<ROWS> &p, int list, int h, int len, int64_t r) {
  ListRow x{-1, -1};
  const int per = a.n * a.group, G = a.p.batch;
  const int64_t m = quotient(r, per);
  if (m >= (list < G ? p.first[list + 1] - p.first[list] : 1)) return x;
  const int b = list < G ? p.order[p.first[list] + (int)m] : list - G, rest = (int)(r - m * per);
  const int i = (int)((uint32_t)rest / (uint32_t)a.group);
  if (i >= p.rows[b]) return x;
  x.pos = max(list < G ? len + min(p.before[b] + i, -1) : p.before[b] + i, -1);
  x.at = (((int64_t)b * a.c.n_kv_heads + h) * a.group + rest - i * a.group) * a.n + i;
  return x;
}

// The kernel for many rows of bf16 caches and the join of what it leaves
// (attend8_shared_rows.cu).
cudaError_t launch_shared_rows(const SharedArgs &a, int ctas, cudaStream_t st);
cudaError_t launch_shared_join(const SharedArgs &a, cudaStream_t st);

}  // namespace lkv
