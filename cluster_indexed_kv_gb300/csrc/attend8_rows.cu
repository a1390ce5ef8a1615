// attend8_rows.cu -- causal attention of many rows over the 8-bit cache
// (lkv_cache8_attend for prompts and chunks of bf16 caches) on tcgen05.
#include <type_traits>

#include "attend8.cuh"

namespace lkv {

// A CTA takes 256 rows (token-major, as in k_attend8) of one (sequence, KV
// head), as two tiles of 128, and walks their visible blocks 128 tokens (8
// blocks, a step) at a time:
//   - 4 producer warps turn codes into fp16 tiles (exact), K token-major and V
//     transposed, both K-major with 128-byte swizzle; the next tile's codes
//     are in registers meanwhile;
//   - one thread issues the products: S = Q K^T (fp16, fp32 in tensor memory)
//     and O += P V with P read from tensor memory;
//   - 4 warps a row tile, a thread a row, take S to weights P (fp16, over S's
//     columns), 64 tokens at a time: the first 64's product runs while the
//     next 64 are weighed, and while they work on one row tile, the tensor
//     cores work on the other's P V and next S.
// The weights are those of k_attend8: y = score + log2(u), u the V scale of
// the block in units of the largest visible one, w = 2^(y - reference), out =
// sum w code / sum w / u; a row's reference moves only when a block's weights
// pass 2^15 in all, so O is hardly ever touched between products.
//
// A CTA a tile leaves SMs idle where there are few tiles or a broken last wave:
// then the launch is streamed, all tiles' steps shared out evenly over a CTA an
// SM, and the parts of tiles that several CTAs share are joined (rows_plan).
//
// Bound, a step of 256 rows: the products take 2048 clocks; shared memory about
// 2000 (Q, K and V tiles read by the products, K and V written), the
// exponentials (32 a clock and SM) 1024. It takes about 4000: nothing is
// saturated (tensor pipe 44%, issue slots 41%), the chain of a row tile is as
// long as that: S 650, weights 2150 (450 of them the first read of S), the
// last half's P V 300, and the barriers between them, with the other row tile's
// products in between. 2048 tokens over 32K, 32 query and 8 KV heads on a
// GB300: 1020 to 1030 us, 1.04 PFLOP/s, 55% of the measured bf16 rate. Slower: a row
// tile's first softmax thread issuing its products (no issuing warp, 168
// registers, 1214 us); S in halves of 64 tokens, each with its barrier (1135);
// a quarter of the exponentials as polynomials (1086).
constexpr int kRwTok = kRowsStep;                // tokens of a K / V tile
constexpr int kRwBlocks = kRwTok / kBlock;
constexpr int kRwRows = kRowsTile / 2;           // rows of a row tile
constexpr int kRwProducer = 8;                   // first producer warp
constexpr int kRwIssuer = 12;                    // the issuing warp
constexpr int kRwThreads = 13 * 32;
constexpr uint32_t kRwTile = kRwTok * kHeadDim * 2;  // 32 KB: two 64-column halves of 16 KB
constexpr uint32_t kRwHalf = kRwTile / 2;
constexpr uint32_t kRwSmem = 6 * kRwTile + 1024;     // Q: 2, K: 2, V: 2
constexpr int kRwSlot = 2 * kRwRows * (kHeadDim + 3); // floats of a part in the workspace
constexpr int kRwStart = 6;                      // steps' time that beginning a tile costs
constexpr uint32_t kRwIdesc = (1u << 4) | ((uint32_t)(kRwTok >> 3) << 17) | ((uint32_t)(kRwRows >> 4) << 24);  // fp16 x fp16 -> fp32

__device__ __forceinline__ uint64_t rw_desc(uint32_t saddr) {  // K-major, 128-byte swizzle, 8-row groups 1 KB apart
  uint64_t d = (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}"
               ::"r"(d), "l"(a), "l"(b), "r"(kRwIdesc), "r"(acc));
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t acc) {
  asm volatile("{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}"
               ::"r"(d), "r"(a), "l"(b), "r"(kRwIdesc), "r"(acc));
}
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_at(bar)) : "memory");
}
__device__ __forceinline__ void tmem_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 16 columns of the thread's lane; valid after tmem_wait16 on the same array.
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_wait16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t at, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t at, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
      ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
// 32 columns of the thread's lane; valid after tmem_wait32 on the same array.
__device__ __forceinline__ void tmem_ld32(uint32_t at, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, "
      "%18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]),
        "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(at));
}
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float2 fma_2(float2 a, float2 b, float2 c) {
  float2 d;
  asm("{\n .reg .b64 ra, rb, rc, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n mov.b64 rc, {%6, %7};\n"
      " fma.rn.f32x2 rd, ra, rb, rc;\n mov.b64 {%0, %1}, rd;\n}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return d;
}
__device__ __forceinline__ float2 add_2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n add.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}"
      : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

struct RowsSync {
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], scfull[4], drained;
  uint64_t pfull[2][2], odone[2][2];  // [row tile][half of the tokens]: one phase a step
};

// Wait for the phase; false, and the abort flag raised, when it does not come
// in time or another wait of the CTA has given up.
__device__ __forceinline__ bool rows_wait(uint64_t *bar, uint32_t phase, volatile int *abort) {
  if (bar_try(bar, phase)) return true;
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  while (!bar_try(bar, phase)) {
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (*abort || t - t0 > kCopyLimitNs) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// The same for a whole warp, uniformly.
__device__ __forceinline__ bool rows_wait_warp(uint64_t *bar, uint32_t phase, volatile int *abort) {
  return __all_sync(0xffffffffu, rows_wait(bar, phase, abort));
}

// The e of a largest magnitude (bits) < 2^e, within the fp32 scales' reach.
__device__ __forceinline__ int exponent_of(uint32_t bits) { return min(max((int)(bits >> 23) - 126, -100), 126); }

// A row's softmax: reference, sum of w / u before and in this tile, the block
// sum of weights past which the reference moves, and whether there is one.
struct RowState {
  float ref, l, sum, limit;
  bool seen;
};

// The rare turn of the softmax, out of its loop's way: references of a warp's
// rows move (kPShift below a row's largest y, up only once there is one), what
// tensor memory holds of the tile's weights and of O follows, and the four
// blocks from b on are weighed from their scores. The row sees all of their
// tokens (open) or what token_range says. The step's first half finds O (if
// there has been a product) at rest; its second half waits for the first
// half's product (odone), which has also read that half's weights.
__device__ __noinline__ RowState move_reference(RowState z, uint32_t s_at, uint32_t o_at, const float4 *scale, float rc, bool open, int pos,
                                                int window, int sinks, int b, bool has_o, uint64_t *odone, uint32_t phase,
                                                volatile int *abort) {
  float far = -INFINITY;
  auto scores = [&](int c, uint32_t(&x)[32]) {  // y of two of the four blocks
    tmem_ld32(s_at + 16 * b + 32 * c, x);
    tmem_wait32(x);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 sc = scale[b + 2 * c + k];
      const float f = rc * sc.x, at = sc.y - z.ref;
      int see[3];
      token_range(__float_as_int(sc.w), pos, window, sinks, see);
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const float v = __fmaf_rn(__uint_as_float(x[16 * k + e]), f, at);
        x[16 * k + e] = __float_as_uint(open || sees(see, e) ? v : -INFINITY);
      }
    }
  };
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    uint32_t x[32];
    scores(c, x);
#pragma unroll
    for (int e = 0; e < 32; ++e) far = fmaxf(far, __uint_as_float(x[e]));
  }
  float by = far - kPShift;
  if (z.seen ? by < 0.f : far == -INFINITY) by = 0.f;
  const float k = z.seen ? exp2f(-by) : 1.f;
  z.seen |= far > -INFINITY;
  z.limit = z.seen ? 0x1p15f : -1.f;
  z.ref += by;
  z.l *= k;
  z.sum *= k;
  if (__any_sync(0xffffffffu, k != 1.f)) {
    // (if it is not in time the CTA gives up)
    if (odone) rows_wait_warp(odone, phase, abort);
    if (has_o) {
      tmem_after();
#pragma unroll 1
      for (int d = 0; d < kHeadDim; d += 32) {
        uint32_t x[32];
        tmem_ld32(o_at + d, x);
        tmem_wait32(x);
#pragma unroll
        for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * k);
        tmem_st32(o_at + d, x);
      }
      tmem_wait_st();
    }
  }
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {  // weights over columns whose scores have been read: 16 c.. behind 32 c..
    uint32_t x[32], p[16];
    scores(c, x);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float t = 0.f;
#pragma unroll
      for (int e = 16 * k; e < 16 * k + 16; e += 2) {
        const float w0 = ex2(__uint_as_float(x[e])), w1 = ex2(__uint_as_float(x[e + 1]));
        t += w0 + w1;
        p[e / 2] = h2_bits(__floats2half2_rn(w0, w1));
      }
      z.sum = __fmaf_rn(t, scale[b + 2 * c + k].z, z.sum);
    }
    tmem_st16(s_at + 8 * b + 16 * c, p);
  }
  return z;
}

// What a CTA is at: steps [s0, s1) of a tile. In shared memory, read again
// where it is needed after the loop over steps, which has no registers left.
struct Segment {
  Tile tile;
  int64_t slice;
  int r0, s0, s1;
  int whole;               // all of the tile's steps (or its end, if it has none)
  int units;               // streamed: of the share (steps, and kRwStart of them for each tile's beginning)
  int done;                // streamed: steps of earlier segments (the barriers' phases go on)
  int64_t x, begin, end;   // streamed: the CTA's share of all tiles' steps: where it is, began and ends
};

// Which tile a CTA of a streamed launch has the first part of, the next ones
// being the next CTAs' first: 0 parts where it finished all that it began.
struct __align__(16) RowsJoin {
  int parts, slice, row_tile, second;  // second: this CTA's is its second part
};

template <int CODE, bool STREAMED>
__global__ void __launch_bounds__(kRwThreads, 1) k_attend8_rows(const __grid_constant__ AttendArgs a) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) RowsSync sy;
  __shared__ float4 scales[4][kRwBlocks];  // a block's K scale, log2 and reciprocal of its V scale's share of the unit, first token
  __shared__ uint32_t tmem_s;
  __shared__ volatile int abort_s;
  __shared__ uint32_t top_s;               // largest V scale of the visible blocks (bits)
  __shared__ uint32_t tail_s[2];           // largest magnitudes of the tails (bits)
  __shared__ __align__(16) uint16_t tails[2][kBlock * kHeadDim];  // K's and V's partial block, zeros behind its rows
  __shared__ std::conditional_t<STREAMED, Stream, int> stream;
  __shared__ Segment seg;
  const lkv_cache8 &c = a.c;
  const uint32_t base = (smem_at(raw) + 1023u) & ~1023u;
  unsigned char *const area = raw + (base - smem_at(raw));
  const uint32_t q_at = base, k_at = base + 2 * kRwTile, v_at = base + 4 * kRwTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = a.n * a.group, G = c.batch * a.row_tiles;

  wait_prerequisites();
  if constexpr (STREAMED) launch_dependents();
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
    for (int i = 0; i < 4; ++i) bar_init(&sy.scfull[i], 1);
    bar_init(&sy.drained, 1);
    bar_init_fence();
    abort_s = 0;
  }
  if (warp == kRwIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(&tmem_s)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncthreads();

  if constexpr (STREAMED) {
    stream.fill(a, 2 * kRwRows, kRwBlocks, kRwStart);
    if (threadIdx.x == 0) {
      stream.share(G, seg.x, seg.end);
      seg.begin = seg.x;
      seg.done = 0;
      // the tile that the share ends in: joined by this CTA's record if it has its first step but not its last
      RowsJoin join{0, 0, 0, 0};
      if (seg.x < seg.end) {
        const int gi = stream.group(seg.end - 1, G), n = stream.nu[gi];
        const int h = (int)((seg.end - 1 - stream.at[gi]) / n);
        const int64_t first = stream.at[gi] + (int64_t)h * n, step0 = first + kRwStart;
        if (seg.x <= step0 && step0 < seg.end && seg.end < first + n) {
          const int64_t total = stream.at[G];
          join.parts = stream.owner(first + n - 1, total, min((int64_t)gridDim.x, total)) - (int)blockIdx.x + 1;
          join.slice = gi % c.batch * c.n_kv_heads + h;
          join.row_tile = gi / c.batch;
          join.second = seg.x < first;
        }
      }
      *(RowsJoin *)(a.ws + 2 * (int64_t)gridDim.x * kRwSlot + blockIdx.x * (sizeof(RowsJoin) / 4)) = join;
    }
    __syncthreads();
  }
  while (!STREAMED || seg.x < seg.end) {
    if (threadIdx.x == 0) {
      int b, rt;
      if constexpr (STREAMED) {
        const int gi = stream.group(seg.x, G), n = stream.nu[gi];
        const int64_t off = seg.x - stream.at[gi];
        b = gi % c.batch;
        rt = gi / c.batch;
        seg.slice = (int64_t)b * c.n_kv_heads + off / n;
        const int u0 = (int)(off % n), u1 = (int)min((int64_t)n, u0 + (seg.end - seg.x));
        seg.units = u1 - u0;
        seg.s0 = max(u0 - kRwStart, 0);
        seg.s1 = max(u1 - kRwStart, 0);
        seg.whole = seg.s0 == 0 && u1 == n;
        seg.tile = Tile(a, b, rt, 2 * kRwRows);
      } else {
        const int64_t S = (int64_t)c.batch * c.n_kv_heads;
        seg.slice = blockIdx.x % S;
        b = (int)(seg.slice / c.n_kv_heads);
        rt = a.row_tiles - 1 - (int)(blockIdx.x / S);  // the rows with most to see come first
        seg.tile = Tile(a, b, rt, 2 * kRwRows);
        seg.s0 = 0;
        seg.s1 = (seg.tile.nb + kRwBlocks - 1) / kRwBlocks;
        seg.whole = 1;
      }
      seg.r0 = rt * 2 * kRwRows;
      top_s = tail_s[0] = tail_s[1] = 0;
    }
    __syncthreads();
    if (STREAMED && seg.s0 == seg.s1 && !seg.whole) {  // a tile's start alone: its steps are the next CTA's
      __syncthreads();
      if (threadIdx.x == 0) seg.x += seg.units;
      __syncthreads();
      continue;
    }
    const Tile tile = seg.tile;
    const int64_t slice = seg.slice;
    const int r0 = seg.r0, s0 = seg.s0, s1 = seg.s1, steps = s1 - s0, done = STREAMED ? seg.done : 0;
    // whether the second row tile has rows (streamed: it always takes part, so
    // that all barriers go through the same phases)
    const bool two = STREAMED || (r0 + kRwRows < R && (r0 + kRwRows) / a.group < tile.cnt);
    const int full = tile.len / kBlock;   // blocks before it are quantised
    const bool tail = tile.hi >= full && tile.nb > 0 && s1 * kRwBlocks >= tile.nb;  // the partial block is among them, as the last
    const int tail_rows = tile.len - full * kBlock;
    const float *const ksc = c.k_scale + slice * (c.capacity / kBlock), *const vsc = c.v_scale + slice * (c.capacity / kBlock);

    float rc = 0.f;
    int pos = -1;
    bool valid = false;
    if (warp < kRwProducer) {
      // queries as fp16 in units of a power of two into the swizzled tile, 16
      // lanes a row; a thread's own row (the one it will weigh) keeps its unit
      const int row = r0 + (int)threadIdx.x, own = row / a.group, half = lane >> 4, run = lane & 15;
      valid = row < R && own < tile.cnt;
      if (valid) pos = max(tile.len - tile.cnt + own, -1);
#pragma unroll 1
      for (int it = 0; it < 16; it += 8) {
        uint4 w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int at = r0 + warp * 32 + 2 * (it + k) + half, i = at / a.group;
          const bool there = at < R && i < tile.cnt;
          w[k] = there ? *(const uint4 *)((const uint16_t *)a.q + ((slice * a.group + at % a.group) * a.n + i) * kHeadDim + 8 * run)
                       : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          uint32_t m = __vmaxu2(__vmaxu2(w[k].x & 0x7fff7fffu, w[k].y & 0x7fff7fffu), __vmaxu2(w[k].z & 0x7fff7fffu, w[k].w & 0x7fff7fffu));
#pragma unroll
          for (int d = 8; d > 0; d /= 2) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, d));
          const int e = exponent_of(max(m << 16, m & 0xffff0000u));
          const float f = pow2f(-e), unit_q = pow2f(__shfl_sync(0xffffffffu, e, (lane & 1) * 16));
          if (lane >> 1 == it + k) rc = unit_q * a.scale_log2;
          const uint32_t x[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
          uint32_t h[4];
#pragma unroll
          for (int v = 0; v < 4; ++v)
            h[v] = h2_bits(__floats2half2_rn(__uint_as_float(x[v] << 16) * f, __uint_as_float(x[v] & 0xffff0000u) * f));
          const int rr = (warp & 3) * 32 + 2 * (it + k) + half;
          unsigned char *to = area + (warp >> 2) * kRwTile + (run >> 3) * kRwHalf + rr * 128;
          *(uint4 *)(to + (((run & 7) ^ (rr & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    } else {
      // the unit of the V scales, and the tails with their largest values
      const int t = threadIdx.x - 32 * kRwProducer, stride = kRwThreads - 32 * kRwProducer;
      uint32_t top = 0;
#pragma unroll 4
      for (int u = s0 * kRwBlocks + t; u < min(s1 * kRwBlocks, tile.nb); u += stride) {
        const int b = tile.block(u);
        if (b < full) top = max(top, __float_as_uint(vsc[b]));
      }
      top = __reduce_max_sync(0xffffffffu, top);
      if (lane == 0 && top) atomicMax(&top_s, top);
      if (tail) {
        constexpr int kRun = kBlock * kHeadDim / 8;  // 16-byte runs of a tail: a multiple of a warp's 32
#pragma unroll 4
        for (int k = t; k < 2 * kRun; k += stride) {
          const uint16_t *from = (const uint16_t *)(k < kRun ? c.k_tail : c.v_tail) + slice * kBlock * kHeadDim;
          uint4 w = make_uint4(0, 0, 0, 0);
          if (k % kRun / 16 < tail_rows) w = *(const uint4 *)(from + k % kRun * 8);
          *(uint4 *)(tails[k / kRun] + k % kRun * 8) = w;
          uint32_t m = __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
          m = __reduce_max_sync(0xffffffffu, max(m << 16, m & 0xffff0000u));
          if (lane == 0) atomicMax(&tail_s[k / kRun], m);
        }
      }
    }
    tmem_before();
    __syncthreads();
    tmem_after();
    const uint32_t tmem = tmem_s;
    const int ke = exponent_of(tail_s[0]), ve = exponent_of(tail_s[1]);
    const int unit = max(max((int)(top_s >> 23) - 127, -126), tail ? ve : -126);  // V scales count in units of 2^unit

    if (warp >= kRwProducer && warp < kRwIssuer) {
      // ---------------------------------------------------------------- producers
      const int pw = warp - kRwProducer;
      const uint8_t *kc = (const uint8_t *)c.k_codes + slice * c.capacity * kHeadDim;
      const uint8_t *vc = (const uint8_t *)c.v_codes + slice * c.capacity * kHeadDim;
      // K: 4 whole rows a load, 16 codes a lane: a load takes a pass for each
      // 128-byte line (8 half rows a load: 296 against 284 us for 32 tokens over
      // 32K, 64 slices). V: tokens 8 tc.., d 16 dc.., which fills its tile
      // without bank conflicts.
      const int kr_row = lane >> 3, kr_half = (lane >> 2) & 1, kr_run = lane & 3;
      const int tc = (pw * 32 + lane) & 15, dc = (pw * 32 + lane) >> 4;
      const float kf = pow2f(-ke), vf = pow2f(-max(ve, unit - kUnitSpan));
      uint4 kr[8], vr[8];
      auto load_k = [&](int j) {
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const int u = j * kRwBlocks + 2 * pw + (t >> 2), b = tile.block(u);
          const bool there = u < tile.nb && b < full;
          const uint8_t *p = kc + ((int64_t)b * kBlock + 4 * (t & 3) + kr_row) * kHeadDim + 16 * (lane & 7);
          kr[t] = there ? __ldg((const uint4 *)p) : make_uint4(0, 0, 0, 0);
        }
      };
      auto load_v = [&](int j) {
        const int u = j * kRwBlocks + (tc >> 1), b = tile.block(u);
        const bool there = u < tile.nb && b < full;
        const uint8_t *p = vc + ((int64_t)b * kBlock + 8 * (tc & 1)) * kHeadDim + 16 * dc;
#pragma unroll
        for (int i = 0; i < 8; ++i) vr[i] = there ? __ldg((const uint4 *)(p + i * kHeadDim)) : make_uint4(0, 0, 0, 0);
      };
      if (steps > 0) {
        load_k(s0);
        load_v(s0);
      }
      for (int g = done; g < done + steps; ++g) {
        const int j = g - done + s0, st = g & 1;
        // the blocks' scales
        if (pw == 0) {
          if (lane < kRwBlocks) {
            const int u = j * kRwBlocks + lane, b = tile.block(u);
            float4 s = make_float4(0.f, 0.f, 1.f, __int_as_float(kNoToken));
            if (u < tile.nb) {
              float k = pow2f(ke), v = pow2f(max(ve, unit - kUnitSpan) - unit);
              if (b < full) {
                k = ksc[b];
                v = fmaxf(vsc[b] * pow2f(-unit), pow2f(-kUnitSpan));
              }
              s = make_float4(k, log2f(v), 1.f / v, __int_as_float(b * kBlock));
            }
            scales[g & 3][lane] = s;
          }
          __syncwarp();
        }
        if (!rows_wait_warp(&sy.kempty[st], ((g >> 1) & 1) ^ 1, &abort_s)) break;
        unsigned char *const kt = area + 2 * kRwTile + st * kRwTile, *const vt = area + 4 * kRwTile + st * kRwTile;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          // a run's 16-byte chunks go to places 2 run and 2 run + 1, the second
          // half's in the other order: 8 lanes fill 8 places of a row at a time
          const int r = 32 * pw + 4 * t + kr_row;
          const uint4 w = kr_half ? make_uint4(kr[t].z, kr[t].w, kr[t].x, kr[t].y) : kr[t];
          uint32_t x[8];
          codes_row<CODE>(w.x, x[0], x[1]);
          codes_row<CODE>(w.y, x[2], x[3]);
          codes_row<CODE>(w.z, x[4], x[5]);
          codes_row<CODE>(w.w, x[6], x[7]);
          unsigned char *to = kt + kr_half * kRwHalf + r * 128;
          *(uint4 *)(to + (((2 * kr_run + kr_half) ^ (r & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
          *(uint4 *)(to + (((2 * kr_run + 1 - kr_half) ^ (r & 7)) << 4)) = make_uint4(x[4], x[5], x[6], x[7]);
        }
        if (j + 1 < s1) load_k(j + 1);
        const bool ends = tail && (j + 1) * kRwBlocks >= tile.nb;  // the step's last block is the partial one
        const int tail_at = (tile.nb - 1) % kRwBlocks * kBlock;
        if (ends) {
          __syncwarp();  // over the zeros of the rows' own warp
          if (pw == tail_at / 32) {
#pragma unroll 1
            for (int r = 0; r < tail_rows; ++r) {
              const int row = tail_at + r, d = 4 * lane;
              const uint2 x = *(const uint2 *)(tails[0] + r * kHeadDim + d);
              const uint32_t h0 = h2_bits(__floats2half2_rn(__uint_as_float(x.x << 16) * kf, __uint_as_float(x.x & 0xffff0000u) * kf));
              const uint32_t h1 = h2_bits(__floats2half2_rn(__uint_as_float(x.y << 16) * kf, __uint_as_float(x.y & 0xffff0000u) * kf));
              *(uint2 *)(kt + (d >> 6) * kRwHalf + row * 128 + ((((d & 63) >> 3) ^ (row & 7)) << 4) + (d & 7) * 2) = make_uint2(h0, h1);
            }
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          bar_arrive(&sy.kfull[st]);
          if (pw == 0) bar_arrive(&sy.scfull[g & 3]);
        }
        if (!rows_wait_warp(&sy.vempty[st], ((g >> 1) & 1) ^ 1, &abort_s)) break;
        {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = e == 0 ? vr[i].x : e == 1 ? vr[i].y : e == 2 ? vr[i].z : vr[i].w;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t x[4], y[4];  // d = 16 dc + 4 e + 2 h and the next: 8 tokens each
#pragma unroll
              for (int m = 0; m < 4; ++m) codes_across<CODE>(w[2 * m], w[2 * m + 1], h, x[m], y[m]);
              const int d = 16 * dc + 4 * e + 2 * h;
              unsigned char *to = vt + (tc >> 3) * kRwHalf + d * 128;
              *(uint4 *)(to + (((tc & 7) ^ (d & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
              *(uint4 *)(to + 128 + (((tc & 7) ^ ((d + 1) & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
            }
          }
        }
        if (j + 1 < s1) load_v(j + 1);
        if (ends && (tc >> 1) == tail_at / kBlock) {  // this thread's 8 tokens and 16 values of d
#pragma unroll 1
          for (int e = 0; e < 16; ++e) {
            const int d = 16 * dc + e, first = 8 * (tc & 1);
            uint32_t x[4];
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              const int row = first + 2 * m;
              const float lo = bf16_bits_to_f32(tails[1][row * kHeadDim + d]), hi = bf16_bits_to_f32(tails[1][(row + 1) * kHeadDim + d]);
              x[m] = h2_bits(__floats2half2_rn(lo * vf, hi * vf));
            }
            *(uint4 *)(vt + (tc >> 3) * kRwHalf + d * 128 + (((tc & 7) ^ (d & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) bar_arrive(&sy.vfull[st]);
      }
    } else if (warp == kRwIssuer) {
      // ---------------------------------------------------------------- products
      if (lane == 0) {
        auto qk = [&](int w, int st) {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const uint32_t at = (k >> 2) * kRwHalf + (k & 3) * 32;
            mma_ss(tmem + w * 128, rw_desc(q_at + w * kRwTile + at), rw_desc(k_at + st * kRwTile + at), k > 0);
          }
          mma_commit(&sy.sfull[w]);
        };
        // O += P V of a step's first and then second 64 tokens, each as soon as
        // its weights are there
        auto pv = [&](int w, int g) {
          const uint64_t y = rw_desc(v_at + (g & 1) * kRwTile);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (!rows_wait(&sy.pfull[w][h], g & 1, &abort_s)) return false;
            tmem_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_ts(tmem + 256 + w * 128, tmem + w * 128 + 32 * h + 8 * k, y + ((h * kRwHalf + k * 32) >> 4), g > done || h > 0 || k > 0);
            mma_commit(&sy.odone[w][h]);
          }
          return true;
        };
        bool ok = steps > 0 && rows_wait(&sy.kfull[done & 1], (done >> 1) & 1, &abort_s);
        if (ok) {
          tmem_after();
          qk(0, done & 1);
          if (two) qk(1, done & 1);
          mma_commit(&sy.kempty[done & 1]);
        }
        for (int g = done; ok && g < done + steps; ++g) {
          const int st = g & 1, nx = (g + 1) & 1;
          const bool more = g + 1 < done + steps;
          ok = rows_wait(&sy.vfull[st], (g >> 1) & 1, &abort_s) && pv(0, g);
          if (!ok) break;
          if (more) {
            ok = rows_wait(&sy.kfull[nx], ((g + 1) >> 1) & 1, &abort_s);
            if (!ok) break;
            tmem_after();
            qk(0, nx);
          }
          if (two) {
            ok = pv(1, g);
            if (!ok) break;
          }
          mma_commit(&sy.vempty[st]);
          if (more) {
            if (two) qk(1, nx);
            mma_commit(&sy.kempty[nx]);
          }
        }
      }
      __syncwarp();
    } else if (warp < 4 || two) {
      // ---------------------------------------------------------------- softmax
      const int w = warp >> 2;
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t s_at = tmem + lanes + w * 128, o_at = tmem + lanes + 256 + w * 128;
      const int q0 = r0 + w * kRwRows;
      const int pmin = tile.len - tile.cnt + q0 / a.group;
      const int pmax = tile.len - tile.cnt + min((min(q0 + kRwRows, R) - 1) / a.group, tile.cnt - 1);
      const int first = a.window > 0 ? pmax - a.window + 1 : 0, last = pmin - (kBlock - 1);  // of whole blocks that every row sees
      float ref = 0.f, l = 0.f, limit = valid ? -1.f : INFINITY;  // limit: of a block's sum of weights
      bool seen = !valid;
      bool ok = true;
      for (int g = done; ok && g < done + steps; ++g) {
        ok = rows_wait_warp(&sy.scfull[g & 3], (g >> 2) & 1, &abort_s);
        if (!ok) break;
        const bool open = __float_as_int(scales[g & 3][0].w) >= first && __float_as_int(scales[g & 3][kRwBlocks - 1].w) <= last;
        ok = rows_wait_warp(&sy.sfull[w], g & 1, &abort_s);
        if (!ok) break;
        tmem_after();
        float sum = 0.f;
        uint32_t r[32];
        tmem_ld32(s_at, r);
        // four blocks at a time, two by two: scores become weights, over the
        // columns of blocks that have been read
#pragma unroll 1
        for (int b = 0; b < kRwBlocks; b += 4) {
          uint32_t p[32];
          float t[4];
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const float4 sc0 = scales[g & 3][b + 2 * v], sc1 = scales[g & 3][b + 2 * v + 1];
            float y[32];
            tmem_wait32(r);
            {
              const float f0 = rc * sc0.x, at0 = sc0.y - ref, f1 = rc * sc1.x, at1 = sc1.y - ref;
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float f = e < 16 ? f0 : f1, at = e < 16 ? at0 : at1;
                const float2 z = fma_2(make_float2(__uint_as_float(r[e]), __uint_as_float(r[e + 1])), make_float2(f, f), make_float2(at, at));
                y[e] = z.x;
                y[e + 1] = z.y;
              }
            }
            if (v == 0 || b + 4 < kRwBlocks) tmem_ld32(s_at + 16 * (b + 2 * v + 2), r);
            if (!open) {
              int see[2][3];
#pragma unroll
              for (int k = 0; k < 2; ++k) token_range(__float_as_int(k ? sc1.w : sc0.w), pos, a.window, a.sinks, see[k]);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!sees(see[e >> 4], e & 15)) y[e] = -INFINITY;
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
            tmem_wait32(r);  // the scores on their way, before registers change hands
            const RowState z = move_reference(RowState{ref, l, sum, limit, seen}, s_at, o_at, scales[g & 3], rc, open, pos, a.window,
                                              a.sinks, b, g > done || b > 0, b > 0 ? &sy.odone[w][0] : nullptr, g & 1, &abort_s);
            ref = z.ref;
            l = z.l;
            sum = z.sum;
            limit = z.limit;
            seen = z.seen;
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) sum = __fmaf_rn(t[k], scales[g & 3][b + k].z, sum);
            tmem_st32(s_at + 8 * b, p);
          }
          tmem_wait_st();
          tmem_before();
          __syncwarp();
          if (lane == 0) bar_arrive(&sy.pfull[w][b >> 2]);
        }
        l += sum;
      }
      if (ok && steps > 0) ok = rows_wait_warp(&sy.odone[w][1], (done + steps - 1) & 1, &abort_s);
      tmem_after();
      const volatile Segment &at = seg;
      const int row = at.r0 + (int)threadIdx.x;
      if (!at.whole) {  // a part: O as it is (4 values of each row in turn), the exponents of its and l's units, and l
        float *slot = a.ws + (2 * (int64_t)blockIdx.x + (at.x == at.begin ? 0 : 1)) * kRwSlot;
        const int r = threadIdx.x;
        if (ok) {
#pragma unroll 1
          for (int d = 0; d < kHeadDim; d += 16) {
            uint32_t v[16];
            tmem_ld16(o_at + d, v);
            tmem_wait16(v);
#pragma unroll
            for (int e = 0; e < 16; e += 4) *(uint4 *)(slot + (d + e) * 2 * kRwRows + 4 * r) = make_uint4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          }
        }
        // (a row whose scores are all NaN has no reference, but l and O, which are NaN, count)
        const bool any = valid && seen;
        slot[2 * kRwRows * kHeadDim + r] = any ? ref + (float)unit : -INFINITY;
        slot[2 * kRwRows * (kHeadDim + 1) + r] = any ? ref : -INFINITY;
        slot[2 * kRwRows * (kHeadDim + 2) + r] = valid ? l : 0.f;
      } else {
        const float scale = valid && l != 0.f ? 1.f / l : 0.f, back = pow2f(unit);
        uint4 *out = (uint4 *)((uint16_t *)a.out + ((at.slice * a.group + row % a.group) * a.n + row / a.group) * kHeadDim);
#pragma unroll 1
        for (int d = 0; d < kHeadDim; d += 16) {
          uint32_t r[16];
          if (ok && steps > 0) {
            tmem_ld16(o_at + d, r);
            tmem_wait16(r);
          }
          float x[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) x[e] = scale != 0.f && steps > 0 ? __uint_as_float(r[e]) * scale * back : 0.f;
          if (row < R) {
            out[d / 8] = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
            out[d / 8 + 1] = make_uint4(pack_bf16(x[8], x[9]), pack_bf16(x[10], x[11]), pack_bf16(x[12], x[13]), pack_bf16(x[14], x[15]));
          }
        }
      }
    } else {
      // no row of the second tile is a token: its outputs are zeros
      const int row = r0 + (int)threadIdx.x;
      if (row < R) {
        uint4 *out = (uint4 *)((uint16_t *)a.out + ((slice * a.group + row % a.group) * a.n + row / a.group) * kHeadDim);
#pragma unroll 1
        for (int d = 0; d < kHeadDim / 8; ++d) out[d] = make_uint4(0, 0, 0, 0);
      }
    }
    // the next tile's queries, scales and scores go over this one's
    tmem_before();
    __syncthreads();
    tmem_after();
    if (!STREAMED || abort_s) break;
    if (threadIdx.x == 0) {
      seg.x += seg.units;
      seg.done += seg.s1 - seg.s0;
    }
    __syncthreads();
  }
  if (warp == kRwIssuer) {
    if (lane == 0) {  // every product has completed before the tensor memory is freed
      mma_commit(&sy.drained);
      bar_wait(&sy.drained, 0);
    }
    __syncwarp();
    tmem_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_s), "r"(512) : "memory");
  }
  if (threadIdx.x == 0 && abort_s) atomicOr(c.ticket + c.batch, kAnomTimeout);
}

// Joins the parts of the tiles that several CTAs of a streamed launch share:
// blockIdx.x the CTA with the first part, kRwMergeRows rows a CTA, a thread 4
// values of one at d and 4 at d + 64.
constexpr int kRwMergeRows = 16;
__global__ void __launch_bounds__(256) k_attend8_rows_merge(const __grid_constant__ AttendArgs a) {
  const int first = blockIdx.x;
  wait_prerequisites();  // by every CTA: this kernel's end stands for the first one's
  const RowsJoin join = *(const RowsJoin *)(a.ws + 2 * (int64_t)gridDim.x * kRwSlot + first * (sizeof(RowsJoin) / 4));
  if (join.parts <= 1) return;
  const int np = join.parts, b = join.slice / a.c.n_kv_heads;
  const int cnt = a.counts ? min(max(a.counts[b], 0), a.n) : a.n;
  auto slot = [&](int j) { return a.ws + (2 * (int64_t)(first + j) + (j == 0 ? join.second : 0)) * kRwSlot; };
  const int r = blockIdx.y * kRwMergeRows + threadIdx.x % kRwMergeRows, d = 4 * (threadIdx.x / kRwMergeRows);
  const int row = join.row_tile * 2 * kRwRows + r, i = row / a.group;
  if (row >= a.n * a.group) return;
  float top = -INFINITY, topt = -INFINITY, l = 0.f, o[8] = {};
#pragma unroll 4
  for (int j = 0; j < np; ++j) {
    const float *p = slot(j) + 2 * kRwRows * kHeadDim + r;
    top = fmaxf(top, p[0]);
    topt = fmaxf(topt, p[2 * kRwRows]);
  }
#pragma unroll 4
  for (int j = 0; j < np; ++j) {
    const float *p = slot(j) + 2 * kRwRows * kHeadDim + r;
    const float f = share(p[0], top);
    l += share(p[2 * kRwRows], topt) * p[4 * kRwRows];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float4 v = *(const float4 *)(slot(j) + (d + 64 * k) * 2 * kRwRows + 4 * r);
      o[4 * k] += f * v.x;
      o[4 * k + 1] += f * v.y;
      o[4 * k + 2] += f * v.z;
      o[4 * k + 3] += f * v.w;
    }
  }
  const bool none = i >= cnt || l == 0.f;
  const float scale = none ? 0.f : 1.f / l, back = none ? 0.f : exp2f(top - topt);
  uint16_t *out = (uint16_t *)a.out + (((int64_t)join.slice * a.group + row % a.group) * a.n + i) * kHeadDim + d;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = none ? 0.f : o[4 * k + e] * scale * back;
    *(uint2 *)(out + 64 * k) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
  }
}

// A call's time in steps of one CTA (2.1 us on a GB300), and how it is split:
// a CTA a tile, or streamed where that ends sooner. A CTA a tile takes as long
// as its waves of equal tiles, or, where later rows see much more than earlier
// ones (those start first), the mean share and a short tile. A streamed launch
// shares the steps out evenly, for 6% slower ones and what a second beginning,
// storing parts and joining them cost: 14 steps. Measured, int8, 4 query heads
// a KV head, a CTA a tile and streamed: 2048 tokens over 32K, 8 KV heads (256
// tiles) 1131 and 1030 us, 4 KV heads 586 and 541; 64 tokens over 32K, 64
// slices 575 and 300, 8 slices 564 and 78; 2048 over 4K, 4 KV heads 96 and 115;
// 256 slices of a window of 1024, 64 tokens 111 and 145.
double rows_plan(const lkv_cache8 &c, int64_t rows, int64_t tokens, int64_t steps, int sms, int *ctas) {
  const int64_t row_tiles = (rows + 2 * kRwRows - 1) / (2 * kRwRows), tiles = (int64_t)c.batch * c.n_kv_heads * row_tiles;
  const int64_t fewer = tokens / kRwTok < steps ? tokens / kRwTok : steps - 1;  // steps of the first rows' tiles than of the last's
  const double share = (double)tiles * (kRwStart + steps - 0.5 * fewer) / sms, one = kRwStart + steps;
  const double waves = (double)((tiles + sms - 1) / sms) * one, packed = share + (one - fewer);
  const double least = waves < packed ? waves : packed, whole = least > one ? least : one, streamed = 1.06 * share + 14;
  *ctas = 0;
  if (streamed >= whole || c.batch * row_tiles > kAtGroups) return whole;
  *ctas = (int)(steps * tiles < sms ? steps * tiles : sms);
  return streamed;
}

int64_t rows_bytes(int ctas) { return ctas * (2 * kRwSlot * 4 + (int64_t)sizeof(RowsJoin)); }

cudaError_t launch_attend_rows(const AttendArgs &in, int ctas, cudaStream_t st) {
  AttendArgs a = in;
  const int64_t R = (int64_t)a.n * a.group, S = (int64_t)a.c.batch * a.c.n_kv_heads;
  a.row_tiles = (int32_t)((R + 2 * kRwRows - 1) / (2 * kRwRows));
  a.streamed = ctas > 0;
  const int64_t tiles = S * a.row_tiles;
  if (tiles > 0x7fffffff) return cudaErrorInvalidValue;
  auto *fn = a.c.code == LKV_CODE_INT8 ? (ctas ? k_attend8_rows<LKV_CODE_INT8, true> : k_attend8_rows<LKV_CODE_INT8, false>)
                                       : (ctas ? k_attend8_rows<LKV_CODE_E4M3, true> : k_attend8_rows<LKV_CODE_E4M3, false>);
  cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRwSmem);
  if (e != cudaSuccess) return e;
  e = launch_next(fn, dim3((unsigned)(ctas ? ctas : tiles)), kRwThreads, kRwSmem, st, a);
  if (e != cudaSuccess || !ctas) return e;
  return launch_next(k_attend8_rows_merge, dim3((unsigned)ctas, 2 * kRwRows / kRwMergeRows), 256, 0, st, a);
}

}  // namespace lkv
