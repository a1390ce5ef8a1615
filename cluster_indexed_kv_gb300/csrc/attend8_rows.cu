// attend8_rows.cu -- causal attention of many rows over the 8-bit cache
// (lkv_cache8_attend for prompts and chunks of bf16 caches) on tcgen05.
#include "attend8.cuh"

namespace lkv {

// A CTA takes 256 rows (token-major, as in k_attend8) of one (sequence, KV
// head), as two tiles of 128, and walks their visible blocks 128 tokens (8
// blocks) at a time:
//   - 4 producer warps turn codes into fp16 tiles (exact), K token-major and V
//     transposed, both K-major with 128-byte swizzle; the next tile's codes
//     are in registers meanwhile;
//   - one thread issues the products: S = Q K^T (fp16, fp32 in tensor memory)
//     and O += P V with P read from tensor memory;
//   - 4 warps a row tile, a thread a row, take S to weights P (fp16, over S's
//     columns). While they work on one row tile, the tensor cores work on the
//     other's P V and next S.
// The weights are those of k_attend8: y = score + log2(u), u the V scale of
// the block in units of the largest visible one, w = 2^(y - reference), out =
// sum w code / sum w / u; a row's reference moves only when a y passes it by
// 2^8, so O is hardly ever touched between products.
//
// Bound: the exponentials (16 a clock and SM) and the products take the same
// 2048 clocks for 256 rows x 128 tokens.
constexpr int kRwTok = 128;                      // tokens of a K / V tile
constexpr int kRwBlocks = kRwTok / kBlock;
constexpr int kRwRows = 128;                     // rows of a row tile
constexpr int kRwProducer = 8;                   // first producer warp
constexpr int kRwIssuer = 12;                    // the issuing warp
constexpr int kRwThreads = 13 * 32;
constexpr uint32_t kRwTile = kRwTok * kHeadDim * 2;  // 32 KB: two 64-column halves of 16 KB
constexpr uint32_t kRwHalf = kRwTile / 2;
constexpr uint32_t kRwSmem = 6 * kRwTile + 1024;     // Q: 2, K: 2, V: 2
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
// 8 columns, waited for.
__device__ __forceinline__ void tmem_ld8(uint32_t at, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\ttcgen05.wait::ld.sync.aligned;"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t at, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
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
__device__ __forceinline__ void tmem_st4(uint32_t at, const uint32_t (&r)[4]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
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
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], odone[2], scfull[4], drained;
  uint64_t pfull[2][2];  // [row tile][half of the tokens]
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

// Which tokens of block unit u a row at position pos sees: those up to
// see[0], and of them those above see[1] or below see[2].
__device__ __forceinline__ void token_range(int u, int sb, int lo, int nb, int pos, int window, int sinks, int (&see)[3]) {
  const int tok = (u < sb ? u : u - sb + lo) * kBlock;
  see[0] = u < nb ? pos - tok : -1;
  see[1] = window > 0 ? pos - window - tok : -1;
  see[2] = sinks - tok;
}
__device__ __forceinline__ bool sees(const int (&see)[3], int i) { return i <= see[0] && (i > see[1] || i < see[2]); }

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
__device__ __noinline__ RowState move_reference(RowState z, uint32_t s_at, uint32_t o_at, const float4 *scale, float rc, bool open, int u0, int sb,
                                                int lo, int nb, int pos, int window, int sinks, int b, bool has_o, uint64_t *odone,
                                                volatile int *abort) {
  float far = -INFINITY;
  auto scores = [&](int c, uint32_t(&x)[8]) {  // y of columns 8 c.. of the four blocks
    tmem_ld8(s_at + 16 * b + 8 * c, x);
    const float4 sc = scale[b + (c >> 1)];
    const float f = rc * sc.x, at = sc.y - z.ref;
    int see[3];
    token_range(u0 + b + (c >> 1), sb, lo, nb, pos, window, sinks, see);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float v = __fmaf_rn(__uint_as_float(x[e]), f, at);
      x[e] = __float_as_uint(open || sees(see, 8 * (c & 1) + e) ? v : -INFINITY);
    }
  };
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {
    uint32_t x[8];
    scores(c, x);
#pragma unroll
    for (int e = 0; e < 8; ++e) far = fmaxf(far, __uint_as_float(x[e]));
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
    if (odone) rows_wait_warp(odone, 0, abort);
    if (has_o) {
      tmem_after();
#pragma unroll 1
      for (int d = 0; d < kHeadDim; d += 8) {
        uint32_t x[8];
        tmem_ld8(o_at + d, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * k);
        tmem_st8(o_at + d, x);
      }
      tmem_wait_st();
    }
  }
#pragma unroll 1
  for (int c = 0; c < 8; ++c) {  // weights over columns whose scores have been read: 4 c.. behind 8 c..
    uint32_t x[8], p[4];
    scores(c, x);
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = ex2(__uint_as_float(x[e]));
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = h2_bits(__floats2half2_rn(w[2 * e], w[2 * e + 1]));
    z.sum = __fmaf_rn(((w[0] + w[1]) + (w[2] + w[3])) + ((w[4] + w[5]) + (w[6] + w[7])), scale[b + (c >> 1)].z, z.sum);
    tmem_st4(s_at + 8 * b + 4 * c, p);
  }
  return z;
}

template <int CODE>
__global__ void __launch_bounds__(kRwThreads, 1) k_attend8_rows(const __grid_constant__ AttendArgs a) {
  extern __shared__ unsigned char raw[];
  __shared__ __align__(8) RowsSync sy;
  __shared__ float4 scales[4][kRwBlocks];  // K scale, log2 and reciprocal of the V scale's share of the unit
  __shared__ uint32_t tmem_s;
  __shared__ volatile int abort_s;
  __shared__ uint32_t top_s;               // largest V scale of the visible blocks (bits)
  __shared__ int tail_s[2];                // exponents of the tails
  const lkv_cache8 &c = a.c;
  const uint32_t base = (smem_at(raw) + 1023u) & ~1023u;
  unsigned char *const area = raw + (base - smem_at(raw));
  const uint32_t q_at = base, k_at = base + 2 * kRwTile, v_at = base + 4 * kRwTile;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t S = (int64_t)c.batch * c.n_kv_heads, slice = blockIdx.x % S;
  const int rt = a.row_tiles - 1 - (int)(blockIdx.x / S);  // the rows with most to see come first
  const Tile tile(a, (int)(slice / c.n_kv_heads), rt, 2 * kRwRows);
  const int R = a.n * a.group, r0 = rt * 2 * kRwRows;
  const int steps = (tile.nb + kRwBlocks - 1) / kRwBlocks;
  const bool two = r0 + kRwRows < R && (r0 + kRwRows) / a.group < tile.cnt;  // the second row tile has rows
  const int full = tile.len / kBlock;   // blocks before it are quantised
  const bool tail = tile.hi >= full && tile.nb > 0;
  const uint16_t *const k_tail = (const uint16_t *)c.k_tail + slice * kBlock * kHeadDim;
  const uint16_t *const v_tail = (const uint16_t *)c.v_tail + slice * kBlock * kHeadDim;
  const int tail_rows = tile.len - full * kBlock;
  const float *const ksc = c.k_scale + slice * (c.capacity / kBlock), *const vsc = c.v_scale + slice * (c.capacity / kBlock);

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      bar_init(&sy.kfull[i], 4);
      bar_init(&sy.kempty[i], 1);
      bar_init(&sy.vfull[i], 4);
      bar_init(&sy.vempty[i], 1);
      bar_init(&sy.sfull[i], 1);
      bar_init(&sy.pfull[i][0], 4);
      bar_init(&sy.pfull[i][1], 4);
      bar_init(&sy.odone[i], 1);
    }
    for (int i = 0; i < 4; ++i) bar_init(&sy.scfull[i], 1);
    bar_init(&sy.drained, 1);
    bar_init_fence();
    abort_s = 0;
    top_s = 0;
    tail_s[0] = tail_s[1] = -126;
  }
  if (warp == kRwIssuer) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_at(&tmem_s)), "r"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  __syncthreads();

  // the unit of the V scales, and the tails' exponents
  {
    uint32_t top = 0;
    for (int u = threadIdx.x; u < tile.nb; u += kRwThreads) {
      const int b = tile.block(u);
      if (b < full) top = max(top, __float_as_uint(vsc[b]));
    }
    top = __reduce_max_sync(0xffffffffu, top);
    if (lane == 0 && top) atomicMax(&top_s, top);
    if (tail && (warp == kRwProducer || warp == kRwProducer + 1)) {
      const uint16_t *t = warp == kRwProducer ? k_tail : v_tail;
      float m = 0.f;
      for (int r = 0; r < tail_rows; ++r) {
        const uint2 w = *(const uint2 *)(t + r * kHeadDim + 4 * lane);
        m = fmaxf(m, fmaxf(fmaxf(fabsf(__uint_as_float(w.x << 16)), fabsf(__uint_as_float(w.x & 0xffff0000u))),
                           fmaxf(fabsf(__uint_as_float(w.y << 16)), fabsf(__uint_as_float(w.y & 0xffff0000u)))));
      }
      const uint32_t e = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
      if (lane == 0) tail_s[warp - kRwProducer] = min(max((int)(e >> 23) - 126, -100), 126);
    }
  }

  // a thread a row: its query as fp16 in units of a power of two, into the swizzled tile
  float rc = 0.f;
  int pos = -1;
  bool valid = false;
  if (warp < kRwProducer) {
    const int row = r0 + (int)threadIdx.x, i = row / a.group, rr = threadIdx.x & (kRwRows - 1);
    valid = row < R && i < tile.cnt;
    if (valid) pos = tile.len - tile.cnt + i;
    const uint4 *p = (const uint4 *)((const uint16_t *)a.q + ((slice * a.group + (valid ? row % a.group : 0)) * a.n + (valid ? i : 0)) * kHeadDim);
    uint32_t m = 0;
#pragma unroll 4
    for (int u = 0; u < 16; ++u) {
      const uint4 w = valid ? p[u] : make_uint4(0, 0, 0, 0);
      m = __vmaxu2(m, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
    }
    m = max(m << 16, m & 0xffff0000u);
    const int e = min(max((int)(m >> 23) - 126, -100), 126);
    const float f = pow2f(-e);
    rc = pow2f(e) * a.scale_log2;
    unsigned char *to = area + (threadIdx.x / kRwRows) * kRwTile + rr * 128;
#pragma unroll 4
    for (int u = 0; u < 16; ++u) {
      const uint4 w = valid ? p[u] : make_uint4(0, 0, 0, 0);
      const uint32_t x[4] = {w.x, w.y, w.z, w.w};
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        h[k] = h2_bits(__floats2half2_rn(__uint_as_float(x[k] << 16) * f, __uint_as_float(x[k] & 0xffff0000u) * f));
      *(uint4 *)(to + (u >> 3) * kRwHalf + (((u & 7) ^ (rr & 7)) << 4)) = make_uint4(h[0], h[1], h[2], h[3]);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  }
  tmem_before();
  __syncthreads();
  tmem_after();
  const uint32_t tmem = tmem_s;
  const int ve = tail_s[1];
  const int unit = max(max((int)(top_s >> 23) - 127, -126), tail ? ve : -126);  // V scales count in units of 2^unit

  if (warp >= kRwProducer && warp < kRwIssuer) {
    // ---------------------------------------------------------------- producers
    const int pw = warp - kRwProducer, pt = pw * 32 + lane;
    const uint8_t *kc = (const uint8_t *)c.k_codes + slice * c.capacity * kHeadDim;
    const uint8_t *vc = (const uint8_t *)c.v_codes + slice * c.capacity * kHeadDim;
    const int ks_row = lane >> 2, ks_j = lane & 3;      // K: 8 rows x 4 runs of 16 a load
    const int tc = pt & 15, dc = pt >> 4;               // V: tokens 8 tc.., d 16 dc..
    const float kf = pow2f(-tail_s[0]), vf = pow2f(-max(ve, unit - kUnitSpan));
    uint4 kr[8], vr[8];
    auto load_k = [&](int j) {
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int u = j * kRwBlocks + 2 * pw + (it >> 1), b = tile.block(u);
        const bool there = u < tile.nb && b < full;
        const uint8_t *p = kc + ((int64_t)b * kBlock + 8 * (it & 1) + ks_row) * kHeadDim + 16 * ks_j;
#pragma unroll
        for (int h = 0; h < 2; ++h) kr[2 * it + h] = there ? __ldg((const uint4 *)(p + 64 * h)) : make_uint4(0, 0, 0, 0);
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
      load_k(0);
      load_v(0);
    }
    for (int j = 0; j < steps; ++j) {
      const int st = j & 1;
      // the blocks' scales
      if (pw == 0) {
        if (lane < kRwBlocks) {
          const int u = j * kRwBlocks + lane, b = tile.block(u);
          float4 s = make_float4(0.f, 0.f, 1.f, 0.f);
          if (u < tile.nb) {
            float k = pow2f(tail_s[0]), v = pow2f(max(ve, unit - kUnitSpan) - unit);
            if (b < full) {
              k = ksc[b];
              v = vsc[b];
              v = v > 0.f ? fmaxf(v * pow2f(-unit), pow2f(-kUnitSpan)) : 1.f;
            }
            s = make_float4(k, log2f(v), 1.f / v, 0.f);
          }
          scales[j & 3][lane] = s;
        }
        __syncwarp();
      }
      if (!rows_wait_warp(&sy.kempty[st], ((j >> 1) & 1) ^ 1, &abort_s)) break;
      unsigned char *const kt = area + 2 * kRwTile + st * kRwTile, *const vt = area + 4 * kRwTile + st * kRwTile;
#pragma unroll
      for (int it = 0; it < 4; ++it) {
        const int r = 32 * pw + 8 * it + ks_row;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 w = kr[2 * it + h];
          uint32_t x[8];
          codes_row<CODE>(w.x, x[0], x[1]);
          codes_row<CODE>(w.y, x[2], x[3]);
          codes_row<CODE>(w.z, x[4], x[5]);
          codes_row<CODE>(w.w, x[6], x[7]);
          unsigned char *to = kt + h * kRwHalf + r * 128;
          *(uint4 *)(to + (((2 * ks_j) ^ (r & 7)) << 4)) = make_uint4(x[0], x[1], x[2], x[3]);
          *(uint4 *)(to + (((2 * ks_j + 1) ^ (r & 7)) << 4)) = make_uint4(x[4], x[5], x[6], x[7]);
        }
      }
      if (j + 1 < steps) load_k(j + 1);
      const bool ends = tail && j + 1 == steps;  // the tile's last block is the partial one
      const int tail_at = (tile.nb - 1) % kRwBlocks * kBlock;
      if (ends) {
        __syncwarp();  // over the zeros of the rows' own warp
        if (pw == tail_at / 32) {
#pragma unroll 1
          for (int r = 0; r < tail_rows; ++r) {
            const int row = tail_at + r, d = 4 * lane;
            const uint2 x = *(const uint2 *)(k_tail + r * kHeadDim + d);
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
        if (pw == 0) bar_arrive(&sy.scfull[j & 3]);
      }
      if (!rows_wait_warp(&sy.vempty[st], ((j >> 1) & 1) ^ 1, &abort_s)) break;
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
      if (j + 1 < steps) load_v(j + 1);
      if (ends && (tc >> 1) == tail_at / kBlock) {  // this thread's 8 tokens and 16 values of d
#pragma unroll 1
        for (int e = 0; e < 16; ++e) {
          const int d = 16 * dc + e, first = 8 * (tc & 1);
          uint32_t x[4];
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int row = first + 2 * m;
            const float lo = row < tail_rows ? bf16_bits_to_f32(v_tail[row * kHeadDim + d]) : 0.f;
            const float hi = row + 1 < tail_rows ? bf16_bits_to_f32(v_tail[(row + 1) * kHeadDim + d]) : 0.f;
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
      auto pv = [&](int w, int j) {
        const uint64_t y = rw_desc(v_at + (j & 1) * kRwTile);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!rows_wait(&sy.pfull[w][h], j & 1, &abort_s)) return false;
          tmem_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ts(tmem + 256 + w * 128, tmem + w * 128 + 32 * h + 8 * k, y + ((h * kRwHalf + k * 32) >> 4), j > 0 || h > 0 || k > 0);
          mma_commit(&sy.odone[w]);
        }
        return true;
      };
      bool ok = steps > 0 && rows_wait(&sy.kfull[0], 0, &abort_s);
      if (ok) {
        tmem_after();
        qk(0, 0);
        if (two) qk(1, 0);
        mma_commit(&sy.kempty[0]);
      }
      for (int j = 0; ok && j < steps; ++j) {
        const int st = j & 1, nx = (j + 1) & 1;
        ok = rows_wait(&sy.vfull[st], (j >> 1) & 1, &abort_s) && pv(0, j);
        if (!ok) break;
        if (j + 1 < steps) {
          ok = rows_wait(&sy.kfull[nx], ((j + 1) >> 1) & 1, &abort_s);
          if (!ok) break;
          tmem_after();
          qk(0, nx);
        }
        if (two) {
          ok = pv(1, j);
          if (!ok) break;
        }
        mma_commit(&sy.vempty[st]);
        if (j + 1 < steps) {
          if (two) qk(1, nx);
          mma_commit(&sy.kempty[nx]);
        }
      }
      // every product has completed before the tensor memory is freed
      mma_commit(&sy.drained);
      bar_wait(&sy.drained, 0);
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
    const int open0 = a.window > 0 ? max(0, pmax - a.window + kBlock) / kBlock : 0, open1 = (pmin + 1) / kBlock;
    float ref = 0.f, l = 0.f, limit = valid ? -1.f : INFINITY;  // limit: of a block's sum of weights
    bool seen = !valid;
    bool ok = true;
    for (int j = 0; ok && j < steps; ++j) {
      ok = rows_wait_warp(&sy.scfull[j & 3], (j >> 2) & 1, &abort_s) && rows_wait_warp(&sy.sfull[w], j & 1, &abort_s);
      if (!ok) break;
      tmem_after();
      // units of the tile that every row sees as a whole
      const int u0 = j * kRwBlocks, b_first = tile.block(u0), b_last = tile.block(u0 + kRwBlocks - 1);
      const bool open = u0 + kRwBlocks <= tile.nb && b_first >= open0 && b_last < open1;
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
        for (int g = 0; g < 2; ++g) {
          const float4 sc0 = scales[j & 3][b + 2 * g], sc1 = scales[j & 3][b + 2 * g + 1];
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
          if (g == 0 || b + 4 < kRwBlocks) tmem_ld32(s_at + 16 * (b + 2 * g + 2), r);
          if (!open) {
            int see[2][3];
#pragma unroll
            for (int k = 0; k < 2; ++k) token_range(u0 + b + 2 * g + k, tile.sb, tile.lo, tile.nb, pos, a.window, a.sinks, see[k]);
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
            for (int e = 0; e < 4; ++e) p[16 * g + 4 * k + e] = h2_bits(__floats2half2_rn(y[8 * k + 2 * e], y[8 * k + 2 * e + 1]));
          }
          z[0] = add_2(z[0], z[1]);
          z[2] = add_2(z[2], z[3]);
          t[2 * g] = z[0].x + z[0].y;
          t[2 * g + 1] = z[2].x + z[2].y;
        }
        // a weight is at most its block's sum: below the limit none leaves fp16's range
        if (__any_sync(0xffffffffu, !(fmaxf(fmaxf(t[0], t[1]), fmaxf(t[2], t[3])) <= limit))) {
          tmem_wait32(r);  // the scores on their way, before registers change hands
          const RowState z = move_reference(RowState{ref, l, sum, limit, seen}, s_at, o_at, scales[j & 3], rc, open, u0, tile.sb, tile.lo, tile.nb,
                                            pos, a.window, a.sinks, b, j > 0 || b > 0, b > 0 ? &sy.odone[w] : nullptr, &abort_s);
          ref = z.ref;
          l = z.l;
          sum = z.sum;
          limit = z.limit;
          seen = z.seen;
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) sum = __fmaf_rn(t[k], scales[j & 3][b + k].z, sum);
          tmem_st32(s_at + 8 * b, p);
        }
        tmem_wait_st();
        tmem_before();
        __syncwarp();
        if (lane == 0) bar_arrive(&sy.pfull[w][b >> 2]);
      }
      l += sum;
    }
    // the last two products into O (scores follow all products before them)
    if (ok && steps > 0) ok = rows_wait_warp(&sy.odone[w], 0, &abort_s) && rows_wait_warp(&sy.odone[w], 1, &abort_s);
    tmem_after();
    const int row = r0 + (int)threadIdx.x;
    const float scale = valid && l != 0.f ? 1.f / l : 0.f, back = pow2f(unit);
    uint4 *out = (uint4 *)((uint16_t *)a.out + ((slice * a.group + row % a.group) * a.n + row / a.group) * kHeadDim);
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
  } else {
    // no row of the second tile is a token: its outputs are zeros
    const int row = r0 + (int)threadIdx.x;
    if (row < R) {
      uint4 *out = (uint4 *)((uint16_t *)a.out + ((slice * a.group + row % a.group) * a.n + row / a.group) * kHeadDim);
#pragma unroll 1
      for (int d = 0; d < kHeadDim / 8; ++d) out[d] = make_uint4(0, 0, 0, 0);
    }
  }
  tmem_before();
  __syncthreads();
  if (warp == kRwIssuer) {
    tmem_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
  if (threadIdx.x == 0 && abort_s) atomicOr(c.ticket + c.batch, kAnomTimeout);
}

cudaError_t launch_attend_rows(const AttendArgs &in, cudaStream_t st) {
  AttendArgs a = in;
  const int64_t R = (int64_t)a.n * a.group, S = (int64_t)a.c.batch * a.c.n_kv_heads;
  a.row_tiles = (int32_t)((R + 2 * kRwRows - 1) / (2 * kRwRows));
  const int64_t grid = S * a.row_tiles;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  auto *fn = a.c.code == LKV_CODE_INT8 ? k_attend8_rows<LKV_CODE_INT8> : k_attend8_rows<LKV_CODE_E4M3>;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kRwSmem);
  if (e != cudaSuccess) return e;
  fn<<<(unsigned)grid, kRwThreads, kRwSmem, st>>>(a);
  return cudaGetLastError();
}

}  // namespace lkv
