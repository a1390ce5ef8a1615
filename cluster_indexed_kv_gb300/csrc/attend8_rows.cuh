// attend8_rows.cuh -- attention of many rows over the 8-bit cache on tcgen05: what
// the kernels of lkv_cache8_attend and lkv_cache8_attend_shared share.
#pragma once

#include "attend8.cuh"

namespace lkv {

constexpr int kRwTok = kRowsStep;                // tokens of a K / V tile
constexpr int kRwBlocks = kRwTok / kBlock;
constexpr int kRwRows = kRowsTile / 2;           // rows of a row tile
constexpr int kRwProducer = 8;                   // first producer warp
constexpr int kRwIssuer = 12;                    // the issuing warp
constexpr int kRwThreads = 13 * 32;
constexpr uint32_t kRwTile = kRwTok * kHeadDim * 2;  // 32 KB: two 64-column halves of 16 KB
constexpr uint32_t kRwHalf = kRwTile / 2;
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
__device__ __forceinline__ bool rows_wait(uint64_t *bar, uint32_t phase, volatile int *abort, uint64_t limit = kCopyLimitNs) {
  if (bar_try(bar, phase)) return true;
  uint64_t t0, t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
  while (!bar_try(bar, phase)) {
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    if (*abort || t - t0 > limit) {
      *abort = 1;
      return false;
    }
  }
  return true;
}
// The same for a whole warp, uniformly.
__device__ __forceinline__ bool rows_wait_warp(uint64_t *bar, uint32_t phase, volatile int *abort, uint64_t limit = kCopyLimitNs) {
  return __all_sync(0xffffffffu, rows_wait(bar, phase, abort, limit));
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
static __device__ __noinline__ RowState move_reference(RowState z, uint32_t s_at, uint32_t o_at, const float4 *scale, float rc, bool open, int pos,
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

}  // namespace lkv
