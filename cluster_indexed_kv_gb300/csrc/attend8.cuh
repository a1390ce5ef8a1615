// attend8.cuh -- what the kernels of the attention over the 8-bit cache share.
#pragma once

#include <cuda_fp16.h>

#include "cache8.cuh"
#include "tma.cuh"

namespace lkv {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kPShift = 6.f;
constexpr float kSlack = 8.f;
constexpr int kNoUnit = -1000;
// V scales below 2^-90 of the largest are taken for that, 0 among them (a scale
// of 0 may stand over codes that are not: those of values too small for it).
constexpr int kUnitSpan = 90;

struct AttendArgs {
  lkv_cache8 c;
  const void *q;
  void *out;
  const int32_t *counts;
  int32_t n, group, window, sinks;
  int32_t row_tiles;
  int32_t streamed;   // the CTAs share all tiles' blocks evenly (see k_attend8)
  float *ws;          // streamed: 2 partials a CTA
  float scale_log2;   // scale * log2(e)
};

__device__ __forceinline__ uint32_t h2_bits(__half2 h) { return *(const uint32_t *)&h; }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

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

// Bytes 2 h and 2 h + 1 of two tokens' words as two fp16 (or bf16) pairs across
// the tokens: exact in either.
template <int CODE, bool BF16 = false>
__device__ __forceinline__ void codes_across(uint32_t wa, uint32_t wb, int h, uint32_t &even, uint32_t &odd) {
  if constexpr (CODE == LKV_CODE_INT8 && BF16) {
    // 0x4300 | x is 128 + x in bf16 for x below 128, and 256 for the sign bit alone
    const uint32_t u = __byte_perm(wa, wb, h ? 0x7632 : 0x5410);
    auto pair = [](uint32_t w) {
      const uint32_t low = w & 0xff7fff7fu, off = w & 0xff80ff80u;
      const __nv_bfloat162 d = __hsub2(*(const __nv_bfloat162 *)&low, *(const __nv_bfloat162 *)&off);
      return *(const uint32_t *)&d;
    };
    even = pair(__byte_perm(u, 0x43434343u, 0x4240));
    odd = pair(__byte_perm(u, 0x43434343u, 0x4341));
  } else if constexpr (CODE == LKV_CODE_INT8) {
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
    if constexpr (BF16) {
      const float2 e2 = __half22float2(*(const __half2 *)&even), o2 = __half22float2(*(const __half2 *)&odd);
      even = pack_bf16(e2.x, e2.y);
      odd = pack_bf16(o2.x, o2.y);
    }
  }
}

// The rows of a tile (one row tile of one sequence's KV head) and the blocks they see:
// the first `sb` (sinks), then lo..hi.
struct Tile {
  int len, cnt, pmin, pmax, lo, hi, sb, nb;
  Tile() = default;
  __device__ __forceinline__ Tile(const AttendArgs &a, int b, int rt, int RT) {
    len = min(max(__ldcg(a.c.lengths + b), 0), a.c.capacity);
    cnt = a.counts ? min(max(__ldcg(a.counts + b), 0), a.n) : a.n;
    const int R = a.n * a.group, r0 = rt * RT;
    const int imin = r0 / a.group, imax = min((min(r0 + RT, R) - 1) / a.group, cnt - 1);
    pmin = len - cnt + imin;
    pmax = imin <= imax ? len - cnt + imax : -1;
    lo = a.window > 0 ? max(0, pmin - a.window + 1) / kBlock : 0;
    hi = pmax >= 0 ? pmax / kBlock : -1;
    sb = a.window > 0 && hi >= 0 ? min((min(a.sinks, len) + kBlock - 1) / kBlock, lo) : 0;
    nb = hi >= 0 ? sb + hi - lo + 1 : 0;
  }
  __device__ __forceinline__ int block(int u) const { return u < sb ? u : u - sb + lo; }
};

// Which of a block's tokens (the first is token `tok`) a row at position pos
// sees: those up to see[0], and of them those above see[1] or below see[2].
// Nothing overflows for pos >= -1 and windows below and sinks up to a capacity of 2^30;
// kNoToken, of a block that is not there, lies behind every position.
constexpr int kNoToken = 1 << 30;
__host__ __device__ __forceinline__ void token_range(int tok, int pos, int window, int sinks, int (&see)[3]) {
  see[0] = pos - tok;
  see[1] = window > 0 ? see[0] - window : -1;
  see[2] = sinks - tok;
}
__host__ __device__ __forceinline__ bool sees(const int (&see)[3], int i) { return i <= see[0] && (i > see[1] || i < see[2]); }

constexpr int kAtGroups = 512;  // (sequence, row tile) pairs that a streamed launch takes

// A streamed launch's work: the units (runs of `per` blocks, behind `start`
// units that stand for what beginning a tile costs) of all tiles in a row, (sequence, row tile) by (sequence, row tile) and KV head by KV head, CTA
// i of P taking those from total * i / P on (P the CTAs, but no more than units).
struct Stream {
  int64_t at[kAtGroups + 1];  // units before each (sequence, row tile)
  int nu[kAtGroups];          // units of one of its tiles
  __device__ void fill(const AttendArgs &a, int RT, int per, int start) {
    const int G = a.c.batch * a.row_tiles;
    for (int i = threadIdx.x; i < G; i += blockDim.x) nu[i] = start + (Tile(a, i % a.c.batch, i / a.c.batch, RT).nb + per - 1) / per;
    __syncthreads();
    if (threadIdx.x < 32) {
      int64_t sum = 0;
      for (int i0 = 0; i0 < G; i0 += 32) {
        const int i = i0 + threadIdx.x;
        int64_t x = i < G ? (int64_t)nu[i] * a.c.n_kv_heads : 0;
#pragma unroll
        for (int d = 1; d < 32; d *= 2) {
          const int64_t y = __shfl_up_sync(0xffffffffu, x, d);
          if ((int)threadIdx.x >= d) x += y;
        }
        if (i < G) at[i + 1] = sum + x;
        sum += __shfl_sync(0xffffffffu, x, 31);
      }
      if (threadIdx.x == 0) at[0] = 0;
    }
    __syncthreads();
  }
  // the CTA's share
  __device__ __forceinline__ void share(int G, int64_t &x0, int64_t &x1) const {
    const int64_t total = at[G], P = min((int64_t)gridDim.x, total);
    x0 = blockIdx.x < P ? total * blockIdx.x / P : 0;
    x1 = blockIdx.x < P ? total * (blockIdx.x + 1) / P : 0;
  }
  // the (sequence, row tile) that unit x of the row belongs to
  __device__ __forceinline__ int group(int64_t x, int G) const {
    int lo = 0, hi = G;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (at[mid] <= x) lo = mid;
      else hi = mid;
    }
    return lo;
  }
  // the CTA of P that unit x of the row belongs to: the last one that begins
  // at or before it, total * i / P < x + 1
  __device__ __forceinline__ int owner(int64_t x, int64_t total, int64_t P) const {
    return (int)((P * (x + 1) - 1) / total);
  }
};

// 2^(m - top), 0 for a share that saw nothing
__device__ __forceinline__ float share(float m, float top) { return m == -INFINITY ? 0.f : exp2f(m - top); }

// The kernel for many rows (attend8_rows.cu), for bf16 caches. How it splits a
// call of `rows` rows a slice, the last of which see at most `steps` times 128
// tokens and the first `tokens` tokens fewer: CTAs of a streamed launch, or 0;
// returns the time that takes, in steps. Then the workspace, and the launch.
constexpr int kRowsTile = 256, kRowsStep = 128;  // rows and tokens of a tile's step
double rows_plan(const lkv_cache8 &c, int64_t rows, int64_t tokens, int64_t steps, int sms, int *ctas);
int64_t rows_bytes(int ctas);
cudaError_t launch_attend_rows(const AttendArgs &a, int ctas, cudaStream_t st);

}  // namespace lkv
