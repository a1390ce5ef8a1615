// attend8.cu -- causal attention over the 8-bit cache (lkv_cache8_attend).
#include "attend8_few.cuh"

namespace lkv {

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
  auto *fn = k_attend8<DT, CODE, NT, kAlone>;
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
