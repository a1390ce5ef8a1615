// attend8_shared.cu -- causal attention of sequences behind shared prefixes over
// 8-bit caches (lkv_cache8_attend_shared).
#include "attend8_few.cuh"

namespace lkv {

// Tiles of 16: blocks that a CTA takes at least, as fewer make parts for nothing (4
// samples of 2048 tokens with 8, 12 and 16 blocks 17.5, 21 and 16 us).
constexpr int kSharedFewLeast = 16;

// Two launches. The first takes each prefix's blocks once for the rows of all
// sequences behind it and leaves parts (attend8_shared.cuh): in tensor memory's
// tiles of 128 rows (bf16), or in tiles of 16. The second takes each sequence's
// own blocks, beside the first one's last CTAs, and joins its rows with their
// parts; where sequences have many rows the first has taken their own blocks too,
// and the second joins parts alone.
struct SharedPlan {
  int nt;            // row tiles of 8 nt rows, 16: the kernel for many rows
  bool own_parts;    // the own tokens too
  int ctas;
  int64_t tiles;     // at most
  int own_nt, row_tiles, cluster;
  int64_t own_tiles;
  int64_t seq_at, tile_at, parts_at, bytes;  // the workspace, at its beginning what the first launch vouches with
};

static thread_local int32_t vouch_late = 0;  // lkv_diag_shared_late
static thread_local int32_t hold_step = INT32_MAX;  // lkv_diag_shared_hold
static thread_local int64_t hold_limit = (int64_t)kCopyLimitNs;

static const char *plan_shared(const lkv_cache8 *c, const lkv_cache8 *p, int32_t group, int32_t n, int32_t max_len, int sms, SharedPlan *s) {
  const int64_t R = (int64_t)n * group, rows = c->batch * R, S = (int64_t)c->batch * c->n_kv_heads;
  if (rows * c->n_kv_heads > 0x7fffffff - 256) return "too many rows";
  const bool fp32 = c->dtype == LKV_DTYPE_FP32;
  const int64_t len = max_len > 0 && max_len < c->capacity ? max_len : c->capacity, blocks = (len + kBlock - 1) / kBlock;
  // On a GB300, int8, 8 KV heads, 4 query heads: up to 16 rows are faster in tiles
  // of 16 (4 samples of a 2048-token prompt 17 us, in tiles of 128 26 us), more
  // would read the prefix once for each 16.
  s->nt = !fp32 && rows > 16 ? 16 : rows <= 8 ? 1 : 2;
  // From 17 rows a sequence the own tokens go to the tiles of 128 too (27 x 3 tokens
  // of 8 heads over 1000 47 us, in tiles of 16 56; 8 x 8 tokens over 2000 39 and 48),
  // up to 8 they do not (32 x 1 over 600 64 and 43), and between them where that
  // makes few steps a CTA: with 8.2 of 4 x 4 tokens over 4000 39 us, in tiles of 16
  // 54; with 9.7 (8 x 4 over 2000) 35.5 and 37.3; with 13.5 (32 x 4 over 64) 98 and
  // 90; with 16.8 (32 x 3 over 300) 50 and 44.
  const int64_t steps = S * (kSharedStart + (len + kSharedStep - 1) / kSharedStep);
  s->own_parts = s->nt == 16 && (R > 16 || (R > 8 && steps <= 11 * (int64_t)sms));
  const int part_rows = 8 * s->nt;
  s->ctas = s->nt == 16 ? sms : sms * (fp32 && s->nt == 2 ? 1 : 2);
  const int64_t most_ctas = s->ctas;
  s->tiles = ((rows + part_rows - 1) / part_rows + (p->batch < c->batch ? p->batch : c->batch)) * c->n_kv_heads;
  if (s->own_parts) s->tiles += S * ((R + part_rows - 1) / part_rows);
  s->own_nt = R <= 8 ? 1 : 2;
  s->row_tiles = (int)((R + 8 * s->own_nt - 1) / (8 * s->own_nt));
  s->own_tiles = S * s->row_tiles;
  const int64_t slots = (int64_t)sms * (fp32 && s->own_nt == 2 ? 1 : 2);
  int64_t cluster = slots / s->own_tiles, most = blocks / (2 * kAtWarps);  // a turn for every warp
  if (cluster > most) cluster = most;
  s->cluster = (int)(cluster < 1 ? 1 : cluster > kAtMaxCluster ? kAtMaxCluster : cluster);
  if (s->nt != 16) {
    // Where prefixes as long as their cache has room for would fill every CTA, some
    // are left out for the own tokens' to run beside them: 4 samples of 32K tokens 33
    // -> 29 us, of 131K 73 -> 68; in fp32, 16 of 152 CTAs, 44 -> 42 and 122 -> 119. More
    // than an eighth cost more than that: 24 of 152, 6 fp32 samples of 131K 197 -> 220.
    // Their lengths are known on the device alone. Short prefixes in a cache of 131K
    // tokens, against a cache that they fill: 1 to 4 samples, bf16 and fp32, of 64
    // tokens 1.3 to 1.8 us faster, of 512 0.1 to 1.5 faster, of 2048 from 1.4 faster to
    // 0.8 slower (4 samples, 17.8 -> 18.6), of 4096 the same. All CTAs launched, and as
    // many leaving again where the lengths say so: 4 samples of 131K 68 -> 77.
    const int64_t own = s->own_tiles * s->cluster, per_sm = fp32 && s->own_nt == 2 ? 1 : 2;
    const int64_t room = s->ctas > sms ? own : (own + per_sm - 1) / per_sm;
    if (room <= s->ctas / 8 && s->tiles * (p->capacity / kBlock) / kSharedFewLeast > s->ctas - room) s->ctas -= (int)room;
  }
  if (s->tiles > 0x7fffffff || s->own_tiles * s->cluster > 0x7fffffff) return "too many rows";
  s->seq_at = 16;
  s->tile_at = s->seq_at + (int64_t)c->batch * 16;
  s->parts_at = s->tile_at + (s->tiles * 8 + 15) / 16 * 16;
  // parts for all CTAs: the workspace does not depend on the prefixes' capacity
  s->bytes = s->parts_at + (most_ctas + s->tiles) * part_floats(part_rows) * 4;
  return nullptr;
}

template <int DT, int CODE, int NT, int MODE>
static cudaError_t launch_part(const SharedArgs &a, unsigned grid, int cluster, const CUtensorMap &km, const CUtensorMap &vm, cudaStream_t st) {
  auto *fn = k_attend8<DT, CODE, NT, MODE>;
  const int used = (int)sizeof(AtSmem<NT>) > kRingBytes ? (int)sizeof(AtSmem<NT>) : kRingBytes;
  const int smem = 1024 + used + (MODE == kPrefix ? (int)Prefixes<false>::bytes(a.c.batch, a.p.batch, false) : 0);
  static SmemAllowed allowed;
  cudaError_t e = allowed.allow((const void *)fn, 1024 + used + (MODE == kPrefix ? (int)Prefixes<false>::bytes(kSharedMost, kSharedMost, false) : 0));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kAtThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, fn, a, km, vm);
}

template <int DT, int CODE, int MODE>
static cudaError_t launch_part(const SharedArgs &a, int nt, unsigned grid, int cluster, const CUtensorMap &km, const CUtensorMap &vm, cudaStream_t st) {
  return nt == 1 ? launch_part<DT, CODE, 1, MODE>(a, grid, cluster, km, vm, st) : launch_part<DT, CODE, 2, MODE>(a, grid, cluster, km, vm, st);
}

template <int DT, int CODE>
static cudaError_t launch_shared(const SharedArgs &a, const SharedPlan &s, const CUtensorMap (&maps)[4], cudaStream_t st) {
  const cudaError_t e = s.nt == 16 ? launch_shared_rows(a, s.ctas, st) : launch_part<DT, CODE, kPrefix>(a, s.nt, (unsigned)s.ctas, 0, maps[0], maps[1], st);
  if (e != cudaSuccess) return e;
  if (s.own_parts) return launch_shared_join(a, st);
  return launch_part<DT, CODE, kOwn>(a, s.own_nt, (unsigned)(s.own_tiles * s.cluster), s.cluster, maps[2], maps[3], st);
}

// What the arguments of a call have to be, apart from the tensors.
static const char *check_shared(const lkv_cache8 *c, const lkv_cache8 *p, int32_t group, int32_t n, int32_t max_len) {
  if (const char *m = check_cache8(c)) return m;
  if (const char *m = check_cache8(p)) return m;
  if (p->n_kv_heads != c->n_kv_heads || p->dtype != c->dtype || p->code != c->code)
    return "the prefixes have other KV heads, another dtype or another code";
  if (c->batch > kSharedMost || p->batch > kSharedMost) return "at most 1024 sequences and 1024 prefixes";
  if (group < 1 || group > 128) return "group must be 1..128";
  if (n < 0 || n > (1 << 24)) return "n must be 0..2^24";
  if (max_len < 0) return "max_len must be >= 0";
  return nullptr;
}

}  // namespace lkv

extern "C" lkv_status lkv_diag_shared_late(int32_t on) {
  lkv::vouch_late = on != 0;
  return LKV_OK;
}

extern "C" lkv_status lkv_diag_shared_hold(int32_t step, int64_t limit_ns) {
  using namespace lkv;
  if (step >= 0 && (limit_ns < 1 || limit_ns > 1000000000)) return refuse("lkv_diag_shared_hold: limit_ns must be 1..1e9");
  hold_step = step < 0 ? INT32_MAX : step;
  hold_limit = step < 0 ? (int64_t)kCopyLimitNs : limit_ns;
  return LKV_OK;
}

extern "C" lkv_status lkv_cache8_attend_shared_workspace(const lkv_cache8 *c, const lkv_cache8 *prefix, int32_t group, int32_t n,
                                                         int32_t max_len, int64_t *bytes) {
  using namespace lkv;
  const char *where = "lkv_cache8_attend_shared_workspace";
  if (const char *m = check_shared(c, prefix, group, n, max_len)) return refuse_in(where, m);
  if (!bytes) return refuse_in(where, "null result");
  *bytes = 0;
  if (n == 0) return LKV_OK;
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_refuse(where, e);
  SharedPlan s;
  if (const char *m = plan_shared(c, prefix, group, n, max_len, sms, &s)) return refuse_in(where, m);
  *bytes = s.bytes;
  return LKV_OK;
}

extern "C" lkv_status lkv_cache8_attend_shared(const lkv_cache8 *c, const lkv_cache8 *prefix, const int32_t *prefix_of,
                                               const void *q, int32_t group, int32_t n, const int32_t *counts, float scale,
                                               int32_t max_len, void *out, void *workspace, int64_t workspace_bytes, void *stream) {
  using namespace lkv;
  const char *where = "lkv_cache8_attend_shared";
  if (const char *m = check_shared(c, prefix, group, n, max_len)) return refuse_in(where, m);
  const float scale_log2 = scale * kLog2e;
  if (!(scale_log2 - scale_log2 == 0.f)) return refuse_in(where, "scale, or its product with log2(e), is not finite");
  if (n == 0) return LKV_OK;
  if (!q || !out) return refuse_in(where, "null queries or output");
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(counts, 4) || !aligned(prefix_of, 4) || !aligned(workspace, 16))
    return refuse_in(where, "queries, output and workspace must be 16-byte aligned, counts and prefix_of 4-byte aligned");
  const int64_t S = (int64_t)c->batch * c->n_kv_heads, ib = (int64_t)c->batch * 4;
  const int64_t bytes = S * group * n * kHeadDim * (c->dtype == LKV_DTYPE_BF16 ? 2 : 4);
  if (overlaps_cache8(c, out, bytes) || overlaps_cache8(prefix, out, bytes) || overlap(out, bytes, q, bytes) || overlap(out, bytes, counts, ib) ||
      overlap(out, bytes, prefix_of, ib))
    return refuse_in(where, "the output overlaps a cache or an input");
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_refuse(where, e);
  SharedPlan s;
  if (const char *m = plan_shared(c, prefix, group, n, max_len, sms, &s)) return refuse_in(where, m);
  if (!workspace || workspace_bytes < s.bytes) return refuse_in(where, "the workspace is smaller than lkv_cache8_attend_shared_workspace says");
  if (overlaps_cache8(c, workspace, s.bytes) || overlaps_cache8(prefix, workspace, s.bytes) || overlap(workspace, s.bytes, q, bytes) ||
      overlap(workspace, s.bytes, out, bytes) || overlap(workspace, s.bytes, counts, ib) || overlap(workspace, s.bytes, prefix_of, ib))
    return refuse_in(where, "the workspace overlaps another tensor");
  SharedArgs a{};
  a.c = *c;
  a.p = *prefix;
  a.q = q;
  a.out = out;
  a.counts = counts;
  a.prefix_of = prefix_of;
  a.n = n;
  a.group = group;
  a.scale_log2 = scale_log2;
  a.row_tiles = s.row_tiles;
  a.part_rows = 8 * s.nt;
  a.least_units = s.nt == 16 ? 2 : kSharedFewLeast;
  a.own_parts = s.own_parts;
  a.seq = (int4 *)((char *)workspace + s.seq_at);
  a.tile = (int2 *)((char *)workspace + s.tile_at);
  a.parts = (float *)((char *)workspace + s.parts_at);
  a.vouch = (uint64_t *)workspace;
  a.late = vouch_late;
  a.hold = hold_step;
  a.limit_ns = (uint64_t)hold_limit;
  const int64_t SP = (int64_t)prefix->batch * prefix->n_kv_heads;
  CUtensorMap maps[4];  // of the prefixes and of the own tokens, where tiles of 16 take them
  if ((s.nt != 16 && (!codes_map(&maps[0], prefix->k_codes, prefix->capacity, SP, kBlock) || !codes_map(&maps[1], prefix->v_codes, prefix->capacity, SP, kBlock))) ||
      (!s.own_parts && (!codes_map(&maps[2], c->k_codes, c->capacity, S, kBlock) || !codes_map(&maps[3], c->v_codes, c->capacity, S, kBlock)))) {
    set_unbound_error("lkv_cache8_attend_shared: the driver refused a tensor map of the codes");
    return LKV_ECUDA;
  }
  cudaStream_t st = (cudaStream_t)stream;
  const bool bf = c->dtype == LKV_DTYPE_BF16, i8 = c->code == LKV_CODE_INT8;
  if (bf) e = i8 ? launch_shared<1, LKV_CODE_INT8>(a, s, maps, st) : launch_shared<1, LKV_CODE_E4M3>(a, s, maps, st);
  else e = i8 ? launch_shared<0, LKV_CODE_INT8>(a, s, maps, st) : launch_shared<0, LKV_CODE_E4M3>(a, s, maps, st);
  return e == cudaSuccess ? LKV_OK : cuda_refuse(where, e);
}
