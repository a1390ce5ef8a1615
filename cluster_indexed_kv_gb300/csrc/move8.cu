// move8.cu -- taking and keeping tokens of the 8-bit cache: lkv_cache8_take
// (sequences copied, forked, put in order, cut back and freed) and
// lkv_cache8_keep (blocks chosen for each KV head moved together).
#include "cache8.cuh"
#include "tma.cuh"

namespace lkv {

// Both kernels move whole blocks as they are, codes and scale, through shared
// memory: a warp (a CTA is one) has kMoveStages stages, of which all but one are
// being filled or emptied by bulk copies while it turns to the next. Nothing is
// computed but the tail of a sequence that ends inside an older block.
constexpr int kMoveStage = 16384;        // bytes of a stage's codes
constexpr int kMoveStages = 4;
constexpr int kMovePerSm = 3;            // CTAs that an SM's shared memory holds, where their tables are small
constexpr int kSmShared = 228 * 1024;    // an SM's shared memory, of which each CTA takes kSmReserved more than it asks for
constexpr int kSmReserved = 1024;
constexpr int kBlockBytes = kBlock * kHeadDim;
constexpr int kTakeItems = 32;           // destinations of a CTA between two caches
constexpr int kTakeInside = 1024;        // and within one, all of them: 16 bytes of each in a stage
constexpr int32_t kKeepBad = 1 << 30;    // in a ticket: the sequence's lists are refused

// a float to shared memory, by the thread's own groups
__device__ __forceinline__ void word_load(float *to, const float *from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_at(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void word_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void word_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Bytes [from, to) of a block (multiples of 16) in shared memory as the rows of
// a tail that lkv_cache8_read would give, by a whole warp.
template <int DT, int CODE>
__device__ __forceinline__ void to_tail(void *tail, const unsigned char *codes, int from, int to, float scale, int lane) {
  for (int at = from + 4 * lane; at < to; at += 128) {
    float x[4];
    decode4<CODE>(*(const uint32_t *)(codes + at - from), x);
    if (DT == 1)
      *(uint2 *)((uint16_t *)tail + at) = make_uint2(pack_bf16(x[0] * scale, x[1] * scale), pack_bf16(x[2] * scale, x[3] * scale));
    else
      *(float4 *)((float *)tail + at) = make_float4(x[0] * scale, x[1] * scale, x[2] * scale, x[3] * scale);
  }
}

// A tail as it is, by a whole warp.
template <int DT>
__device__ __forceinline__ void copy_tail(void *to, const void *from, int lane) {
  constexpr int N = kBlock * kHeadDim * (DT == 1 ? 2 : 4) / 16;
  uint4 w[N / 32];
#pragma unroll
  for (int i = 0; i < N / 32; ++i) w[i] = ((const uint4 *)from)[i * 32 + lane];
#pragma unroll
  for (int i = 0; i < N / 32; ++i) ((uint4 *)to)[i * 32 + lane] = w[i];
}

template <int DT>
__device__ __forceinline__ char *tail_of(void *tails, int64_t slice) {
  return (char *)tails + slice * kBlock * kHeadDim * (DT == 1 ? 2 : 4);
}

// ---------------------------------------------------------------- take

struct TakeArgs {
  lkv_cache8 to, from;            // from: within one cache, lengths are those before the call
  const int32_t *sequences, *lengths;
  void *new_tails[2];             // within one cache: the sequences' tails, made before any is written
  int32_t items;                  // destinations of a CTA
  int32_t inside;
};

// What a sequence becomes: its source (-1: it is left as it is), how much of it,
// and what is wrong with that.
struct Taken {
  int from, len, have, anomaly;
  __device__ __forceinline__ Taken(const TakeArgs &a, int b) : from(a.sequences ? a.sequences[b] : b), len(0), have(0), anomaly(0) {
    if (from < -1 || from >= a.from.batch) {
      anomaly = kAnomRange;
    } else if (from >= 0) {
      have = a.from.lengths[from];
      len = a.lengths ? a.lengths[b] : have;
      if (have < 0 || have > a.from.capacity || len < 0 || len > have) anomaly = kAnomRange;
      else if (len > a.to.capacity) anomaly = kAnomCapacity;
    }
    if (anomaly) from = -1;
  }
  // its last block, where that is not the source's last one (-1: the source's tail is its own)
  __device__ __forceinline__ int older() const { return len > 0 && (len - 1) / kBlock != (have - 1) / kBlock ? (len - 1) / kBlock : -1; }
  // whether its tail changes
  __device__ __forceinline__ bool moves(const TakeArgs &a, int b) const { return from >= 0 && len > 0 && !(a.inside && from == b && older() < 0); }
};

// The tail of a sequence that is to be `x`, by a whole warp: the source's own, or
// its last block's rows as lkv_cache8_read gives them.
template <int DT, int CODE>
__device__ __forceinline__ void make_tail(const TakeArgs &a, const Taken &x, int h, int kv, void *to, int lane) {
  const int64_t slice = (int64_t)x.from * a.from.n_kv_heads + h;
  const int older = x.older();
  if (older < 0) {
    copy_tail<DT>(to, tail_of<DT>(kv ? a.from.v_tail : a.from.k_tail, slice), lane);
  } else {
    const unsigned char *codes = (const unsigned char *)(kv ? a.from.v_codes : a.from.k_codes) + (slice * a.from.capacity + (int64_t)older * kBlock) * kHeadDim;
    to_tail<DT, CODE>(to, codes, 0, kBlockBytes, (kv ? a.from.v_scale : a.from.k_scale)[slice * (a.from.capacity / kBlock) + older], lane);
  }
}

// A sequence of the plan: its source, its length, and which slot of a stage holds the source's bytes (-1: none is needed).
struct TakeItem { int32_t from, len, slot; };
// How many blocks of a source the stages hold.
struct TakeSlot { int32_t from, hi; };

__host__ __device__ inline int64_t take_smem(int items) {
  const int words = items > kMoveStage / kBlockBytes ? items : kMoveStage / kBlockBytes;
  return 128 + kMoveStages * (int64_t)(kMoveStage + 4 * words) + items * (int64_t)(sizeof(TakeItem) + sizeof(TakeSlot));
}

// A CTA's tasks are columns: the same `unit` bytes of the codes of one KV head,
// K or V, in every sequence of its group. It loads each distinct source's once,
// and only when all of a column have arrived stores them, so that sequences of
// one cache may take one another's tokens in any order: columns do not depend
// on one another. Tails and lengths do: there they are made by a kernel before
// this one, from the cache as it was.
//
// Bound by bytes. On a GB300, 8 KV heads: one prompt of 8191 tokens into 16
// sequences 49 us, 86% of the measured copy rate; 8 sequences of 32768 into
// another cache 176 us (90%), and round within their own 189 us (84%); 24 beams of
// 517 tokens put in order 10.4 us, two launches' latency. Within a cache columns get
// narrower with the distinct sources (all are in one stage), and slow: each of 24, 64
// and 256 sequences from another at 67, 45 and 12% of the copy rate (88, 354 and 2540
// us); 520 of 1100 tokens from nine of them 380 us, each from another 16 ms.
template <int DT, int CODE>
__global__ void __launch_bounds__(32) k_cache8_take(const __grid_constant__ TakeArgs a) {
  extern __shared__ __align__(128) unsigned char area[];
  __shared__ __align__(8) uint64_t full_bar[kMoveStages];
  const int lane = threadIdx.x, group = blockIdx.y, H = a.to.n_kv_heads;
  const int words = max(a.items, kMoveStage / kBlockBytes);
  unsigned char *const stages = area;
  float *const scales = (float *)(area + kMoveStages * kMoveStage);
  TakeItem *const items = (TakeItem *)(scales + kMoveStages * words);
  TakeSlot *const slots = (TakeSlot *)(items + a.items);
  if (lane == 0) {
    for (int i = 0; i < kMoveStages; ++i) bar_init(&full_bar[i], 32);
    bar_init_fence();
  }
  __syncwarp();
  wait_prerequisites();

  // the plan: each CTA makes its group's again
  const int first = group * a.items, count = min(a.items, a.to.batch - first);
  int nslots = 0, most = 0;
  for (int i0 = 0; i0 < count; i0 += 32) {
    const int i = i0 + lane, b = first + i;
    int from = -1, len = 0, hi = 0;
    if (i < count) {
      const Taken x(a, b);
      from = x.from;
      len = x.len;
      if (from >= 0 && !(a.inside && from == b)) hi = len / kBlock;
      if (blockIdx.x == 0) {
        if (x.anomaly) atomicOr(a.to.ticket + a.to.batch, x.anomaly);
        else if (from >= 0) a.to.lengths[b] = len;
      }
    }
    const bool need = hi > 0;
    const uint32_t same = __match_any_sync(0xffffffffu, need ? from : -2 - lane);
    const int leader = __ffs(same) - 1;
    for (uint32_t rest = __reduce_or_sync(0xffffffffu, same & ~(1u << leader)); rest; rest &= rest - 1) {
      const int l2 = __ffs(rest) - 1;
      const int hi2 = __shfl_sync(0xffffffffu, hi, l2), of = __shfl_sync(0xffffffffu, leader, l2);
      if (of == lane) hi = max(hi, hi2);
    }
    const uint32_t lead = __ballot_sync(0xffffffffu, need && leader == lane);
    const int slot = nslots + __popc(lead & ((1u << leader) - 1u));
    if (i < count) items[i] = TakeItem{from, len, need ? slot : -1};
    if (need && leader == lane) slots[slot] = TakeSlot{from, hi};
    nslots += __popc(lead);
    most = max(most, (int)__reduce_max_sync(0xffffffffu, (uint32_t)hi));
  }
  __syncwarp();

  // the widest columns that fit a stage, narrower where that leaves CTAs without work
  int unit = kMoveStage;
  while (unit > 16 && unit * nslots > kMoveStage) unit /= 2;
  auto columns = [&] { return nslots ? ((int64_t)most * kBlockBytes + unit - 1) / unit : 0; };
  while (unit > kBlockBytes && columns() * 2 * H < 4 * (int64_t)gridDim.x) unit /= 2;
  const int64_t ncol = columns(), tasks = ncol * 2 * H;
  const int blocks = max(1, unit / kBlockBytes);  // of a column
  const int64_t slice_codes = (int64_t)a.from.capacity * kHeadDim, slice_scales = a.from.capacity / kBlock;

  auto place = [&](int64_t task, int64_t &c0, int &h, int &kv) {
    c0 = task % ncol * unit;
    kv = (int)(task / ncol) & 1;
    h = (int)(task / ncol) >> 1;
  };
  auto issue = [&](int64_t task, int st) {
    if (task < tasks) {
      int64_t c0;
      int h, kv;
      place(task, c0, h, kv);
      uint32_t bytes = 0;
      for (int j = lane; j < nslots; j += 32) {
        const int64_t r1 = min(c0 + unit, (int64_t)slots[j].hi * kBlockBytes);
        if (r1 > c0) bytes += (uint32_t)(r1 - c0);
      }
      bar_expect(&full_bar[st], bytes);
      for (int j = lane; j < nslots; j += 32) {
        const TakeSlot s = slots[j];
        const int64_t r1 = min(c0 + unit, (int64_t)s.hi * kBlockBytes);
        if (r1 <= c0) continue;
        const int64_t slice = (int64_t)s.from * H + h;
        bulk_load(stages + st * kMoveStage + j * unit, (const char *)(kv ? a.from.v_codes : a.from.k_codes) + slice * slice_codes + c0, (uint32_t)(r1 - c0),
                  &full_bar[st]);
        if (c0 % kBlockBytes) continue;  // a block's scale goes with its first bytes
        const float *from = (kv ? a.from.v_scale : a.from.k_scale) + slice * slice_scales;
        const int k0 = (int)(c0 / kBlockBytes);
        for (int k = 0; k < blocks; ++k)
          if (k0 + k < s.hi) word_load(scales + st * words + j * blocks + k, from + k0 + k);
      }
    }
    word_commit();
  };

  const int64_t step = gridDim.x;
  for (int i = 0; i < kMoveStages; ++i) issue(blockIdx.x + i * step, i);
  uint32_t phase = 0;
  bool dead = false;
  int64_t task = blockIdx.x;
  for (int i = 0; task < tasks; ++i, task += step) {
    const int st = i % kMoveStages;
    if (!__all_sync(0xffffffffu, bar_wait(&full_bar[st], (phase >> st) & 1))) {
      dead = true;
      break;
    }
    phase ^= 1u << st;
    word_wait<kMoveStages - 2>();  // one group a stage, the stages behind this one but for the next to be filled
    __syncwarp();
    int64_t c0;
    int h, kv;
    place(task, c0, h, kv);
    const int k0 = (int)(c0 / kBlockBytes);
    for (int it = lane; it < count; it += 32) {
      const TakeItem x = items[it];
      if (x.slot < 0) continue;
      const int64_t slice = (int64_t)(first + it) * H + h;
      const int full = x.len / kBlock;
      const int64_t r1 = min(c0 + unit, (int64_t)full * kBlockBytes);
      if (r1 <= c0) continue;
      bulk_store((char *)(kv ? a.to.v_codes : a.to.k_codes) + slice * a.to.capacity * kHeadDim + c0, stages + st * kMoveStage + x.slot * unit, (uint32_t)(r1 - c0));
      if (c0 % kBlockBytes == 0)
        for (int k = 0; k < blocks; ++k)
          if (k0 + k < full) (kv ? a.to.v_scale : a.to.k_scale)[slice * (a.to.capacity / kBlock) + k0 + k] = scales[st * words + x.slot * blocks + k];
    }
    bulk_commit();
    if (i > 0) {  // the stage before is empty once its stores have read it
      bulk_wait_read<1>();
      __syncwarp();
      issue(task + (kMoveStages - 1) * step, (i - 1) % kMoveStages);
    }
  }
  if (dead) {  // what is in flight lands before the warp ends
    if (lane == 0) atomicOr(a.to.ticket + a.to.batch, kAnomTimeout);
    for (int i = 0; i < kMoveStages; ++i) bar_wait(&full_bar[i], (phase >> i) & 1);
  }
  word_wait<0>();
  bulk_wait_all();

  for (int64_t t = blockIdx.x; t < (int64_t)count * 2 * H; t += step) {
    const int b = first + (int)(t / (2 * H)), h = (int)(t % (2 * H)) >> 1, kv = (int)t & 1;
    const Taken x(a, b);
    if (!x.moves(a, b)) continue;
    const int64_t slice = (int64_t)b * H + h;
    char *const tail = tail_of<DT>(kv ? a.to.v_tail : a.to.k_tail, slice);
    if (a.inside) copy_tail<DT>(tail, tail_of<DT>(a.new_tails[kv], slice), lane);
    else make_tail<DT, CODE>(a, x, h, kv, tail, lane);
  }
}

// Within one cache, before its sequences take one another's tokens: the lengths
// as they are, and the tails as they will be. A warp a tail.
template <int DT, int CODE>
__global__ void __launch_bounds__(128) k_cache8_take_tails(const __grid_constant__ TakeArgs a, int32_t *lengths) {
  wait_prerequisites();
  const int64_t warp = (int64_t)blockIdx.x * 4 + threadIdx.x / 32, i = (int64_t)blockIdx.x * 128 + threadIdx.x;
  if (i < a.to.batch) lengths[i] = a.to.lengths[i];
  const int H = a.to.n_kv_heads, kv = (int)warp & 1;
  const int64_t slice = warp >> 1;
  if (slice >= (int64_t)a.to.batch * H) return;
  const int b = (int)(slice / H), h = (int)(slice % H);
  const Taken x(a, b);
  if (x.moves(a, b)) make_tail<DT, CODE>(a, x, h, kv, tail_of<DT>(a.new_tails[kv], slice), threadIdx.x & 31);
}

// ---------------------------------------------------------------- keep

struct KeepArgs {
  lkv_cache8 to, from;
  const int32_t *blocks, *counts;
  int32_t m;
  int32_t split;      // CTAs of a (sequence, KV head) and tensor
};

// Whether a sequence's count and its lists can be kept: a CTA a (KV head,
// sequence). What is wrong goes into the sequence's ticket, which is 0 at rest.
__global__ void __launch_bounds__(256) k_cache8_keep_check(const __grid_constant__ KeepArgs a) {
  wait_prerequisites();
  const int h = blockIdx.x, b = blockIdx.y, count = a.counts[b], len = a.from.lengths[b];
  if (count == -1) return;
  int anomaly = 0;
  if (count < 0 || count > a.m || len < 0 || len > a.from.capacity || count > len / kBlock) anomaly = kAnomRange;
  else if ((int64_t)count * kBlock + len % kBlock > a.to.capacity) anomaly = kAnomCapacity;
  else {
    const int32_t *list = a.blocks + ((int64_t)b * a.to.n_kv_heads + h) * a.m;
    const int full = len / kBlock;
    for (int j = threadIdx.x; j < count; j += 256) {
      const int x = list[j], before = j ? list[j - 1] : -1;
      if (x <= before || x >= full) anomaly = kAnomRange;
    }
  }
  if (anomaly) {
    atomicOr(a.to.ticket + b, kKeepBad);
    atomicOr(a.to.ticket + a.to.batch, anomaly);
  }
}

// What the kernels of a keep know of their (sequence, KV head) and tensor.
struct KeepLane {
  int64_t slice;
  int b, kv, part, count, len, last;
  bool go, older;
  const int32_t *list;
  const char *from;
  char *to;
  const float *from_scale;
  float *to_scale;
  __device__ __forceinline__ explicit KeepLane(const KeepArgs &a) {
    part = (int)(blockIdx.x % a.split);
    kv = (int)(blockIdx.x / a.split) & 1;
    slice = blockIdx.x / a.split >> 1;
    b = (int)(slice / a.to.n_kv_heads);
    count = a.counts[b];
    len = __ldcg(a.from.lengths + b);
    go = count >= 0 && !(__ldcg(a.to.ticket + b) & kKeepBad);
    list = a.blocks + slice * a.m;
    from = (const char *)(kv ? a.from.v_codes : a.from.k_codes) + slice * a.from.capacity * kHeadDim;
    to = (char *)(kv ? a.to.v_codes : a.to.k_codes) + slice * a.to.capacity * kHeadDim;
    from_scale = (kv ? a.from.v_scale : a.from.k_scale) + slice * (a.from.capacity / kBlock);
    to_scale = (kv ? a.to.v_scale : a.to.k_scale) + slice * (a.to.capacity / kBlock);
    // where no partial block follows, the last kept block is the last one; older: the source's tail is not its
    last = go && count > 0 && len % kBlock == 0 ? list[count - 1] : -1;
    older = last >= 0 && last != (len - 1) / kBlock;
  }
  // Every CTA of the sequence has read its length when it arrives (one thread); the last sets it.
  __device__ __forceinline__ void arrive(const KeepArgs &a) const {
    if (((atomicAdd(a.to.ticket + b, 1) + 1) & ~kKeepBad) != 2 * a.to.n_kv_heads * a.split) return;
    a.to.ticket[b] = 0;
    if (go) a.to.lengths[b] = count * kBlock + len % kBlock;
  }
};

// Between two caches: a CTA (a warp) takes a run of a list.
//
// Bound by bytes. On a GB300, half the blocks of 8 x 32768 tokens (8 KV heads,
// int8): 97 us, 82% of the measured copy rate, the check of the lists among it;
// of one such sequence 16 us.
template <int DT, int CODE>
__global__ void __launch_bounds__(32) k_cache8_keep(const __grid_constant__ KeepArgs a) {
  extern __shared__ __align__(128) unsigned char area[];
  __shared__ __align__(8) uint64_t full_bar[kMoveStages];
  __shared__ float scales[kMoveStages][32];
  constexpr int per = kMoveStage / kBlockBytes;  // blocks of a stage, a lane each
  const int lane = threadIdx.x;
  if (lane == 0) {
    for (int i = 0; i < kMoveStages; ++i) bar_init(&full_bar[i], 32);
    bar_init_fence();
  }
  __syncwarp();
  wait_prerequisites();
  const KeepLane z(a);
  int j0 = 0, j1 = 0;
  if (z.go) {
    j0 = (int)((int64_t)z.count * z.part / a.split);
    j1 = (int)((int64_t)z.count * (z.part + 1) / a.split);
  }
  int next;  // a lane's block of the stage to come: read a stage ahead
  auto fetch = [&](int64_t j) { next = lane < per && j + lane < j1 ? z.list[j + lane] : 0; };
  auto issue = [&](int64_t j, int st) {
    if (j < j1) {
      const bool mine = lane < per && j + lane < j1;
      bar_expect(&full_bar[st], mine ? kBlockBytes : 0);
      if (mine) {
        bulk_load(area + st * kMoveStage + lane * kBlockBytes, z.from + (int64_t)next * kBlockBytes, kBlockBytes, &full_bar[st]);
        word_load(&scales[st][lane], z.from_scale + next);
      }
      fetch(j + per);
    }
    word_commit();
  };
  fetch(j0);
  for (int i = 0; i < kMoveStages; ++i) issue(j0 + (int64_t)i * per, i);
  uint32_t phase = 0;
  bool dead = false;
  int i = 0;
  for (int64_t j = j0; j < j1; j += per, ++i) {
    const int st = i % kMoveStages;
    if (!__all_sync(0xffffffffu, bar_wait(&full_bar[st], (phase >> st) & 1))) {
      dead = true;
      break;
    }
    phase ^= 1u << st;
    word_wait<kMoveStages - 2>();
    __syncwarp();
    if (lane < per && j + lane < j1) {
      bulk_store(z.to + (j + lane) * kBlockBytes, area + st * kMoveStage + lane * kBlockBytes, kBlockBytes);
      z.to_scale[j + lane] = scales[st][lane];
    }
    const int64_t at = z.count - 1 - j;  // of the last kept block, in this stage
    if (z.older && at >= 0 && at < per && z.count <= j1)
      to_tail<DT, CODE>(tail_of<DT>(z.kv ? a.to.v_tail : a.to.k_tail, z.slice), area + st * kMoveStage + at * kBlockBytes, 0, kBlockBytes, scales[st][at], lane);
    bulk_commit();
    if (i > 0) {
      bulk_wait_read<1>();
      __syncwarp();
      issue(j + (int64_t)(kMoveStages - 1) * per, (i - 1) % kMoveStages);
    }
  }
  if (dead) {
    if (lane == 0) atomicOr(a.to.ticket + a.to.batch, kAnomTimeout);
    for (int k = 0; k < kMoveStages; ++k) bar_wait(&full_bar[k], (phase >> k) & 1);
  }
  word_wait<0>();
  bulk_wait_all();
  if (z.go && z.part == 0 && (z.len % kBlock != 0 || (z.last >= 0 && !z.older)))
    copy_tail<DT>(tail_of<DT>(z.kv ? a.to.v_tail : a.to.k_tail, z.slice), tail_of<DT>(z.kv ? a.from.v_tail : a.from.k_tail, z.slice), lane);
  __syncwarp();
  if (lane == 0) z.arrive(a);
}

// Within one cache: a CTA takes the same `unit` bytes of every block of a list,
// in order, kInsideLoads of 16 a thread at a time. Block j comes from one at or
// behind j, so what a run of blocks overwrites lies before what later runs read,
// and its own sources have been read when every thread is at the barrier. Lists
// of different heads and parts of blocks do not depend on one another.
//
// Bound by bytes, or by what few CTAs keep on their way. On a GB300, half the
// blocks of 8 x 32768 tokens 129 us, 61% of the measured copy rate; of one such
// sequence 21 us (67 us with bulk copies of 256 bytes, which the copy engine
// takes as long for as for 2 KB).
constexpr int kInsideThreads = 256, kInsideLoads = 4;
constexpr int kInsideBytes = kInsideThreads * kInsideLoads * 16;  // of a run
template <int DT, int CODE>
__global__ void __launch_bounds__(kInsideThreads) k_cache8_keep_inside(const __grid_constant__ KeepArgs a) {
  wait_prerequisites();
  const KeepLane z(a);
  const int unit = kBlockBytes / a.split, at = z.part * unit, chunks = unit / 16, per = kInsideBytes / unit;  // 16-byte chunks of a unit, blocks of a run
  const int count = z.go ? z.count : 0;
  // the thread's k-th chunk of a run: block block(k), bytes byte(k) of it
  auto block = [&](int k) { return (k * kInsideThreads + (int)threadIdx.x) / chunks; };
  auto byte = [&](int k) { return at + (k * kInsideThreads + (int)threadIdx.x) % chunks * 16; };
  const bool scales = z.part == 0 && (int)threadIdx.x < per;
  uint4 x[kInsideLoads], y[kInsideLoads];
  float sx = 0.f, sy = 0.f;
  auto load = [&](int64_t j, uint4 (&w)[kInsideLoads], float &s) {
#pragma unroll
    for (int k = 0; k < kInsideLoads; ++k) {
      w[k] = make_uint4(0, 0, 0, 0);
      if (j + block(k) < count) w[k] = __ldcg((const uint4 *)(z.from + (int64_t)z.list[j + block(k)] * kBlockBytes + byte(k)));
    }
    if (scales && j + threadIdx.x < count) s = __ldcg(z.from_scale + z.list[j + threadIdx.x]);
  };
  auto store = [&](int64_t j, const uint4 (&w)[kInsideLoads], float s) {
#pragma unroll
    for (int k = 0; k < kInsideLoads; ++k) {
      if (j + block(k) >= count) continue;
      *(uint4 *)(z.to + (j + block(k)) * kBlockBytes + byte(k)) = w[k];
      if (z.older && j + block(k) == count - 1) {  // the last kept block's values into the tail
        const float scale = __ldcg(z.from_scale + z.last);
        const uint32_t u[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float v[4];
          decode4<CODE>(u[e], v);
          char *tail = tail_of<DT>(z.kv ? a.to.v_tail : a.to.k_tail, z.slice) + (byte(k) + 4 * e) * (DT == 1 ? 2 : 4);
          if (DT == 1) *(uint2 *)tail = make_uint2(pack_bf16(v[0] * scale, v[1] * scale), pack_bf16(v[2] * scale, v[3] * scale));
          else *(float4 *)tail = make_float4(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale);
        }
      }
    }
    if (scales && j + threadIdx.x < count) z.to_scale[j + threadIdx.x] = s;
  };
  if (count > 0) load(0, x, sx);
  for (int64_t j = 0; j < count; j += 2 * per) {
    load(j + per, y, sy);
    __syncthreads();
    store(j, x, sx);
    load(j + 2 * per, x, sx);
    __syncthreads();
    store(j + per, y, sy);
  }
  __syncthreads();
  if (threadIdx.x == 0) z.arrive(a);
}

// What two caches of one call have to be; *inside: they are the same one.
static const char *check_pair(const lkv_cache8 *to, const lkv_cache8 **from, bool *inside) {
  if (const char *m = check_cache8(to)) return m;
  if (!*from) *from = to;
  if (const char *m = check_cache8(*from)) return m;
  const lkv_cache8 *f = *from;
  if (f->n_kv_heads != to->n_kv_heads || f->dtype != to->dtype || f->code != to->code)
    return "the source has other KV heads, another dtype or another code";
  *inside = f->k_codes == to->k_codes;
  if (*inside) {
    if (f->v_codes != to->v_codes || f->k_scale != to->k_scale || f->v_scale != to->v_scale || f->k_tail != to->k_tail ||
        f->v_tail != to->v_tail || f->lengths != to->lengths || f->ticket != to->ticket || f->batch != to->batch || f->capacity != to->capacity)
      return "the source shares some of the cache's arrays";
    return cache8_arrays_overlap(to) ? "two of the cache's arrays overlap" : nullptr;
  }
  if (cache8_arrays_overlap(to)) return "two of the cache's arrays overlap";
  if (caches_overlap(to, f)) return "the source shares some of the cache's arrays";
  return nullptr;
}

static int64_t tails_bytes(const lkv_cache8 *c) {
  const int64_t tail = (int64_t)c->batch * c->n_kv_heads * kBlock * kHeadDim * (c->dtype == LKV_DTYPE_BF16 ? 2 : 4);
  return 2 * tail + ((int64_t)c->batch * 4 + 15) / 16 * 16;
}

// A warp a CTA, with `smem` bytes of the at most `most` that the kernel takes.
template <auto FN, class Args>
static cudaError_t launch_sized(dim3 grid, size_t smem, size_t most, cudaStream_t st, const Args &a) {
  static SmemAllowed allowed;
  const cudaError_t e = allowed.allow((const void *)FN, (int)most);
  return e != cudaSuccess ? e : launch_next(FN, grid, 32, smem, st, a);
}

}  // namespace lkv

extern "C" lkv_status lkv_cache8_take_workspace(const lkv_cache8 *c, const lkv_cache8 *source, int64_t *bytes) {
  using namespace lkv;
  bool inside = false;
  if (const char *m = check_pair(c, &source, &inside)) return refuse_in("lkv_cache8_take_workspace", m);
  if (!bytes) return refuse("lkv_cache8_take_workspace: null result");
  *bytes = inside ? tails_bytes(c) : 0;
  return LKV_OK;
}

extern "C" lkv_status lkv_cache8_take(const lkv_cache8 *c, const lkv_cache8 *source, const int32_t *sequences,
                                      const int32_t *lengths, void *workspace, int64_t workspace_bytes, void *stream) {
  using namespace lkv;
  bool inside = false;
  if (const char *m = check_pair(c, &source, &inside)) return refuse_in("lkv_cache8_take", m);
  if (inside && c->batch > kTakeInside) return refuse("lkv_cache8_take: at most 1024 sequences within one cache");
  if (!aligned(sequences, 4) || !aligned(lengths, 4) || !aligned(workspace, 16))
    return refuse("lkv_cache8_take: sequences and lengths must be 4-byte aligned, the workspace 16-byte aligned");
  const int64_t ib = (int64_t)c->batch * 4;
  if (overlaps_cache8(c, sequences, ib) || overlaps_cache8(c, lengths, ib))
    return refuse("lkv_cache8_take: an input overlaps the cache's arrays");
  const int64_t need = inside ? tails_bytes(c) : 0;
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return refuse("lkv_cache8_take: the workspace is smaller than lkv_cache8_take_workspace says");
    if (overlaps_cache8(c, workspace, need) || overlap(workspace, need, sequences, ib) || overlap(workspace, need, lengths, ib))
      return refuse("lkv_cache8_take: the workspace overlaps another tensor");
  }
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_refuse("lkv_cache8_take", e);
  cudaStream_t st = (cudaStream_t)stream;
  TakeArgs a{};
  a.to = *c;
  a.from = *source;
  a.sequences = sequences;
  a.lengths = lengths;
  a.inside = inside;
  a.items = inside ? c->batch : c->batch < kTakeItems ? c->batch : kTakeItems;
  const bool bf = c->dtype == LKV_DTYPE_BF16, i8 = c->code == LKV_CODE_INT8;
  if (inside) {
    const int64_t slices = (int64_t)c->batch * c->n_kv_heads, tails = slices * kBlock * kHeadDim * (bf ? 2 : 4);
    a.new_tails[0] = workspace;
    a.new_tails[1] = (char *)workspace + tails;
    int32_t *const before = (int32_t *)((char *)workspace + 2 * tails);
    auto *fn = bf ? (i8 ? k_cache8_take_tails<1, LKV_CODE_INT8> : k_cache8_take_tails<1, LKV_CODE_E4M3>)
                  : (i8 ? k_cache8_take_tails<0, LKV_CODE_INT8> : k_cache8_take_tails<0, LKV_CODE_E4M3>);
    e = launch_next(fn, dim3((unsigned)((2 * slices + 3) / 4)), 128, 0, st, a, before);
    if (e != cudaSuccess) return cuda_refuse("lkv_cache8_take", e);
    a.from.lengths = before;
  }
  const int groups = (c->batch + a.items - 1) / a.items;  // below 2^16: 2^20 sequences at most
  // As many CTAs as there is room for at once, as each has an even share: within a
  // cache of some 300 sequences or more, with their tables, two an SM.
  const size_t smem = (size_t)take_smem(a.items), most = (size_t)take_smem(kTakeInside);
  const int fit = kSmShared / ((int)smem + kSmReserved + 64), wide = (fit < kMovePerSm ? fit : kMovePerSm) * sms;
  const dim3 grid((unsigned)((wide + groups - 1) / groups), (unsigned)groups);
  if (bf) e = i8 ? launch_sized<k_cache8_take<1, LKV_CODE_INT8>>(grid, smem, most, st, a) : launch_sized<k_cache8_take<1, LKV_CODE_E4M3>>(grid, smem, most, st, a);
  else e = i8 ? launch_sized<k_cache8_take<0, LKV_CODE_INT8>>(grid, smem, most, st, a) : launch_sized<k_cache8_take<0, LKV_CODE_E4M3>>(grid, smem, most, st, a);
  return e == cudaSuccess ? LKV_OK : cuda_refuse("lkv_cache8_take", e);
}

extern "C" lkv_status lkv_cache8_keep(const lkv_cache8 *c, const lkv_cache8 *source, const int32_t *blocks, int32_t m,
                                      const int32_t *counts, void *stream) {
  using namespace lkv;
  bool inside = false;
  if (const char *w = check_pair(c, &source, &inside)) return refuse_in("lkv_cache8_keep", w);
  if (source->batch != c->batch) return refuse("lkv_cache8_keep: the source has another number of sequences");
  if (m < 0) return refuse("lkv_cache8_keep: m must be >= 0");
  if (!counts || (m > 0 && !blocks)) return refuse("lkv_cache8_keep: null blocks or counts");
  if (!aligned(blocks, 4) || !aligned(counts, 4)) return refuse("lkv_cache8_keep: blocks and counts must be 4-byte aligned");
  if (c->batch > 65535) return refuse("lkv_cache8_keep: at most 65535 sequences");
  const int64_t slices = (int64_t)c->batch * c->n_kv_heads;
  if (overlaps_cache8(c, blocks, slices * m * 4) || overlaps_cache8(c, counts, (int64_t)c->batch * 4))
    return refuse("lkv_cache8_keep: an input overlaps the cache's arrays");
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return cuda_refuse("lkv_cache8_keep", e);
  cudaStream_t st = (cudaStream_t)stream;
  KeepArgs a{};
  a.to = *c;
  a.from = *source;
  a.blocks = blocks;
  a.counts = counts;
  a.m = m;
  // CTAs for a GPU full of them: runs of 8 blocks of a list at least, or parts
  // of 128 bytes of its blocks, no more than the GPU holds at once (of 8 x 32768
  // tokens in place, 256 CTAs and 512: 128 and 157 us)
  const int64_t want = ((int64_t)kMovePerSm * sms + 2 * slices - 1) / (2 * slices);
  a.split = 1;
  if (inside)
    while (a.split < 16 && 2 * slices * 2 * a.split <= 2 * sms) a.split *= 2;
  else
    a.split = (int32_t)(want < (m + 7) / 8 ? want : (m + 7) / 8 < 1 ? 1 : (m + 7) / 8);
  if (2 * slices * a.split > 0x7fffffff) return refuse("lkv_cache8_keep: too many sequences");
  e = launch_next(k_cache8_keep_check, dim3((unsigned)c->n_kv_heads, (unsigned)c->batch), 256, 0, st, a);
  if (e != cudaSuccess) return cuda_refuse("lkv_cache8_keep", e);
  const dim3 grid((unsigned)(2 * slices * a.split));
  const size_t smem = kMoveStages * kMoveStage;
  const bool bf = c->dtype == LKV_DTYPE_BF16, i8 = c->code == LKV_CODE_INT8;
  if (inside) {
    auto *fn = bf ? (i8 ? k_cache8_keep_inside<1, LKV_CODE_INT8> : k_cache8_keep_inside<1, LKV_CODE_E4M3>)
                  : (i8 ? k_cache8_keep_inside<0, LKV_CODE_INT8> : k_cache8_keep_inside<0, LKV_CODE_E4M3>);
    e = launch_next(fn, grid, kInsideThreads, 0, st, a);
    return e == cudaSuccess ? LKV_OK : cuda_refuse("lkv_cache8_keep", e);
  }
  if (bf) e = i8 ? launch_sized<k_cache8_keep<1, LKV_CODE_INT8>>(grid, smem, smem, st, a) : launch_sized<k_cache8_keep<1, LKV_CODE_E4M3>>(grid, smem, smem, st, a);
  else e = i8 ? launch_sized<k_cache8_keep<0, LKV_CODE_INT8>>(grid, smem, smem, st, a) : launch_sized<k_cache8_keep<0, LKV_CODE_E4M3>>(grid, smem, smem, st, a);
  return e == cudaSuccess ? LKV_OK : cuda_refuse("lkv_cache8_keep", e);
}
