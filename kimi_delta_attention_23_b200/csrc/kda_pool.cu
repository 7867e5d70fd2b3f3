// kda_pool.cu -- slots of a state pool copied, forked, freed and packed.
//
// Every call is a plan and a move.  The plan (one CTA, or every CTA for itself in a copy of few pairs) checks the request against the pool and
// writes the list of (source, destination) slots that the move carries out, so nothing about it is
// known on the host and the calls can be captured.  The move is bound by HBM: each byte is read
// and written once (a free: written once).
//
// Measured: 64 forks of 2 MB slots 43 us (268 MB, 95 % of the copy rate) behind a plan of 4 us; a copy of one
// 1 MB slot 1.9 us; 4096 slots of 740 bytes packed in 9.7 us, of which the plan is 7.
//
//   fork     the i-th valid request gets the lowest free slot not taken by an earlier one
//   compact  the j-th empty slot below the number of live ones receives the j-th live slot above it
//   copy     as one simultaneous assignment: every source is read as it was before the call, so
//            swaps, rotations and chains come out right.  A list in which no destination is another
//            pair's source moves like the others.  Any other list is carried out strip by strip: a
//            CTA owns a strip of a few columns of all listed slots, brings every source's piece of
//            it into shared memory, waits, and writes every destination's; no other CTA touches
//            those columns, so no copy of the pool and no order among the pairs is needed.
#include "kda_common.cuh"
#include "kda_ops_internal.h"

namespace kda {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMoveThreads = 256;
constexpr int kVecsPerLane = 8;
constexpr int kWarpVecs = 32 * kVecsPerLane;  // vectors that a warp moves at a time
constexpr int kMaxStripBytes = 192 * 1024;
constexpr int kFewStripBytes = 32 * 1024;  // 128 bytes of each of kMoveThreads pairs

// work layout: [0] number of pairs, [1] whether a destination is another pair's source, then
// src[n], dst[n], and the plan's own table [max_slots]
struct Work {
  int32_t* head;
  int32_t* src;
  int32_t* dst;
  int32_t* table;
};
__host__ __device__ __forceinline__ Work work_of(const PoolArgs& a, int32_t cap) {
  return {a.work, a.work + 4, a.work + 4 + cap, a.work + 4 + 2 * (size_t)cap};
}

// Exclusive prefix sums of one number per thread, and the total.
__device__ __forceinline__ int block_prefix(int x, int* s_warp, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sum = x;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += y;
  }
  if (lane == 31) s_warp[warp] = sum;
  __syncthreads();
  int w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const int before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  __syncthreads();  // s_warp may be written again
  return (warp > 0 ? before : 0) + sum - x;
}
static_assert(kPlanThreads == 1024, "block_prefix adds up 32 warps");

__device__ void plan_copy(const PoolArgs& a, const Work w) {
  __shared__ int s_count, s_hazard;
  if (threadIdx.x == 0) s_count = s_hazard = 0;
  auto inside = [&](int32_t s) { return s >= 0 && s < a.max_slots; };
  // table[slot]: the lowest pair that writes the slot, of those that a list names (others unused)
  for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
    const int32_t s = a.src[i], d = a.dst[i];
    if (inside(s) && inside(d)) {
      w.table[s] = INT32_MAX;
      w.table[d] = INT32_MAX;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
    const int32_t s = a.src[i], d = a.dst[i];
    if (inside(s) && inside(d)) atomicMin(&w.table[d], i);
    else if (s != -1 || d != -1) report(a.status, KDA_ERR_DEVICE_CHECK);  // (-1, -1): padding
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
    const int32_t s = a.src[i], d = a.dst[i];
    if (!inside(s) || !inside(d)) continue;
    if (w.table[d] != i) {
      report(a.status, KDA_ERR_DEVICE_CHECK);  // a destination named twice: the first pair counts
    } else if (s != d) {
      const int32_t over = w.table[s];  // the pair that overwrites this pair's source
      if (over != INT32_MAX && a.src[over] != s) s_hazard = 1;
      const int at = atomicAdd(&s_count, 1);
      w.src[at] = s;
      w.dst[at] = d;
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    w.head[0] = s_count;
    w.head[1] = s_hazard;
  }
}

// Slots are dealt to the threads in runs of equal length, so that one prefix sum over the runs' counts
// gives every slot its number of live slots before it, and with it every rank that a plan needs.
struct Run {
  int first, end;
};
__device__ __forceinline__ Run run_of(int slots) {
  const int each = (slots + kPlanThreads - 1) / kPlanThreads;
  const int first = min((int)threadIdx.x * each, slots);
  return {first, min(first + each, slots)};
}
__device__ __forceinline__ int count_live(const int32_t* live, Run run) {
  int n = 0;
  for (int s = run.first; s < run.end; ++s) n += live[s] != 0;
  return n;
}

__device__ void plan_fork(const PoolArgs& a, const Work w) {
  __shared__ int s_warp[kPlanThreads / 32];
  // the free slots, lowest first, as many as the list can ask for
  const Run run = run_of(a.max_slots);
  int live;
  int before = block_prefix(count_live(a.live, run), s_warp, live);
  for (int s = run.first; s < run.end; ++s) {
    const bool l = a.live[s] != 0;
    if (!l && s - before < a.n) w.table[s - before] = s;
    before += l;
  }
  const int free_slots = min(a.max_slots - live, a.n);
  __syncthreads();
  int asked = 0;
  for (int base = 0; base < a.n; base += kPlanThreads) {
    const int i = base + threadIdx.x;
    const int32_t s = i < a.n ? a.src[i] : -1;
    const bool ok = s >= 0 && s < a.max_slots && a.live[s] != 0;
    int total;
    const int r = asked + block_prefix(ok, s_warp, total);
    if (i < a.n) {
      const bool got = ok && r < free_slots;
      const int32_t d = got ? w.table[r] : -1;
      a.dst_out[i] = d;
      if (got) {
        w.src[r] = s;
        w.dst[r] = d;
      } else if (s != -1) {
        report(a.status, KDA_ERR_DEVICE_CHECK);  // no such live slot, or no free one left
      }
    }
    asked += total;
  }
  __syncthreads();  // the live flags have been read
  const int m = min(asked, free_slots);
  for (int r = threadIdx.x; r < m; r += kPlanThreads) a.live[w.table[r]] = 1;
  if (threadIdx.x == 0) {
    w.head[0] = m;
    w.head[1] = 0;
  }
}

__device__ void plan_free(const PoolArgs& a, const Work w) {
  __shared__ int s_count;
  if (threadIdx.x == 0) s_count = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
    const int32_t s = a.src[i];
    if (s >= 0 && s < a.max_slots && atomicExch(&a.live[s], 0) != 0) {
      w.dst[atomicAdd(&s_count, 1)] = s;
    } else if (s != -1) {
      report(a.status, KDA_ERR_DEVICE_CHECK);  // no such slot, or not live (any more)
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    w.head[0] = s_count;
    w.head[1] = 0;
  }
}

__device__ void plan_compact(const PoolArgs& a, const Work w) {
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int s_kept;
  const Run run = run_of(a.max_slots);
  int live;
  const int first = block_prefix(count_live(a.live, run), s_warp, live);
  if (live == a.max_slots) {
    if (threadIdx.x == 0) s_kept = live;
  } else if (run.first <= live && live < run.end) {  // live slots that stay: those below the number of live ones
    int before = first;
    for (int s = run.first; s < live; ++s) before += a.live[s] != 0;
    s_kept = before;
  }
  __syncthreads();
  const int kept = s_kept, holes = live - kept;
  int before = first;
  for (int s = run.first; s < run.end; ++s) {
    const bool l = a.live[s] != 0;
    if (s < live && !l) w.dst[s - before] = s;
    if (s >= live && l) w.src[before - kept] = s;
    w.table[s] = l ? s : -1;
    a.live[s] = s < live;
    before += l;
  }
  __syncthreads();
  for (int r = threadIdx.x; r < holes; r += kPlanThreads) w.table[w.src[r]] = w.dst[r];
  __syncthreads();
  for (int i = threadIdx.x; i < a.n; i += kPlanThreads) {
    const int32_t s = a.indices[i];
    const int32_t to = s >= 0 && s < a.max_slots ? w.table[s] : -1;
    if (to >= 0) a.indices[i] = to;
    else if (s != -1) report(a.status, KDA_ERR_DEVICE_CHECK);  // no live slot: left as it is
  }
  if (threadIdx.x == 0) {
    a.num_live[0] = live;
    w.head[0] = holes;
    w.head[1] = 0;
  }
}

__global__ void __launch_bounds__(kPlanThreads) pool_plan_kernel(const PoolArgs a, const Work w, const PoolOp op) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the move may take its place on the SMs
  if (op == kPoolCopy) plan_copy(a, w);
  else if (op == kPoolFork) plan_fork(a, w);
  else if (op == kPoolFree) plan_free(a, w);
  else plan_compact(a, w);
}

// Each warp takes up to kWarpVecs consecutive vectors of one slot at a time.
template <typename V, bool kZero>
__device__ void move_flat(const PoolArgs& a, const Work& w, int m) {
  const int64_t vecs = a.slot_elems / (int64_t)(sizeof(V) / 4);
  const int64_t segs = (vecs + kWarpVecs - 1) / kWarpVecs;
  const int64_t per_layer = segs * m, units = per_layer * a.layers;
  const int lane = threadIdx.x & 31;
  const int64_t warps = (int64_t)gridDim.x * (kMoveThreads / 32);
  for (int64_t u = (int64_t)blockIdx.x * (kMoveThreads / 32) + (threadIdx.x >> 5); u < units; u += warps) {
    const int64_t layer = u / per_layer, in_layer = u - layer * per_layer;
    const int64_t pair = in_layer / segs, v0 = (in_layer - pair * segs) * kWarpVecs + lane;
    V* base = reinterpret_cast<V*>(a.pool) + layer * a.max_slots * vecs;
    V* to = base + w.dst[pair] * vecs + v0;
    if constexpr (kZero) {
#pragma unroll
      for (int j = 0; j < kVecsPerLane; ++j)
        if (v0 + 32 * j < vecs) to[32 * j] = V{};
    } else {
      const V* from = base + w.src[pair] * vecs + v0;
      V r[kVecsPerLane];
#pragma unroll
      for (int j = 0; j < kVecsPerLane; ++j)
        if (v0 + 32 * j < vecs) r[j] = from[32 * j];
#pragma unroll
      for (int j = 0; j < kVecsPerLane; ++j)
        if (v0 + 32 * j < vecs) to[32 * j] = r[j];
    }
  }
}

// A strip of 2^shift columns of every listed slot: all read, then all written.
template <typename V>
__device__ void move_strips(const PoolArgs& a, const Work& w, int m, int smem_bytes, V* buf) {
  const int64_t vecs = a.slot_elems / (int64_t)(sizeof(V) / 4);
  // the widest strip that holds all pairs and still leaves every CTA one
  int shift = 0;
  while (shift < 12 && ((int64_t)m << (shift + 1)) * (int64_t)sizeof(V) <= smem_bytes &&
         (vecs * a.layers) >> (shift + 1) >= gridDim.x)
    ++shift;
  const int64_t strips = (vecs + (1 << shift) - 1) >> shift;
  for (int64_t u = blockIdx.x; u < strips * a.layers; u += gridDim.x) {
    const int64_t layer = u / strips, v0 = (u - layer * strips) << shift;
    V* base = reinterpret_cast<V*>(a.pool) + layer * a.max_slots * vecs;
    for (int it = threadIdx.x; it < m << shift; it += kMoveThreads) {
      const int64_t v = v0 + (it & ((1 << shift) - 1));
      if (v < vecs) buf[it] = base[w.src[it >> shift] * vecs + v];
    }
    __syncthreads();
    for (int it = threadIdx.x; it < m << shift; it += kMoveThreads) {
      const int64_t v = v0 + (it & ((1 << shift) - 1));
      if (v < vecs) base[w.dst[it >> shift] * vecs + v] = buf[it];
    }
    __syncthreads();
  }
}

template <typename V, PoolOp kOp>
__global__ void __launch_bounds__(kMoveThreads) pool_move_kernel(const PoolArgs a, const Work w, int smem_bytes) {
  extern __shared__ __align__(16) unsigned char buf[];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan is written
  const int m = w.head[0];
  if (m == 0) return;
  if (kOp == kPoolCopy && w.head[1]) move_strips<V>(a, w, m, smem_bytes, reinterpret_cast<V*>(buf));
  else move_flat<V, kOp == kPoolFree>(a, w, m);
}

// A copy of at most kMoveThreads pairs in one launch: every CTA works out the plan itself, a thread per
// pair, in as many steps as there are pairs.
template <typename V>
__global__ void __launch_bounds__(kMoveThreads) pool_copy_few_kernel(const PoolArgs a, int smem_bytes) {
  extern __shared__ __align__(16) unsigned char buf[];
  __shared__ int32_t s_src[kMoveThreads], s_dst[kMoveThreads], s_from[kMoveThreads], s_to[kMoveThreads];
  __shared__ int s_taken[kMoveThreads / 32];
  const int i = threadIdx.x;
  int32_t s = -1, d = -1;
  if (i < a.n) {
    s = a.src[i];
    d = a.dst[i];
  }
  bool ok = s >= 0 && s < a.max_slots && d >= 0 && d < a.max_slots;
  bool wrong = !ok && (s != -1 || d != -1);
  s_src[i] = ok ? s : -1;
  s_dst[i] = ok ? d : -1;
  __syncthreads();
  bool named = false;
  for (int j = 0; j < i && j < a.n; ++j) named |= ok && s_dst[j] == d;
  wrong |= named;  // a destination named twice: the first pair counts
  ok = ok && !named && s != d;
  if (blockIdx.x == 0 && wrong) report(a.status, KDA_ERR_DEVICE_CHECK);
  bool over = false;  // whether another pair writes this pair's source
  for (int j = 0; j < a.n; ++j) over |= s_dst[j] == s && s_src[j] != s;
  // the pairs that count, in the list's order: all CTAs share the work by their place in it
  const unsigned taken = __ballot_sync(0xffffffffu, ok);
  if ((i & 31) == 0) s_taken[i >> 5] = __popc(taken);
  const bool hazard = __syncthreads_or(ok && over);
  int m = 0, at = __popc(taken & ((1u << (i & 31)) - 1));
  for (int k = 0; k < kMoveThreads / 32; ++k) {
    at += k < i >> 5 ? s_taken[k] : 0;
    m += s_taken[k];
  }
  if (ok) {
    s_from[at] = s;
    s_to[at] = d;
  }
  __syncthreads();
  const Work w{nullptr, s_from, s_to, nullptr};
  if (m == 0) return;
  if (hazard) move_strips<V>(a, w, m, smem_bytes, reinterpret_cast<V*>(buf));
  else move_flat<V, false>(a, w, m);
}

template <typename V>
cudaError_t launch_move(const PoolArgs& a, const Work& w, PoolOp op, int32_t cap, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t vecs = a.slot_elems / (int64_t)(sizeof(V) / 4);
  const int64_t units = (vecs + kWarpVecs - 1) / kWarpVecs * cap * a.layers;
  const int64_t ctas = (units + kMoveThreads / 32 - 1) / (kMoveThreads / 32);
  const unsigned grid = (unsigned)(ctas < 8 * sms ? ctas : 8 * sms);
  if (op == kPoolCopy && a.n <= kMoveThreads) {
    pool_copy_few_kernel<V><<<grid, kMoveThreads, kFewStripBytes, stream>>>(a, kFewStripBytes);
    return cudaGetLastError();
  }
  pool_plan_kernel<<<1, kPlanThreads, 0, stream>>>(a, w, op);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  int smem = 0;
  void (*kernel)(const PoolArgs, const Work, int);
  if (op == kPoolCopy) {
    // a strip of 128 bytes of every pair where that fits, else narrower ones
    const int64_t want = (int64_t)cap * 128;
    smem = want < kMaxStripBytes ? (int)want : kMaxStripBytes;
    kernel = pool_move_kernel<V, kPoolCopy>;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxStripBytes);
  } else if (op == kPoolFree) {
    kernel = pool_move_kernel<V, kPoolFree>;
  } else {
    kernel = pool_move_kernel<V, kPoolFork>;
  }
  if (e != cudaSuccess) return e;
  // the move's launch overlaps the plan; it waits for the plan's end itself
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kMoveThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a, w, smem);
}

// entries of the pair lists: what one call can move at most
int32_t list_size(int32_t n, int32_t max_slots, PoolOp op) {
  const int32_t most = op == kPoolCompact ? max_slots / 2 : n < max_slots ? n : max_slots;
  return most > 0 ? most : 1;
}

}  // namespace

size_t pool_work_ints(int32_t n, int32_t max_slots) {
  const size_t most = n > max_slots ? n : max_slots;
  return 4 + 3 * most;
}

bool pool_needs_work(PoolOp op, int32_t n) { return op != kPoolCopy || n > kMoveThreads; }

cudaError_t launch_pool(const PoolArgs& a, PoolOp op, cudaStream_t stream) {
  const int32_t cap = list_size(a.n, a.max_slots, op);
  const Work w = work_of(a, a.n > a.max_slots ? a.n : a.max_slots);
  const bool vec = a.slot_elems % 4 == 0 && (reinterpret_cast<uintptr_t>(a.pool) & 15u) == 0;
  return vec ? launch_move<uint4>(a, w, op, cap, stream) : launch_move<uint32_t>(a, w, op, cap, stream);
}

}  // namespace kda
