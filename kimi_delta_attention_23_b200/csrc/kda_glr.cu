// kda_glr.cu -- the gated linear recurrence over a varlen batch, forward and backward, and its
// single-token step.
//
// Per sequence, head and channel (the diagonal-state relative of the KDA recurrence, with the same
// gate and the same per-head beta):
//     z = raw_gate + dt_bias,  g = -exp(a_log) softplus(z)  (safe: max(g, lb)),  a = exp(g)
//     h = a h + beta s x,      s = 1, or sqrt(1 - a^2) when the input is normalised;   out = h
// and backwards, with D_t the gradient of h_t:
//     D_t = dout_t + a_{t+1} D_{t+1}
//     dx = D beta s,   dbeta = sum_c D s x,   dg = D (a h_{t-1} + beta x ds/da a),   ds/da = -a / s
//     draw = -dg exp(a_log) sigmoid(z)  (0 where the safe gate is clamped),  da_log = sum dg g
//
// An element is 6 to 16 bytes and some 35 (forward) to 75 (backward) instructions, so neither HBM nor the
// issue slots have room to spare, and a scan that read its inputs twice would lose to HBM at once.  It
// needs no second reading when whoever reads a tile also finishes it: a cluster of CTAs walks along one
// (sequence, head), each CTA taking every cluster-size-th tile of 64 tokens x d channels.  Inside the CTA
// a warp holds consecutive tokens (a lane: four channels) and reduces them to one affine map
// h -> A h + B per channel; the maps are folded in token order, over the warps through shared memory,
// over the cluster's tiles through distributed shared memory.  Every CTA folds the same maps in the
// same order, so results do not depend on timing, and the carry never goes through global memory.
//
// Measured (B200, H = 32, d = 128): forward, 131072 tokens in bf16 with the normalised input, 0.912 ms for
// 3.24 GB (3.6 TB/s, 54 % of the copy rate): 128 of the 148 SMs work (32 heads x 4 CTAs), at 68 % of their
// issue slots.  32768 packed tokens with fp32 gates: forward 0.252 ms (1.07 GB), backward 0.589 ms (1.88 GB,
// 49 %), where 16 warps in step leave issue slots empty behind waits and shared-memory latency.  With the
// normalised input the backward pass takes 0.88 ms, in bf16 throughout 0.89: it works the decay and the root
// out anew for the maps, the states and the gradients, and spills.
//
// The backward pass walks the tiles in reverse.  The forward pass has kept the state entering each
// tile (1/64 of the fp32 size of the outputs), so h_{t-1} is rebuilt inside the tile and only D is
// carried.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cstddef>

#include "kda_cluster.cuh"
#include "kda_glr_math.cuh"
#include "kda_ops_internal.h"

namespace kda {
namespace {
using namespace glr;
namespace cg = cooperative_groups;

constexpr int kTile = kGlrBlock;  // tokens of a tile
constexpr int kRow = 128;         // elements of a tile row in shared memory
constexpr int kMaxCluster = 8;

// How rows of d channels come to shared memory: by tensor copies where rows start on 16 bytes; else
// four channels per lane at once, in words of 4 bytes, or element by element through registers.
enum Access { kTensor = 0, kVec4 = 1, kWord = 2, kElem = 3 };
constexpr float kLeast = -3.0e38f;  // an infinite gate counts as this one: its decay is 0 all the same
constexpr uint64_t kWaitNs = 1000000000ull;  // limit of a wait for a copy or for another warp

struct Maps {
  CUtensorMap x, raw, out;
};

template <int kBytes>
__device__ __forceinline__ void cp_async(void* dst, const void* src) {
  const uint32_t d = static_cast<uint32_t>(__cvta_generic_to_shared(dst));
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(d), "l"(src), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// One row of d channels to shared memory, by the warp that will read it.
template <typename T>
__device__ __forceinline__ void copy_row(T* dst, const T* src, int d, int lane, Access how) {
  if (how <= kVec4) {
    if (4 * lane < d) cp_async<4 * sizeof(T)>(dst + 4 * lane, src + 4 * lane);
  } else if (how == kWord) {
    constexpr int kPer = 4 / sizeof(T);
    for (int c = kPer * lane; c < d; c += 32 * kPer) cp_async<4>(dst + c, src + c);
  } else {
    for (int c = lane; c < d; c += 32) dst[c] = src[c];
  }
}

// A lane's four channels (4 lane ..) of an fp32 vector of d.
__device__ __forceinline__ void load4(const float* p, int d, int lane, float2& lo, float2& hi) {
  const int c = 4 * lane;
  lo = make_float2(c < d ? p[c] : 0.f, c + 1 < d ? p[c + 1] : 0.f);
  hi = make_float2(c + 2 < d ? p[c + 2] : 0.f, c + 3 < d ? p[c + 3] : 0.f);
}
template <typename T>
__device__ __forceinline__ void put4(T* p, int d, int lane, float2 lo, float2 hi, bool vec) {
  const int c = 4 * lane;
  if (vec) {
    if (c < d) store4(p + c, lo, hi);
  } else {
    if (c < d) from_f32(p + c, lo.x);
    if (c + 1 < d) from_f32(p + c + 1, lo.y);
    if (c + 2 < d) from_f32(p + c + 2, hi.x);
    if (c + 3 < d) from_f32(p + c + 3, hi.y);
  }
}

// An affine map h -> a h + b of a lane's four channels.
struct Map4 {
  float2 a0, a1, b0, b1;
};

// The forward kernel is launched with 96 registers per thread; its 4 carrying warps leave 32 of theirs to
// the 16 computing ones: 16 x 104 + 4 x 64 = 20 x 96 (131072 tokens: 1011 -> 903 us).  The backward
// kernel's carrying warps need what they have.
constexpr int kLaunchRegs = 96, kComputeRegs = 104, kCarryRegs = 64;
static_assert(16 * kComputeRegs + 4 * kCarryRegs <= 20 * kLaunchRegs, "more registers than the CTA has");

template <int kId, int kThreads>
__device__ __forceinline__ void named_barrier_sync() {
  asm volatile("bar.sync %0, %1;" ::"n"(kId), "n"(kThreads) : "memory");
}

// The sequence of this cluster; false (reported) if its offsets or slot are out of range.
__device__ __forceinline__ bool sequence(const int32_t* cu, int b, int64_t T, int32_t& s0, int32_t& n) {
  s0 = cu[b];
  n = cu[b + 1] - s0;
  return s0 >= 0 && n >= 0 && (int64_t)s0 + n <= T;
}

// A wait with a limit; kOthers where the cluster's other CTAs write what is waited for.  One that ran out is
// the CTA's last: its threads then run through to the end, sending and fetching nothing more.
template <bool kOthers>
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile int* gave_up, int32_t* status) {
  const uint32_t at = sm100::smem_addr(bar);
  // nearly always there: a sleeping wait takes longer to say so
  if (kOthers ? sm100::mbar_try_wait_cluster(at, parity) : sm100::mbar_try_wait(at, parity)) return true;
  if (*gave_up) return false;
  if (kOthers ? sm100::mbar_wait_sleep_cluster(at, parity, kWaitNs) : sm100::mbar_wait_sleep(at, parity, kWaitNs))
    return true;
  *gave_up = 1;
  report(status, KDA_ERR_DEVICE_TIMEOUT);
  return false;
}

// A pair to the same place in the shared memory of CTA `rank` of the cluster, counted on that CTA's
// barrier.  The message orders itself: a cluster barrier would make every thread wait until its
// outputs have been written to global memory.
__device__ __forceinline__ void send_map(float2* to, uint64_t* bar, int rank, float a, float b) {
  uint32_t dst, rbar;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(dst) : "r"(sm100::smem_addr(to)), "r"(rank));
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(rbar) : "r"(sm100::smem_addr(bar)), "r"(rank));
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];" ::"r"(dst),
               "r"(__float_as_uint(a)), "r"(__float_as_uint(b)), "r"(rbar)
               : "memory");
}
// ------------------------------------------------------------------------------------ forward
//
// 16 warps compute, 4 tokens of a 64-token tile each; 4 warps carry: a thread per channel, which folds
// the tokens' maps, trades the tile's map with the other CTAs and hands every warp the state that enters
// its tokens; one of its threads brings in the tiles, a tensor copy per input (256-byte copies of single
// rows took the issuing warps about 50 cycles each).  The computing warps never wait for a
// carry of their own step: they work out the gates and maps of the next tile first, and only then
// finish the last one, whose a and b they have kept in registers.

constexpr int kFwdWarps = 16;
constexpr int kFwdRows = kTile / kFwdWarps;  // consecutive tokens of a warp
constexpr int kCarryWarps = kRow / 32;
constexpr int kFwdThreads = 32 * (kFwdWarps + kCarryWarps);

template <typename TX, typename TR, typename TO>
struct FwdSmem {
  static constexpr int kStages = sizeof(TX) + sizeof(TR) <= 4 ? 4 : sizeof(TX) + sizeof(TR) <= 6 ? 3 : 2;
  static constexpr int kMaxRanks = kMaxCluster;
  alignas(128) TX x[kStages][kTile * kRow];
  alignas(128) TR raw[kStages][kTile * kRow];
  alignas(128) TO out[kTile * kRow];
  float2 map[2][kFwdWarps][kRow];       // (A, B) of a warp's tokens; A then becomes the entering state
  float2 tile_map[2][kMaxRanks][kRow];  // of a step's tiles
  uint64_t full[kStages];               // a tile has arrived
  uint64_t mapped[2], entered[2];       // the warps' maps are there; the states entering them are
  uint64_t tiles_in[2];                 // the tiles' maps have arrived
  int gave_up;
};

template <typename TX, typename TR, typename TO, bool kNorm, bool kSafe>
__global__ void __launch_bounds__(kFwdThreads, 1) glr_fwd_kernel(const GlrArgs p, const __grid_constant__ Maps maps,
                                                                 const Access how, const bool out_map, const bool vec_out) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  using Smem = FwdSmem<TX, TR, TO>;
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  constexpr int kStages = Smem::kStages;

  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int chain = blockIdx.x / ranks, b = chain / p.H, h = chain - b * p.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.d;

  int32_t s0, n;
  const int32_t slot = p.slots[b];
  if (!sequence(p.cu, b, p.total_tokens, s0, n) || slot < 0 || slot >= p.max_slots) {
    if (threadIdx.x == 0) report(p.status, KDA_ERR_DEVICE_CHECK);
    return;
  }
  if (n == 0) return;
  const size_t row = (size_t)p.H * d;  // elements from a token to the next
  const size_t first = (size_t)s0 * row + (size_t)h * d;
  const int tiles = (n + kTile - 1) / kTile, steps = (tiles + ranks - 1) / ranks;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) sm100::mbar_init(sm100::smem_addr(&sm.full[s]), 1);
    for (int s = 0; s < 2; ++s) {
      sm100::mbar_init(sm100::smem_addr(&sm.mapped[s]), kFwdWarps);
      sm100::mbar_init(sm100::smem_addr(&sm.entered[s]), kCarryWarps);
      sm100::mbar_init(sm100::smem_addr(&sm.tiles_in[s]), 1);
    }
    sm100::fence_mbar_init();
    sm.gave_up = 0;
  }
  cluster.sync();
  auto wait = [&](uint64_t* bar, int parity) { return wait_for<false>(bar, parity & 1, &sm.gave_up, p.status); };
  auto wait_others = [&](uint64_t* bar, int parity) { return wait_for<true>(bar, parity & 1, &sm.gave_up, p.status); };
  // Nothing of a CTA may be under way to its shared memory when it ends, nor anything of the others': before the
  // cluster's closing barrier the issuing thread waits, even after another wait has run out and again with a
  // limit, for the copies it has started.
  auto drain = [&](int fetched) {
    if (how == kTensor && threadIdx.x == 32 * kFwdWarps)
      for (int s = max(0, min(fetched, steps) - kStages); s < min(fetched, steps); ++s)
        sm100::mbar_wait_bounded(sm100::smem_addr(&sm.full[s % kStages]), s / kStages & 1, kWaitNs);
    __syncwarp();
  };
  const bool withhold = (p.flags & KDA_DEBUG_WITHHOLD_HANDOFF) && rank == ranks - 1;

  const int pitch = how == kTensor ? d : kRow;  // elements of a tile's row

  if (warp >= kFwdWarps) {
    // ---------------------------------------------------------------- carrying warps
    sm100::regs_decrease<kCarryRegs>();
    const int c = threadIdx.x - 32 * kFwdWarps;
    auto fetch = [&](int step) {
      if (how != kTensor || c != 0 || step >= steps) return;
      const int stage = step % kStages, tile = step * ranks + rank, t = s0 + tile * kTile;
      const uint32_t bar = sm100::smem_addr(&sm.full[stage]);
      if (tile >= tiles) return sm100::mbar_arrive(bar);  // nothing there: whatever is left in the rows will do
      sm100::mbar_arrive_expect_tx(bar, kTile * d * (uint32_t)(sizeof(TX) + sizeof(TR)));
      sm100::tma_load_3d(sm100::smem_addr(sm.x[stage]), &maps.x, 0, h, t, bar);
      sm100::tma_load_3d(sm100::smem_addr(sm.raw[stage]), &maps.raw, 0, h, t, bar);
    };
    for (int s = 0; s < kStages; ++s) fetch(s);
    int fetched = kStages;
    bool live = true;
    float* state = p.pool + ((size_t)slot * p.H + h) * d;
    float carry = c < d ? state[c] : 0.f;
    for (int step = 0; step < steps; ++step) {
      const int par = step & 1;
      live &= wait(&sm.mapped[par], step >> 1);
      float2 of[kFwdWarps];
      float pa = 1.f, pb = 0.f;
#pragma unroll
      for (int w = 0; w < kFwdWarps; ++w) of[w] = sm.map[par][w][c];
#pragma unroll
      for (int w = 0; w < kFwdWarps; ++w) {
        pb = fmaf(pb, of[w].x, of[w].y);
        pa *= of[w].x;
      }
      if (live) {
        if (!(withhold && step == 0))
          for (int k = 0; k < ranks; ++k) send_map(&sm.tile_map[par][rank][c], &sm.tiles_in[par], k, pa, pb);
        if (c == 0)
          sm100::mbar_arrive_expect_tx(sm100::smem_addr(&sm.tiles_in[par]), ranks * kRow * (uint32_t)sizeof(float2));
        fetch(step + kStages);  // into the tile that has just been read
        fetched = step + kStages + 1;
      }
      live &= wait_others(&sm.tiles_in[par], step >> 1);
      float in = carry;
      float2 m[kMaxCluster];
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) m[k] = k < ranks ? sm.tile_map[par][k][c] : make_float2(1.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (k == rank) in = carry;
        carry = fmaf(carry, m[k].x, m[k].y);
      }
      const int tile = step * ranks + rank;
      if (p.checkpoints && c < d && tile < tiles)
        p.checkpoints[((size_t)(s0 / kTile + b + tile) * p.H + h) * d + c] = in;
#pragma unroll
      for (int w = 0; w < kFwdWarps; ++w) {
        sm.map[par][w][c].x = in;
        in = fmaf(in, of[w].x, of[w].y);
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(sm100::smem_addr(&sm.entered[par]));
    }
    drain(fetched);
    sm100::cluster_arrive();
    sm100::cluster_wait();
    // after the barrier: every CTA of the cluster has read the state that this replaces
    if (rank == 0 && c < d) state[c] = carry;
    return;
  }

  // ------------------------------------------------------------------ computing warps
  sm100::regs_increase<kComputeRegs>();
  const HeadGate gate = head_gate(p.a_log[h], kSafe, p.lb);
  const bool prob = p.flags & KDA_BETA_PROB;
  float2 bias0, bias1;
  load4(p.dt_bias + (size_t)h * d, d, lane, bias0, bias1);
  bias0 = mul2(bias0, both(kLog2e));
  bias1 = mul2(bias1, both(kLog2e));
  const int row0 = warp * kFwdRows, own = row0 + (lane & (kFwdRows - 1));
  const float* beta = p.beta + (size_t)s0 * p.H + h;
  TO* out = reinterpret_cast<TO*>(p.out) + first + (size_t)row0 * row;
  // beta of one of the warp's tokens per lane, a step ahead
  auto load_beta = [&](int step) {
    const int t = (step * ranks + rank) * kTile + own;
    return step < steps && t < n ? beta[(size_t)t * p.H] : 0.f;
  };
  float bt = beta_fast(load_beta(0), prob), next_beta = load_beta(1);

  auto copy = [&](int step) {  // without tensor copies, the warp's own rows of a step's tile
    const int t0 = (step * ranks + rank) * kTile + row0, rows = step < steps ? min(max(n - t0, 0), kFwdRows) : 0;
    const size_t at = first + (size_t)t0 * row;
    for (int r = 0; r < rows; ++r) {
      const int to = (row0 + r) * kRow;
      copy_row(sm.x[step % kStages] + to, reinterpret_cast<const TX*>(p.x) + at + r * row, d, lane, how);
      copy_row(sm.raw[step % kStages] + to, reinterpret_cast<const TR*>(p.raw_gate) + at + r * row, d, lane, how);
    }
    cp_async_commit();
  };
  if (how != kTensor)
    for (int s = 0; s < kStages - 1; ++s) copy(s);

  struct Kept {  // a and b = beta s x of the warp's tokens
    float2 a0[kFwdRows], a1[kFwdRows], b0[kFwdRows], b1[kFwdRows];
  };
  auto work_out = [&](int step, Kept& k) {
    const int stage = step % kStages, par = step & 1;
    if (how == kTensor) {
      wait(&sm.full[stage], step / kStages);
    } else {
      __syncwarp();  // the rows that are replaced next have been read
      copy(step + kStages - 1);
      cp_async_wait<kStages - 1>();
      __syncwarp();
    }
    const TR* raws = sm.raw[stage] + row0 * pitch + 4 * lane;
    const TX* xs = sm.x[stage] + row0 * pitch + 4 * lane;
#pragma unroll
    for (int r = 0; r < kFwdRows; ++r) {
      const float bt_r = __shfl_sync(0xffffffffu, bt, r);
      float2 z0, z1, x0, x1;
      unpack4(raws + r * pitch, z0, z1);
      unpack4(xs + r * pitch, x0, x1);
      z0 = pre_log2(z0, bias0);
      z1 = pre_log2(z1, bias1);
      float2 g0 = gate_log2(z0, exp_neg_abs(z0), gate.c), g1 = gate_log2(z1, exp_neg_abs(z1), gate.c);
      if constexpr (kSafe) {
        g0 = clamp2(g0, gate.lb2);
        g1 = clamp2(g1, gate.lb2);
      }
      const Decay e0 = decay_of(g0), e1 = decay_of(g1);
      k.a0[r] = e0.a;
      k.a1[r] = e1.a;
      k.b0[r] = mul2(x0, both(bt_r));
      k.b1[r] = mul2(x1, both(bt_r));
      if constexpr (kNorm) {
        const float2 u0 = one_minus_sq(e0), u1 = one_minus_sq(e1);
        k.b0[r] = mul2(k.b0[r], mul2(u0, rsq2(u0)));
        k.b1[r] = mul2(k.b1[r], mul2(u1, rsq2(u1)));
      }
    }
    const int left = n - (step * ranks + rank) * kTile - row0;
    if (left < kFwdRows) {  // rows past the end, whatever they hold, are the identity
#pragma unroll
      for (int r = 0; r < kFwdRows; ++r) {
        if (r >= left) {
          k.a0[r] = k.a1[r] = both(1.f);
          k.b0[r] = k.b1[r] = both(0.f);
        }
      }
    }
    Map4 m{k.a0[0], k.a1[0], k.b0[0], k.b1[0]};
#pragma unroll
    for (int r = 1; r < kFwdRows; ++r) {
      m.a0 = mul2(m.a0, k.a0[r]);
      m.a1 = mul2(m.a1, k.a1[r]);
      m.b0 = fma2(m.b0, k.a0[r], k.b0[r]);
      m.b1 = fma2(m.b1, k.a1[r], k.b1[r]);
    }
    float4* to = reinterpret_cast<float4*>(&sm.map[par][warp][4 * lane]);
    to[0] = make_float4(m.a0.x, m.b0.x, m.a0.y, m.b0.y);
    to[1] = make_float4(m.a1.x, m.b1.x, m.a1.y, m.b1.y);
    __syncwarp();
    if (lane == 0) sm100::mbar_arrive(sm100::smem_addr(&sm.mapped[par]));
    bt = beta_fast(next_beta, prob);
    next_beta = load_beta(step + 2);
  };
  // outputs leave through shared memory, a tensor copy per warp: plain stores of all warps at the same
  // point of the step held them up for a third of it
  TO* staged = sm.out + row0 * kRow;
  auto finish = [&](int step, const Kept& k) {
    const int par = step & 1, tile = step * ranks + rank, left = n - tile * kTile - row0;
    const bool copied = out_map && left >= kFwdRows;
    sm100::bulk_wait_read_all();  // (the issuing lane's) the last rows have left
    wait(&sm.entered[par], step >> 1);
    const float4* from = reinterpret_cast<const float4*>(&sm.map[par][warp][4 * lane]);
    const float4 lo = from[0], hi = from[1];
    float2 in0 = make_float2(lo.x, lo.z), in1 = make_float2(hi.x, hi.z);
    float2 h0[kFwdRows], h1[kFwdRows];
#pragma unroll
    for (int r = 0; r < kFwdRows; ++r) {
      in0 = h0[r] = fma2(k.a0[r], in0, k.b0[r]);
      in1 = h1[r] = fma2(k.a1[r], in1, k.b1[r]);
    }
    if (copied) {
      __syncwarp();
      if (4 * lane < d) {
#pragma unroll
        for (int r = 0; r < kFwdRows; ++r) store4(staged + r * d + 4 * lane, h0[r], h1[r]);
      }
      sm100::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        sm100::tma_store_3d(&maps.out, sm100::smem_addr(staged), 0, h, s0 + tile * kTile + row0);
        sm100::bulk_commit();
      }
    } else {
      TO* to = out + (size_t)tile * kTile * row;
#pragma unroll
      for (int r = 0; r < kFwdRows; ++r)
        if (r < left) put4(to + r * row, d, lane, h0[r], h1[r], vec_out);
    }
  };
  Kept even, odd;
  work_out(0, even);
  for (int step = 0; step < steps; step += 2) {
    if (step + 1 < steps) work_out(step + 1, odd);
    finish(step, even);
    if (step + 1 >= steps) break;
    if (step + 2 < steps) work_out(step + 2, even);
    finish(step + 1, odd);
  }
  __syncwarp();
  sm100::cluster_arrive_relaxed();  // a computing warp touches no other CTA's memory
  sm100::bulk_wait_all();
  sm100::cluster_wait();
}

// ------------------------------------------------------------------------------------ backward
//
// The same division of labour, from the last tile to the first.  A computing warp first works out the
// gates of a tile and two maps over its tokens: of h forwards and of a D backwards (they share A); the
// carrying threads fold the former from the kept state that enters the tile and pass the latter through
// the cluster; then the gradients follow.  Between the two a warp keeps only the gates, in registers,
// and reads its inputs again from shared memory, where dx and draw_gate take their place and leave by
// tensor copies.

constexpr int kBwdWarps = 16;
constexpr int kBwdRows = kTile / kBwdWarps;
constexpr int kBwdThreads = 32 * (kBwdWarps + kCarryWarps);

struct BwdMaps {
  CUtensorMap x, raw, dout, dx, draw;
};

template <typename TX, typename TR, typename TO>
struct BwdSmem {
  static constexpr int kStages = sizeof(TX) + sizeof(TR) + sizeof(TO) <= 8 ? 3 : 2;
  // what fits beside the tiles: two sets of maps (a tile's may be there before the last one's are used), and
  // the maps of so many CTAs
  static constexpr bool kAhead = sizeof(TX) + sizeof(TR) + sizeof(TO) <= 6;
  static constexpr int kMaxRanks = kAhead ? kMaxCluster : kMaxCluster / 2;
  alignas(128) TX x[kStages][kTile * kRow];
  alignas(128) TR raw[kStages][kTile * kRow];
  alignas(128) TO dout[kStages][kTile * kRow];
  static constexpr int kMapBuffers = kAhead ? 2 : 1;
  float2 map[kMapBuffers][kBwdWarps][kRow];  // (A, B) forwards; then the state before and a D behind a warp's tokens
  float rev[kMapBuffers][kBwdWarps][kRow];   // B backwards
  float2 tile_map[2][kMaxRanks][kRow];
  uint64_t full[kStages], mapped[2], entered[2], tiles_in[2], done[2];
  int gave_up;
};

template <typename TX, typename TR, typename TO, bool kNorm, bool kSafe>
__global__ void __launch_bounds__(kBwdThreads, 1)
    glr_bwd_kernel(const GlrBwdArgs p, const __grid_constant__ BwdMaps maps, const Access how, const bool by_copy,
                   const bool vec_grad) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  using Smem = BwdSmem<TX, TR, TO>;
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  constexpr int kStages = Smem::kStages;
  constexpr bool kAhead = Smem::kAhead;

  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int chain = blockIdx.x / ranks, b = chain / p.H, h = chain - b * p.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.d;

  // partial sums of the parameters' gradients, one set per (sequence, rank)
  float* part = p.partial + ((size_t)(b * ranks + rank) * p.H + h) * (d + 1);
  int32_t s0, n;
  const bool ok = sequence(p.cu, b, p.total_tokens, s0, n);
  if (!ok || n == 0) {
    if (!ok && threadIdx.x == 0) report(p.status, KDA_ERR_DEVICE_CHECK);
    for (int c = threadIdx.x; c <= d; c += kBwdThreads) part[c] = 0.f;
    if (ok && rank == 0)  // the state only passes through an empty sequence
      for (int c = threadIdx.x; c < d; c += kBwdThreads) {
        const size_t at = ((size_t)b * p.H + h) * d + c;
        p.d_initial[at] = p.d_final ? p.d_final[at] : 0.f;
      }
    return;
  }
  const size_t row = (size_t)p.H * d;
  const size_t first = (size_t)s0 * row + (size_t)h * d;
  const int tiles = (n + kTile - 1) / kTile, steps = (tiles + ranks - 1) / ranks;
  const int pitch = how == kTensor ? d : kRow;
  // step 0 takes the last tiles; rank k the k-th from the end of the step's
  auto tile_of = [&](int step) { return tiles - 1 - (step * ranks + rank); };

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) sm100::mbar_init(sm100::smem_addr(&sm.full[s]), 1);
    for (int s = 0; s < 2; ++s) {
      sm100::mbar_init(sm100::smem_addr(&sm.mapped[s]), kBwdWarps);
      sm100::mbar_init(sm100::smem_addr(&sm.entered[s]), kCarryWarps);
      sm100::mbar_init(sm100::smem_addr(&sm.tiles_in[s]), 1);
      sm100::mbar_init(sm100::smem_addr(&sm.done[s]), kBwdWarps);
    }
    sm100::fence_mbar_init();
    sm.gave_up = 0;
  }
  if (how != kTensor && d < kRow) {  // channels past the head must add nothing to the sums over channels
    for (size_t i = threadIdx.x; i < offsetof(Smem, map) / 16; i += kBwdThreads)
      reinterpret_cast<uint4*>(&sm)[i] = make_uint4(0, 0, 0, 0);
  }
  cluster.sync();
  auto wait = [&](uint64_t* bar, int parity) { return wait_for<false>(bar, parity & 1, &sm.gave_up, p.status); };
  auto wait_others = [&](uint64_t* bar, int parity) { return wait_for<true>(bar, parity & 1, &sm.gave_up, p.status); };
  // as in the forward pass
  auto drain = [&](int fetched) {
    if (how == kTensor && threadIdx.x == 32 * kBwdWarps)
      for (int s = max(0, min(fetched, steps) - kStages); s < min(fetched, steps); ++s)
        sm100::mbar_wait_bounded(sm100::smem_addr(&sm.full[s % kStages]), s / kStages & 1, kWaitNs);
    __syncwarp();
  };
  const bool withhold = (p.flags & KDA_DEBUG_WITHHOLD_HANDOFF) && rank == ranks - 1;

  if (warp >= kBwdWarps) {
    // ---------------------------------------------------------------- carrying warps
    const int c = threadIdx.x - 32 * kBwdWarps;
    auto fetch = [&](int step) {
      if (how != kTensor || c != 0 || step >= steps) return;
      const int stage = step % kStages, tile = tile_of(step), t = s0 + tile * kTile;
      const uint32_t bar = sm100::smem_addr(&sm.full[stage]);
      if (tile < 0) return sm100::mbar_arrive(bar);
      sm100::mbar_arrive_expect_tx(bar, kTile * d * (uint32_t)(sizeof(TX) + sizeof(TR) + sizeof(TO)));
      sm100::tma_load_3d(sm100::smem_addr(sm.x[stage]), &maps.x, 0, h, t, bar);
      sm100::tma_load_3d(sm100::smem_addr(sm.raw[stage]), &maps.raw, 0, h, t, bar);
      sm100::tma_load_3d(sm100::smem_addr(sm.dout[stage]), &maps.dout, 0, h, t, bar);
    };
    for (int s = 0; s < kStages - 1; ++s) fetch(s);
    int fetched = kStages - 1;
    bool live = true;
    const float* kept = p.checkpoints + ((size_t)(s0 / kTile + b) * p.H + h) * d + c;
    auto entering = [&](int step) {
      const int tile = tile_of(step);
      return step < steps && tile >= 0 && c < d ? kept[(size_t)tile * row] : 0.f;
    };
    const size_t at = ((size_t)b * p.H + h) * d + c;
    float carry = p.d_final && c < d ? p.d_final[at] : 0.f;  // a D of the token after the cluster's tiles
    float state = entering(0);
    for (int step = 0; step < steps; ++step) {
      const int par = step & 1, buf = kAhead ? par : 0;
      live &= wait(&sm.mapped[par], step >> 1);
      float2 of[kBwdWarps];
      float back[kBwdWarps], pa = 1.f, pb = 0.f;
#pragma unroll
      for (int w = 0; w < kBwdWarps; ++w) {
        of[w] = sm.map[buf][w][c];
        back[w] = sm.rev[buf][w][c];
      }
#pragma unroll
      for (int w = kBwdWarps - 1; w >= 0; --w) {
        pb = fmaf(pb, of[w].x, back[w]);
        pa *= of[w].x;
      }
      if (live) {
        if (!(withhold && step == 0))
          for (int k = 0; k < ranks; ++k) send_map(&sm.tile_map[par][rank][c], &sm.tiles_in[par], k, pa, pb);
        if (c == 0)
          sm100::mbar_arrive_expect_tx(sm100::smem_addr(&sm.tiles_in[par]), ranks * kRow * (uint32_t)sizeof(float2));
      }
#pragma unroll
      for (int w = 0; w < kBwdWarps; ++w) {  // the state entering each warp's tokens, over B
        const float in = state;
        state = fmaf(state, of[w].x, of[w].y);
        of[w].y = in;
      }
      state = entering(step + 1);
      live &= wait_others(&sm.tiles_in[par], step >> 1);
      float in = carry;
      float2 m[kMaxCluster];
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) m[k] = k < ranks ? sm.tile_map[par][k][c] : make_float2(1.f, 0.f);
#pragma unroll
      for (int k = 0; k < kMaxCluster; ++k) {
        if (k == rank) in = carry;
        carry = fmaf(carry, m[k].x, m[k].y);
      }
#pragma unroll
      for (int w = kBwdWarps - 1; w >= 0; --w) {
        sm.map[buf][w][c] = make_float2(of[w].y, in);
        in = fmaf(in, of[w].x, back[w]);
      }
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(sm100::smem_addr(&sm.entered[par]));
      // the next tile goes where the last step's gradients have left
      if (step > 0 && c == 0) live &= wait(&sm.done[(step - 1) & 1], (step - 1) >> 1);
      if (live) {
        fetch(step + kStages - 1);
        fetched = step + kStages;
      }
    }
    if (rank == 0 && c < d) p.d_initial[at] = carry;
    drain(fetched);
    sm100::cluster_arrive();
  } else {
    // ---------------------------------------------------------------- computing warps
    const HeadGate gate = head_gate(p.a_log[h], kSafe, p.lb);
    const bool prob = p.flags & KDA_BETA_PROB;
    float2 bias0, bias1;
    load4(p.dt_bias + (size_t)h * d, d, lane, bias0, bias1);
    bias0 = mul2(bias0, both(kLog2e));
    bias1 = mul2(bias1, both(kLog2e));
    const int row0 = warp * kBwdRows, own = row0 + (lane & (kBwdRows - 1));
    const float* beta = p.beta + (size_t)s0 * p.H + h;
    auto load_beta = [&](int step) {
      const int tile = tile_of(step), t = tile * kTile + own;
      return step < steps && tile >= 0 && t < n ? beta[(size_t)t * p.H] : 0.f;
    };
    auto copy = [&](int step) {  // without tensor copies, the warp's own rows of a step's tile
      const int tile = tile_of(step), t0 = tile * kTile + row0;
      const int rows = step < steps && tile >= 0 ? min(max(n - t0, 0), kBwdRows) : 0;
      const size_t at = first + (size_t)t0 * row;
      for (int r = 0; r < rows; ++r) {
        const int to = (row0 + r) * kRow, stage = step % kStages;
        copy_row(sm.x[stage] + to, reinterpret_cast<const TX*>(p.x) + at + r * row, d, lane, how);
        copy_row(sm.raw[stage] + to, reinterpret_cast<const TR*>(p.raw_gate) + at + r * row, d, lane, how);
        copy_row(sm.dout[stage] + to, reinterpret_cast<const TO*>(p.dout) + at + r * row, d, lane, how);
      }
      cp_async_commit();
    };
    if (how != kTensor)
      for (int s = 0; s < kStages - 1; ++s) copy(s);
    float next_bt = beta_fast(load_beta(0), prob), later_beta = load_beta(1);
    float2 sum_bias0 = both(0.f), sum_bias1 = both(0.f), sum_log = both(0.f);
    const float2 one = both(1.f), zero = both(0.f);

    struct Kept {
      float2 g0[kBwdRows], g1[kBwdRows];  // gates (log2), clamped, and finite
      float bt;
    };
    auto input = [&](float2 x, float bt, const Decay& e) {
      float2 in = mul2(x, both(bt));
      if constexpr (kNorm) {
        const float2 u = one_minus_sq(e);
        in = mul2(in, mul2(u, rsq2(u)));
      }
      return in;
    };
    auto work_out = [&](int step, Kept& k) {
      const int stage = step % kStages, par = step & 1, buf = kAhead ? par : 0;
      k.bt = next_bt;
      if (how == kTensor) {
        wait(&sm.full[stage], step / kStages);
      } else {
        __syncwarp();
        if (kAhead && step > 0) copy(step + kStages - 2);
        cp_async_wait<kStages - 2>();
        __syncwarp();
      }
      const TX* xs = sm.x[stage] + row0 * pitch + 4 * lane;
      const TR* raws = sm.raw[stage] + row0 * pitch + 4 * lane;
      const TO* douts = sm.dout[stage] + row0 * pitch + 4 * lane;
      const int tile = tile_of(step), left = tile >= 0 ? n - tile * kTile - row0 : 0;
      Map4 m{one, one, zero, zero};
      float2 e0 = zero, e1 = zero, a0[kBwdRows], a1[kBwdRows];
#pragma unroll
      for (int r = 0; r < kBwdRows; ++r) {
        const float bt_r = __shfl_sync(0xffffffffu, k.bt, r);
        float2 z0, z1, x0, x1;
        unpack4(raws + r * pitch, z0, z1);
        unpack4(xs + r * pitch, x0, x1);
        z0 = pre_log2(z0, bias0);
        z1 = pre_log2(z1, bias1);
        k.g0[r] = clamp2(gate_log2(z0, exp_neg_abs(z0), gate.c), fmaxf(gate.lb2, kLeast));
        k.g1[r] = clamp2(gate_log2(z1, exp_neg_abs(z1), gate.c), fmaxf(gate.lb2, kLeast));
        const Decay d0 = decay_of(k.g0[r]), d1 = decay_of(k.g1[r]);
        a0[r] = d0.a;
        a1[r] = d1.a;
        float2 b0 = input(x0, bt_r, d0), b1 = input(x1, bt_r, d1);
        if (r >= left) {  // rows past the end are the identity
          a0[r] = a1[r] = one;
          b0 = b1 = zero;
        }
        m.a0 = mul2(m.a0, a0[r]);
        m.a1 = mul2(m.a1, a1[r]);
        m.b0 = fma2(m.b0, a0[r], b0);
        m.b1 = fma2(m.b1, a1[r], b1);
      }
#pragma unroll
      for (int r = kBwdRows - 1; r >= 0; --r) {
        float2 o0, o1;
        unpack4(douts + r * pitch, o0, o1);
        if (r < left) {
          e0 = mul2(a0[r], add2(e0, o0));
          e1 = mul2(a1[r], add2(e1, o1));
        }
      }
      float4* to = reinterpret_cast<float4*>(&sm.map[buf][warp][4 * lane]);
      to[0] = make_float4(m.a0.x, m.b0.x, m.a0.y, m.b0.y);
      to[1] = make_float4(m.a1.x, m.b1.x, m.a1.y, m.b1.y);
      *reinterpret_cast<float4*>(&sm.rev[buf][warp][4 * lane]) = make_float4(e0.x, e0.y, e1.x, e1.y);
      __syncwarp();
      if (lane == 0) sm100::mbar_arrive(sm100::smem_addr(&sm.mapped[par]));
      next_bt = beta_fast(later_beta, prob);
      later_beta = load_beta(step + 2);
    };
    const bool lane_in = 4 * lane < d, wide = vec_grad && lane_in;
    auto finish = [&](int step, const Kept& k) {
      const int stage = step % kStages, par = step & 1, buf = kAhead ? par : 0;
      if (step > 0) {  // the last step's gradients have left shared memory: its tile may be replaced
        if (lane == 0) {
          sm100::bulk_wait_read_all();
          sm100::mbar_arrive(sm100::smem_addr(&sm.done[(step - 1) & 1]));
        }
        __syncwarp();
      }
      wait(&sm.entered[par], step >> 1);
      const int tile = tile_of(step), left = tile >= 0 ? n - tile * kTile - row0 : 0;
      const float4* from = reinterpret_cast<const float4*>(&sm.map[buf][warp][4 * lane]);
      const float4 lo = from[0], hi = from[1];
      if (left <= 0) return;
      float2 h0 = make_float2(lo.x, lo.z), h1 = make_float2(hi.x, hi.z);
      float2 back0 = make_float2(lo.y, lo.w), back1 = make_float2(hi.y, hi.w);
      TX* xs = sm.x[stage] + row0 * pitch + 4 * lane;
      TR* raws = sm.raw[stage] + row0 * pitch + 4 * lane;
      const TO* douts = sm.dout[stage] + row0 * pitch + 4 * lane;
      const size_t at = first + (size_t)(tile * kTile + row0) * row;
      // states before each token
      float2 before[kBwdRows][2];
#pragma unroll
      for (int r = 0; r < kBwdRows; ++r) {
        before[r][0] = h0;
        before[r][1] = h1;
        if (r + 1 < kBwdRows) {
          const float bt_r = __shfl_sync(0xffffffffu, k.bt, r);
          float2 x0, x1;
          unpack4(xs + r * pitch, x0, x1);
          const Decay d0 = decay_of(k.g0[r]), d1 = decay_of(k.g1[r]);
          h0 = fma2(d0.a, h0, input(x0, bt_r, d0));
          h1 = fma2(d1.a, h1, input(x1, bt_r, d1));
        }
      }
      float dots[kBwdRows];
      const bool copied = by_copy && left >= kBwdRows;
#pragma unroll
      for (int r = kBwdRows - 1; r >= 0; --r) {
        dots[r] = 0.f;
        const float bt_r = __shfl_sync(0xffffffffu, k.bt, r);
        if (r >= left) continue;
        float2 z0, z1, x0, x1, D0, D1;
        unpack4(raws + r * pitch, z0, z1);
        unpack4(xs + r * pitch, x0, x1);
        unpack4(douts + r * pitch, D0, D1);
        const Decay d0 = decay_of(k.g0[r]), d1 = decay_of(k.g1[r]);
        const float2 a0 = d0.a, a1 = d1.a;
        D0 = add2(D0, back0);
        D1 = add2(D1, back1);
        back0 = mul2(a0, D0);
        back1 = mul2(a1, D1);
        float2 dg0 = mul2(back0, before[r][0]), dg1 = mul2(back1, before[r][1]);  // D a h_{t-1}
        float2 xs0 = mul2(D0, x0), xs1 = mul2(D1, x1);                  // D x, times s for dbeta
        float2 dx0 = mul2(D0, both(bt_r)), dx1 = mul2(D1, both(bt_r));
        if constexpr (kNorm) {
          const float2 u0 = one_minus_sq(d0), u1 = one_minus_sq(d1);
          const float2 i0 = rsq2(u0), i1 = rsq2(u1), s0v = mul2(u0, i0), s1v = mul2(u1, i1);
          // ds/dg = -a^2 / s
          dg0 = fma2(mul2(xs0, both(-bt_r)), mul2(mul2(a0, a0), i0), dg0);
          dg1 = fma2(mul2(xs1, both(-bt_r)), mul2(mul2(a1, a1), i1), dg1);
          xs0 = mul2(xs0, s0v);
          xs1 = mul2(xs1, s1v);
          dx0 = mul2(dx0, s0v);
          dx1 = mul2(dx1, s1v);
        }
        if constexpr (kSafe) {  // a clamped gate passes no gradient
          dg0 = make_float2(k.g0[r].x > gate.lb2 ? dg0.x : 0.f, k.g0[r].y > gate.lb2 ? dg0.y : 0.f);
          dg1 = make_float2(k.g1[r].x > gate.lb2 ? dg1.x : 0.f, k.g1[r].y > gate.lb2 ? dg1.y : 0.f);
        }
        sum_log = fma2(dg0, k.g0[r], sum_log);
        sum_log = fma2(dg1, k.g1[r], sum_log);
        z0 = pre_log2(z0, bias0);
        z1 = pre_log2(z1, bias1);
        auto sigmoid = [](float z2) { return rcp(1.f + ex2(-z2)); };  // z2 in units of log2
        const float2 dr0 = mul2(mul2(dg0, both(gate.c)), make_float2(sigmoid(z0.x), sigmoid(z0.y)));
        const float2 dr1 = mul2(mul2(dg1, both(gate.c)), make_float2(sigmoid(z1.x), sigmoid(z1.y)));
        sum_bias0 = add2(sum_bias0, dr0);
        sum_bias1 = add2(sum_bias1, dr1);
        dots[r] = lane_in ? (xs0.x + xs0.y) + (xs1.x + xs1.y) : 0.f;
        if (copied) {
          if (lane_in) {
            store4(xs + r * pitch, dx0, dx1);
            store4(raws + r * pitch, dr0, dr1);
          }
        } else if (wide) {
          store4(reinterpret_cast<TX*>(p.dx) + at + r * row + 4 * lane, dx0, dx1);
          store4(reinterpret_cast<TR*>(p.draw) + at + r * row + 4 * lane, dr0, dr1);
        } else if (!vec_grad) {
          put4(reinterpret_cast<TX*>(p.dx) + at + r * row, d, lane, dx0, dx1, false);
          put4(reinterpret_cast<TR*>(p.draw) + at + r * row, d, lane, dr0, dr1, false);
        }
      }
      if (copied) {
        sm100::fence_async_smem();
        __syncwarp();
        if (lane == 0) {
          const int t = s0 + tile * kTile + row0;
          sm100::tma_store_3d(&maps.dx, sm100::smem_addr(sm.x[stage] + row0 * pitch), 0, h, t);
          sm100::tma_store_3d(&maps.draw, sm100::smem_addr(sm.raw[stage] + row0 * pitch), 0, h, t);
          sm100::bulk_commit();
        }
      }
      // ---- dbeta of the warp's four tokens: halves of the lanes take two each, quarters one
      static_assert(kBwdRows == 4, "the reduction is written for four tokens");
      const bool upper = lane & 16, odd = lane & 8;
      float u = (upper ? dots[2] : dots[0]) + __shfl_xor_sync(0xffffffffu, upper ? dots[0] : dots[2], 16);
      float v = (upper ? dots[3] : dots[1]) + __shfl_xor_sync(0xffffffffu, upper ? dots[1] : dots[3], 16);
      float w = (odd ? v : u) + __shfl_xor_sync(0xffffffffu, odd ? u : v, 8);
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
      const int r = lane >> 3;
      const float bt_r = __shfl_sync(0xffffffffu, k.bt, r);
      if ((lane & 7) == 0 && r < left)
        p.dbeta[(size_t)(s0 + tile * kTile + row0 + r) * p.H + h] = prob ? w : w * bt_r * (1.f - bt_r);
    };
    if constexpr (kAhead) {
      Kept even, odd;
      work_out(0, even);
      for (int step = 0; step < steps; step += 2) {
        if (step + 1 < steps) work_out(step + 1, odd);
        finish(step, even);
        if (step + 1 >= steps) break;
        if (step + 2 < steps) work_out(step + 2, even);
        finish(step + 1, odd);
      }
    } else {
      Kept k;
      for (int step = 0; step < steps; ++step) {
        work_out(step, k);
        finish(step, k);
        if (how != kTensor) {
          __syncwarp();
          copy(step + kStages - 1);
        }
      }
    }
    __syncwarp();
    sm100::cluster_arrive_relaxed();  // a computing warp touches no other CTA's memory
    sm100::bulk_wait_all();
    // ---- the warp's share of the parameters' gradients
    float* red = &sm.rev[0][0][0];  // [warps][kRow]
    named_barrier_sync<1, 32 * kBwdWarps>();  // the carrying warps have read the last step's (it has been entered)
    *reinterpret_cast<float4*>(red + warp * kRow + 4 * lane) = make_float4(sum_bias0.x, sum_bias0.y, sum_bias1.x, sum_bias1.y);
    float lg = lane_in ? sum_log.x + sum_log.y : 0.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) lg += __shfl_xor_sync(0xffffffffu, lg, o);
    float* red_log = reinterpret_cast<float*>(&sm.map[0][0][0]);
    if (lane == 0) red_log[warp] = lg;
    named_barrier_sync<1, 32 * kBwdWarps>();
    for (int i = threadIdx.x; i <= d; i += 32 * kBwdWarps) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < kBwdWarps; ++w) s += i < d ? red[w * kRow + i] : red_log[w];
      part[i] = i < d ? s : s * kLn2;  // the last one: dg g, g having been kept times log2 e
    }
  }
  __syncwarp();
  sm100::cluster_wait();
}

// ddt_bias and da_log from the partial sums: one warp per (head, channel or the head's own sum),
// lanes over the parts, joined in a fixed order; in 64 bits, since many parts may cancel.
__global__ void glr_bwd_sum_kernel(const float* partial, int parts, int H, int d, float* da_log, float* ddt_bias) {
  const int64_t i = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  if (i >= (int64_t)H * (d + 1)) return;
  const int lane = threadIdx.x & 31;
  double s = 0.0;
  for (int k = lane; k < parts; k += 32) s += (double)partial[(size_t)k * H * (d + 1) + i];
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (lane == 0) {
    const int h = (int)(i / (d + 1)), c = (int)(i - (int64_t)h * (d + 1));
    if (c < d) ddt_bias[(size_t)h * d + c] = (float)s;
    else da_log[h] = (float)s;
  }
}

// ------------------------------------------------------------------------------------ one token

constexpr int kDecThreads = 128;

// A thread takes one channel, or four where rows allow it: every state element is read and written
// once, next to which the token's inputs are a third.
template <typename TX, typename TR, int kPer>
__global__ void __launch_bounds__(kDecThreads) glr_decode_kernel(const GlrArgs p) {
  const int64_t i = ((int64_t)blockIdx.x * kDecThreads + threadIdx.x) * kPer;  // element of [batch][H][d]
  const int64_t total = (int64_t)p.batch * p.H * p.d;
  if (i >= total) return;
  const int64_t bh = i / p.d;
  const int c = (int)(i - bh * p.d), h = (int)(bh % p.H);
  const int64_t b = bh / p.H;
  const int32_t slot = p.slots[b];
  if (slot < 0 || slot >= p.max_slots) {
    report(p.status, KDA_ERR_DEVICE_CHECK);
    return;
  }
  float* state = p.pool + ((size_t)slot * p.H + h) * p.d + c;
  const TX* x = reinterpret_cast<const TX*>(p.x) + i;
  const TR* raw = reinterpret_cast<const TR*>(p.raw_gate) + i;
  const float* bias = p.dt_bias + (size_t)h * p.d + c;
  float2 s0{}, s1{}, x0{}, x1{}, z0{}, z1{}, v0{}, v1{};
  if constexpr (kPer == 4) {
    unpack4(state, s0, s1);
    unpack4(x, x0, x1);
    unpack4(raw, z0, z1);
    unpack4(bias, v0, v1);
  } else {
    s0.x = *state;
    x0.x = to_f32(*x);
    z0.x = to_f32(*raw);
    v0.x = *bias;
  }
  const HeadGate gate = head_gate(p.a_log[h], p.flags & KDA_GATE_SAFE, p.lb);
  const float bt = beta_f32(p.beta[bh], p.flags & KDA_BETA_PROB);
  auto step = [&](float2 s, float2 xv, float2 z) {
    const float2 g = clamp2(gate_log2(z, exp_neg_abs(z), gate.c), gate.lb2);
    const Decay e = decay_of(g);
    float2 in = mul2(xv, both(bt));
    if (p.flags & KDA_INPUT_NORM) {
      const float2 u = one_minus_sq(e);
      in = mul2(in, mul2(u, rsq2(u)));
    }
    return fma2(e.a, s, in);
  };
  s0 = step(s0, x0, pre_log2(z0, mul2(v0, both(kLog2e))));
  if constexpr (kPer == 4) {
    s1 = step(s1, x1, pre_log2(z1, mul2(v1, both(kLog2e))));
    store4(state, s0, s1);
    if (p.out_bf16) store4(reinterpret_cast<__nv_bfloat16*>(p.out) + i, s0, s1);
    else store4(reinterpret_cast<float*>(p.out) + i, s0, s1);
  } else {
    *state = s0.x;
    store_out(p.out, i, s0.x, p.out_bf16);
  }
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// CTAs per (sequence, head).  One fits an SM at a time, so c of them make ceil(chains c / SMs) rounds of
// 1 / c of a chain; sequences of unequal lengths leave about one more round half empty, and each CTA of a
// cluster adds some 4 % to a step.  One sequence of 131072 tokens and 32 heads, forward / backward: 1 CTA
// 3569 / 14306 us, 2: 1801 / 7124, 4: 919 / 3426, 8: 1407 / 5146; the rule
// takes 4.  8 packed sequences (32768 tokens): 1: 297 / 761, 2: 225 / 554, 4 (4 at most backwards): 251 / 589, 8: 325;
// the rule takes 4 here too, 11 % and 6 % above the best.
int cluster_size(int32_t batch, int64_t T, int32_t H, int most) {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t tiles = (T / batch + kTile - 1) / kTile, chains = (int64_t)batch * H;
  int best = 1;
  double least = 0;
  for (int c = 1; c <= most && (c == 1 || c <= tiles); c *= 2) {
    const double cost = (double)((chains * c + sms - 1) / sms + (batch > 1)) / c * (1 + 0.04 * c);
    if (c == 1 || cost < least) {
      best = c;
      least = cost;
    }
  }
  return best;
}

template <typename Kernel, typename... Args>
cudaError_t launch_cluster(Kernel kernel, unsigned grid, int threads, size_t smem, int ranks, cudaStream_t stream,
                           Args... args) {
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// how rows of d elements of the given tensors can be copied to shared memory
template <typename T>
Access access_of(const void* p, int d) {
  if (d * sizeof(T) % 16 == 0 && aligned(p, 16)) return kTensor;
  if (d % 4 == 0 && aligned(p, 4 * sizeof(T))) return kVec4;
  return (d * sizeof(T)) % 4 == 0 && aligned(p, 4) ? kWord : kElem;
}
Access worse(Access a, Access b) { return a > b ? a : b; }

// [tokens][heads][d] in boxes of one head of so many tokens
template <typename T>
bool encode(CUtensorMap* m, const void* base, int64_t tokens, int heads, int d, int rows = kTile) {
  using Fn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                          const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                          CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Fn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                   q == cudaDriverEntryPointSuccess
               ? reinterpret_cast<Fn>(p)
               : nullptr;
  }();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * sizeof(T), (cuuint64_t)heads * d * sizeof(T)};
  const cuuint32_t box[3] = {(cuuint32_t)d, 1, (cuuint32_t)rows}, each[3] = {1, 1, 1};
  return fn(m, sizeof(T) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3,
            const_cast<void*>(base), dims, strides, box, each, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename TX, typename TR, typename TO>
cudaError_t fwd(const GlrArgs& a, cudaStream_t stream) {
  Access how = worse(access_of<TX>(a.x, a.d), access_of<TR>(a.raw_gate, a.d));
  Maps maps{};
  if (how == kTensor && (a.total_tokens == 0 || !encode<TX>(&maps.x, a.x, a.total_tokens, a.H, a.d) ||
                         !encode<TR>(&maps.raw, a.raw_gate, a.total_tokens, a.H, a.d)))
    how = kVec4;
  const bool out_map = access_of<TO>(a.out, a.d) == kTensor && a.total_tokens > 0 &&
                       encode<TO>(&maps.out, a.out, a.total_tokens, a.H, a.d, kFwdRows);
  const bool vec_out = a.d % 4 == 0 && aligned(a.out, 4 * sizeof(TO));
  const int ranks = cluster_size(a.batch, a.total_tokens, a.H, FwdSmem<TX, TR, TO>::kMaxRanks);
  const int64_t grid = (int64_t)a.batch * a.H * ranks;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const size_t smem = sizeof(FwdSmem<TX, TR, TO>);
  const bool norm = a.flags & KDA_INPUT_NORM, safe = a.flags & KDA_GATE_SAFE;
  const auto kernel = norm ? (safe ? glr_fwd_kernel<TX, TR, TO, true, true> : glr_fwd_kernel<TX, TR, TO, true, false>)
                           : (safe ? glr_fwd_kernel<TX, TR, TO, false, true> : glr_fwd_kernel<TX, TR, TO, false, false>);
  // the warps' shares come out of what a CTA is launched with: with less, they would wait for good
  cudaFuncAttributes built;
  const cudaError_t e = cudaFuncGetAttributes(&built, kernel);
  if (e != cudaSuccess) return e;
  if (built.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  return launch_cluster(kernel, (unsigned)grid, kFwdThreads, smem, ranks, stream, a, maps, how, out_map, vec_out);
}

template <typename TX, typename TR, typename TO>
cudaError_t bwd(const GlrBwdArgs& a, cudaStream_t stream) {
  Access how = worse(worse(access_of<TX>(a.x, a.d), access_of<TR>(a.raw_gate, a.d)), access_of<TO>(a.dout, a.d));
  BwdMaps maps{};
  const int64_t T = a.total_tokens;
  if (how == kTensor && (T == 0 || !encode<TX>(&maps.x, a.x, T, a.H, a.d) || !encode<TR>(&maps.raw, a.raw_gate, T, a.H, a.d) ||
                         !encode<TO>(&maps.dout, a.dout, T, a.H, a.d)))
    how = kVec4;
  // a warp's rows leave by tensor copies where they also start on 128 bytes of shared memory
  const bool by_copy = how == kTensor && access_of<TX>(a.dx, a.d) == kTensor && access_of<TR>(a.draw, a.d) == kTensor &&
                       kBwdRows * a.d * sizeof(TX) % 128 == 0 && kBwdRows * a.d * sizeof(TR) % 128 == 0 &&
                       encode<TX>(&maps.dx, a.dx, T, a.H, a.d, kBwdRows) && encode<TR>(&maps.draw, a.draw, T, a.H, a.d, kBwdRows);
  const bool vec_grad = a.d % 4 == 0 && aligned(a.dx, 4 * sizeof(TX)) && aligned(a.draw, 4 * sizeof(TR));
  const int ranks = cluster_size(a.batch, a.total_tokens, a.H, BwdSmem<TX, TR, TO>::kMaxRanks);
  const int64_t grid = (int64_t)a.batch * a.H * ranks;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const size_t smem = sizeof(BwdSmem<TX, TR, TO>);
  static_assert(sizeof(BwdSmem<TX, TR, TO>) <= 227 * 1024 && sizeof(FwdSmem<TX, TR, TO>) <= 227 * 1024, "");
  const bool norm = a.flags & KDA_INPUT_NORM, safe = a.flags & KDA_GATE_SAFE;
  const auto kernel = norm ? (safe ? glr_bwd_kernel<TX, TR, TO, true, true> : glr_bwd_kernel<TX, TR, TO, true, false>)
                           : (safe ? glr_bwd_kernel<TX, TR, TO, false, true> : glr_bwd_kernel<TX, TR, TO, false, false>);
  cudaError_t e = launch_cluster(kernel, (unsigned)grid, kBwdThreads, smem, ranks, stream, a, maps, how, by_copy, vec_grad);
  if (e != cudaSuccess) return e;
  const int64_t sums = (int64_t)a.H * (a.d + 1);
  glr_bwd_sum_kernel<<<(unsigned)((sums * 32 + 255) / 256), 256, 0, stream>>>(a.partial, a.batch * ranks, a.H, a.d,
                                                                             a.da_log, a.ddt_bias);
  return cudaGetLastError();
}

template <typename TX, typename TR>
cudaError_t decode(const GlrArgs& a, cudaStream_t stream) {
  const bool vec = a.d % 4 == 0 && aligned(a.x, 4 * sizeof(TX)) && aligned(a.raw_gate, 4 * sizeof(TR)) &&
                   aligned(a.pool, 16) && aligned(a.dt_bias, 16) && aligned(a.out, a.out_bf16 ? 8 : 16);
  const int64_t n = (int64_t)a.batch * a.H * a.d / (vec ? 4 : 1);
  const unsigned grid = (unsigned)((n + kDecThreads - 1) / kDecThreads);
  if (vec) glr_decode_kernel<TX, TR, 4><<<grid, kDecThreads, 0, stream>>>(a);
  else glr_decode_kernel<TX, TR, 1><<<grid, kDecThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

int glr_bwd_partials(int32_t batch, int64_t total_tokens, int32_t H) {
  return batch * cluster_size(batch, total_tokens, H, kMaxCluster);
}

cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t stream) {
  using bf16 = __nv_bfloat16;
  if (!a.x_bf16) return fwd<float, float, float>(a, stream);
  if (a.raw_bf16) return a.out_bf16 ? fwd<bf16, bf16, bf16>(a, stream) : fwd<bf16, bf16, float>(a, stream);
  return a.out_bf16 ? fwd<bf16, float, bf16>(a, stream) : fwd<bf16, float, float>(a, stream);
}

cudaError_t launch_glr_bwd(const GlrBwdArgs& a, cudaStream_t stream) {
  using bf16 = __nv_bfloat16;
  if (!a.x_bf16) return bwd<float, float, float>(a, stream);
  if (a.raw_bf16) return a.dout_bf16 ? bwd<bf16, bf16, bf16>(a, stream) : bwd<bf16, bf16, float>(a, stream);
  return a.dout_bf16 ? bwd<bf16, float, bf16>(a, stream) : bwd<bf16, float, float>(a, stream);
}

cudaError_t launch_glr_decode(const GlrArgs& a, cudaStream_t stream) {
  if (!a.x_bf16) return decode<float, float>(a, stream);
  return a.raw_bf16 ? decode<__nv_bfloat16, __nv_bfloat16>(a, stream) : decode<__nv_bfloat16, float>(a, stream);
}

}  // namespace kda
