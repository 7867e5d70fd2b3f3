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
// Work per element is a few dozen instructions against 6 to 10 bytes, so the passes are bound by
// HBM as long as every input is read once.  A scan needs no second reading when whoever reads a
// tile also finishes it: a cluster of CTAs walks along one (sequence, head), each CTA taking every
// cluster-size-th tile of 64 tokens x d channels.  Inside the CTA a warp holds consecutive tokens
// (a lane: four channels), reduces them to one affine map h -> A h + B per channel, and the maps
// are folded in token order: over the warps through shared memory, over the cluster's tiles
// through distributed shared memory.  Every CTA folds the same maps in the same order, so results
// do not depend on timing, and the carry never goes through global memory.
//
// The backward pass walks the tiles in reverse.  The forward pass has kept the state entering each
// tile (1/64 of the fp32 size of the outputs), so h_{t-1} is rebuilt inside the tile and only D is
// carried.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cstddef>

#include "kda_glr_math.cuh"
#include "kda_ops_internal.h"
#include "kda_sm100.cuh"

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

// A warp's affine maps of its lanes' four channels in shared memory: A then B.
struct Map4 {
  float2 a0, a1, b0, b1;
};
struct MapRow {
  float a[kRow], b[kRow];
};
__device__ __forceinline__ Map4 read_map(const MapRow& r, int lane) {
  const float4 a = *reinterpret_cast<const float4*>(r.a + 4 * lane);
  const float4 b = *reinterpret_cast<const float4*>(r.b + 4 * lane);
  return {make_float2(a.x, a.y), make_float2(a.z, a.w), make_float2(b.x, b.y), make_float2(b.z, b.w)};
}
__device__ __forceinline__ void write_map(MapRow& r, int lane, const Map4& m) {
  *reinterpret_cast<float4*>(r.a + 4 * lane) = make_float4(m.a0.x, m.a0.y, m.a1.x, m.a1.y);
  *reinterpret_cast<float4*>(r.b + 4 * lane) = make_float4(m.b0.x, m.b0.y, m.b1.x, m.b1.y);
}

// The sequence of this cluster; false (reported) if its offsets or slot are out of range.
__device__ __forceinline__ bool sequence(const int32_t* cu, int b, int64_t T, int32_t& s0, int32_t& n) {
  s0 = cu[b];
  n = cu[b + 1] - s0;
  return s0 >= 0 && n >= 0 && (int64_t)s0 + n <= T;
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
  }
  cluster.sync();
  auto wait = [&](uint64_t* bar, int parity) {
    if (!sm100::mbar_wait_sleep(sm100::smem_addr(bar), parity & 1, kWaitNs)) report(p.status, KDA_ERR_DEVICE_TIMEOUT);
  };

  const int pitch = how == kTensor ? d : kRow;  // elements of a tile's row

  if (warp >= kFwdWarps) {
    // ---------------------------------------------------------------- carrying warps
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
    float* state = p.pool + ((size_t)slot * p.H + h) * d;
    float carry = c < d ? state[c] : 0.f;
    for (int step = 0; step < steps; ++step) {
      const int par = step & 1;
      wait(&sm.mapped[par], step >> 1);
      float2 of[kFwdWarps];
      float pa = 1.f, pb = 0.f;
#pragma unroll
      for (int w = 0; w < kFwdWarps; ++w) of[w] = sm.map[par][w][c];
#pragma unroll
      for (int w = 0; w < kFwdWarps; ++w) {
        pb = fmaf(pb, of[w].x, of[w].y);
        pa *= of[w].x;
      }
      for (int k = 0; k < ranks; ++k) send_map(&sm.tile_map[par][rank][c], &sm.tiles_in[par], k, pa, pb);
      if (c == 0)
        sm100::mbar_arrive_expect_tx(sm100::smem_addr(&sm.tiles_in[par]), ranks * kRow * (uint32_t)sizeof(float2));
      fetch(step + kStages);  // into the tile that has just been read
      wait(&sm.tiles_in[par], step >> 1);
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
    if (rank == 0 && c < d) state[c] = carry;
    return;
  }

  // ------------------------------------------------------------------ computing warps
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
      k.a0[r] = make_float2(ex2(g0.x), ex2(g0.y));
      k.a1[r] = make_float2(ex2(g1.x), ex2(g1.y));
      k.b0[r] = mul2(x0, both(bt_r));
      k.b1[r] = mul2(x1, both(bt_r));
      if constexpr (kNorm) {
        const float2 u0 = one_minus_sq(g0, k.a0[r]), u1 = one_minus_sq(g1, k.a1[r]);
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
    wait(&sm.entered[par], step >> 1);
    const float4* from = reinterpret_cast<const float4*>(&sm.map[par][warp][4 * lane]);
    const float4 lo = from[0], hi = from[1];
    float2 in0 = make_float2(lo.x, lo.z), in1 = make_float2(hi.x, hi.z);
    const bool copied = out_map && left >= kFwdRows;
    if (copied) {
      sm100::bulk_wait_read_all();  // (the issuing lane's) the rows have left
      __syncwarp();
    }
    TO* to = out + (size_t)tile * kTile * row;
#pragma unroll
    for (int r = 0; r < kFwdRows; ++r, to += row) {
      in0 = fma2(k.a0[r], in0, k.b0[r]);
      in1 = fma2(k.a1[r], in1, k.b1[r]);
      if (copied) {
        if (4 * lane < d) store4(staged + r * d + 4 * lane, in0, in1);
      } else if (r < left) {
        put4(to, d, lane, in0, in1, vec_out);
      }
    }
    if (copied) {
      sm100::fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        sm100::tma_store_3d(&maps.out, sm100::smem_addr(staged), 0, h, s0 + tile * kTile + row0);
        sm100::bulk_commit();
      }
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
  sm100::bulk_wait_all();
}

// ------------------------------------------------------------------------------------ backward

constexpr int kBwdThreads = 512;
constexpr int kBwdWarps = kBwdThreads / 32;
constexpr int kBwdRows = kTile / kBwdWarps;

template <typename TX, typename TR, typename TO>
struct BwdSmem {
  static constexpr int kStages = sizeof(TX) + sizeof(TR) + sizeof(TO) <= 6 ? 3 : 2;
  static constexpr int kMaxRanks = sizeof(TX) == 4 ? kMaxCluster / 2 : kMaxCluster;  // what fits
  TX x[kStages][kTile][kRow];
  TR raw[kStages][kTile][kRow];
  TO dout[kStages][kTile][kRow];
  float beta[kStages][kTile];
  MapRow fwd_map[kBwdWarps];     // of h through a warp's tokens
  float rev_b[kBwdWarps][kRow];  // of a_t D_t back through them (the same A)
  MapRow tile_map[2][kMaxRanks];
};

template <typename TX, typename TR, typename TO, bool kNorm>
__global__ void __launch_bounds__(kBwdThreads, 1)
    glr_bwd_kernel(const GlrBwdArgs p, const Access how, const bool vec_grad) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  using Smem = BwdSmem<TX, TR, TO>;
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  constexpr int kStages = Smem::kStages;

  const cg::cluster_group cluster = cg::this_cluster();
  const int ranks = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int chain = blockIdx.x / ranks, b = chain / p.H, h = chain - b * p.H;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = p.d;

  // partial sums of the parameters' gradients, one set per (sequence, rank)
  float* part_bias = p.partial + ((size_t)(b * ranks + rank) * p.H + h) * (d + 1);
  int32_t s0, n;
  const bool ok = sequence(p.cu, b, p.total_tokens, s0, n);
  if (!ok || n == 0) {
    if (!ok && threadIdx.x == 0) report(p.status, KDA_ERR_DEVICE_CHECK);
    for (int c = threadIdx.x; c <= d; c += kBwdThreads) part_bias[c] = 0.f;
    if (ok && rank == 0)  // the state only passes through an empty sequence
      for (int c = threadIdx.x; c < d; c += kBwdThreads) {
        const size_t at = ((size_t)b * p.H + h) * d + c;
        p.d_initial[at] = p.d_final ? p.d_final[at] : 0.f;
      }
    return;
  }
  const float a_log = p.a_log[h];
  const HeadGate gate = head_gate(a_log, p.flags & KDA_GATE_SAFE, p.lb);
  const bool prob = p.flags & KDA_BETA_PROB;
  float2 bias0, bias1, c0 = both(0.f), c1 = both(0.f);  // c: a D of the token after the cluster's tiles
  load4(p.dt_bias + (size_t)h * d, d, lane, bias0, bias1);
  bias0 = mul2(bias0, both(kLog2e));
  bias1 = mul2(bias1, both(kLog2e));
  if (p.d_final) load4(p.d_final + ((size_t)b * p.H + h) * d, d, lane, c0, c1);

  const size_t row = (size_t)p.H * d;
  const size_t first = (size_t)s0 * row + (size_t)h * d;
  const TX* x = reinterpret_cast<const TX*>(p.x) + first;
  const TR* raw = reinterpret_cast<const TR*>(p.raw_gate) + first;
  const TO* dout = reinterpret_cast<const TO*>(p.dout) + first;
  const float* beta = p.beta + (size_t)s0 * p.H + h;
  const float* kept = p.checkpoints + ((size_t)(s0 / kTile + b) * p.H + h) * d;
  const int tiles = (n + kTile - 1) / kTile, steps = (tiles + ranks - 1) / ranks;

  // step 0 takes the last tiles; rank k the k-th from the end of the step's
  auto tile_of = [&](int step) { return tiles - 1 - (step * ranks + rank); };
  auto fetch = [&](int step) {
    const int stage = step % kStages, tile = tile_of(step), t0 = tile * kTile + warp * kBwdRows;
    if (step < steps && tile >= 0) {
#pragma unroll
      for (int r = 0; r < kBwdRows; ++r) {
        if (t0 + r < n) {
          copy_row(sm.x[stage][warp * kBwdRows + r], x + (t0 + r) * row, d, lane, how);
          copy_row(sm.raw[stage][warp * kBwdRows + r], raw + (t0 + r) * row, d, lane, how);
          copy_row(sm.dout[stage][warp * kBwdRows + r], dout + (t0 + r) * row, d, lane, how);
        }
      }
      if (lane < kBwdRows && t0 + lane < n)
        cp_async<4>(&sm.beta[stage][warp * kBwdRows + lane], beta + (size_t)(t0 + lane) * p.H);
    }
    cp_async_commit();
  };
  if (d < kRow) {  // channels past the head must add nothing to the sums over channels
    static_assert(offsetof(Smem, beta) % 16 == 0, "the inputs are cleared in words of 16 bytes");
    for (size_t i = threadIdx.x; i < offsetof(Smem, beta) / 16; i += kBwdThreads)
      reinterpret_cast<uint4*>(&sm)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) fetch(s);

  float2 sum_bias0 = both(0.f), sum_bias1 = both(0.f), sum_log = both(0.f);
  const float2 one = both(1.f), zero = both(0.f);

  for (int step = 0; step < steps; ++step) {
    __syncwarp();  // the stage that is filled next has been read
    fetch(step + kStages - 1);
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const int stage = step % kStages, par = step & 1;
    const int tile = tile_of(step), t0 = tile * kTile + warp * kBwdRows;
    const bool some = tile >= 0;
    float2 in0 = zero, in1 = zero;  // the state entering the tile
    if (some) load4(kept + (size_t)tile * row, d, lane, in0, in1);

    // ---- gates, inputs and this warp's maps, forwards and backwards
    float bt = 0.f;
    if (lane < kBwdRows) bt = beta_f32(sm.beta[stage][warp * kBwdRows + lane], prob);
    float2 g0[kBwdRows], g1[kBwdRows], a0[kBwdRows], a1[kBwdRows], b0[kBwdRows], b1[kBwdRows];
    float2 q0[kBwdRows], q1[kBwdRows];  // s and, with the normalised input, what ds/dg needs
    Map4 mine{one, one, zero, zero};
#pragma unroll
    for (int r = 0; r < kBwdRows; ++r) {
      const float bt_r = __shfl_sync(0xffffffffu, bt, r);
      a0[r] = a1[r] = one;
      b0[r] = b1[r] = zero;
      if (some && t0 + r < n) {
        float2 z0, z1, x0, x1;
        unpack4(&sm.raw[stage][warp * kBwdRows + r][4 * lane], z0, z1);
        unpack4(&sm.x[stage][warp * kBwdRows + r][4 * lane], x0, x1);
        z0 = pre_log2(z0, bias0);
        z1 = pre_log2(z1, bias1);
        g0[r] = gate_log2(z0, exp_neg_abs(z0), gate.c);
        g1[r] = gate_log2(z1, exp_neg_abs(z1), gate.c);
        const float2 cg0 = clamp2(g0[r], gate.lb2), cg1 = clamp2(g1[r], gate.lb2);
        a0[r] = make_float2(ex2(cg0.x), ex2(cg0.y));
        a1[r] = make_float2(ex2(cg1.x), ex2(cg1.y));
        b0[r] = mul2(x0, both(bt_r));
        b1[r] = mul2(x1, both(bt_r));
        if constexpr (kNorm) {
          const float2 u0 = one_minus_sq(cg0, a0[r]), u1 = one_minus_sq(cg1, a1[r]);
          q0[r] = mul2(u0, rsq2(u0));
          q1[r] = mul2(u1, rsq2(u1));
          b0[r] = mul2(b0[r], q0[r]);
          b1[r] = mul2(b1[r], q1[r]);
        }
        mine.a0 = mul2(mine.a0, a0[r]);
        mine.a1 = mul2(mine.a1, a1[r]);
        mine.b0 = fma2(mine.b0, a0[r], b0[r]);
        mine.b1 = fma2(mine.b1, a1[r], b1[r]);
      }
    }
    float2 e0 = zero, e1 = zero;  // a_t D_t of the warp's first token, from nothing behind the warp
#pragma unroll
    for (int r = kBwdRows - 1; r >= 0; --r) {
      if (some && t0 + r < n) {
        float2 o0, o1;
        unpack4(&sm.dout[stage][warp * kBwdRows + r][4 * lane], o0, o1);
        e0 = mul2(a0[r], add2(e0, o0));
        e1 = mul2(a1[r], add2(e1, o1));
      }
    }
    write_map(sm.fwd_map[warp], lane, mine);
    *reinterpret_cast<float4*>(&sm.rev_b[warp][4 * lane]) = make_float4(e0.x, e0.y, e1.x, e1.y);
    __syncthreads();

    // ---- the state entering this warp's tokens, and what comes back from the warps behind it
    for (int w = 0; w < warp; ++w) {
      const Map4 m = read_map(sm.fwd_map[w], lane);
      in0 = fma2(m.a0, in0, m.b0);
      in1 = fma2(m.a1, in1, m.b1);
    }
    Map4 behind{one, one, zero, zero};
    auto fold_rev = [&](int w) {
      const float4 a = *reinterpret_cast<const float4*>(&sm.fwd_map[w].a[4 * lane]);
      const float4 e = *reinterpret_cast<const float4*>(&sm.rev_b[w][4 * lane]);
      const float2 wa0 = make_float2(a.x, a.y), wa1 = make_float2(a.z, a.w);
      behind.a0 = mul2(behind.a0, wa0);
      behind.a1 = mul2(behind.a1, wa1);
      behind.b0 = fma2(behind.b0, wa0, make_float2(e.x, e.y));
      behind.b1 = fma2(behind.b1, wa1, make_float2(e.z, e.w));
    };
    for (int w = kBwdWarps - 1; w > warp; --w) fold_rev(w);
    if (warp == 0) {
      const Map4 keep = behind;
      fold_rev(0);
      for (int k = 0; k < ranks; ++k) write_map(*cluster.map_shared_rank(&sm.tile_map[par][rank], k), lane, behind);
      behind = keep;
    }
    cluster.sync();
    float2 back0 = c0, back1 = c1;
    for (int k = 0; k < ranks; ++k) {
      if (k == rank) back0 = c0, back1 = c1;
      const Map4 m = read_map(sm.tile_map[par][k], lane);
      c0 = fma2(c0, m.a0, m.b0);
      c1 = fma2(c1, m.a1, m.b1);
    }
    if (!some || t0 >= n) continue;
    back0 = fma2(behind.a0, back0, behind.b0);
    back1 = fma2(behind.a1, back1, behind.b1);

    // ---- states before each token (over b, which they are made of), then the gradients backwards
#pragma unroll
    for (int r = 0; r < kBwdRows; ++r) {
      const float2 h0 = in0, h1 = in1;
      in0 = fma2(a0[r], in0, b0[r]);
      in1 = fma2(a1[r], in1, b1[r]);
      b0[r] = h0;
      b1[r] = h1;
    }
    float dots[kBwdRows];
#pragma unroll
    for (int r = kBwdRows - 1; r >= 0; --r) {
      dots[r] = 0.f;
      const float bt_r = __shfl_sync(0xffffffffu, bt, r);
      if (t0 + r >= n) continue;
      float2 z0, z1, x0, x1, D0, D1;
      unpack4(&sm.raw[stage][warp * kBwdRows + r][4 * lane], z0, z1);
      unpack4(&sm.x[stage][warp * kBwdRows + r][4 * lane], x0, x1);
      unpack4(&sm.dout[stage][warp * kBwdRows + r][4 * lane], D0, D1);
      D0 = add2(D0, back0);
      D1 = add2(D1, back1);
      back0 = mul2(a0[r], D0);
      back1 = mul2(a1[r], D1);
      float2 dg0 = mul2(back0, b0[r]), dg1 = mul2(back1, b1[r]);  // D a h_{t-1}
      float2 xs0 = mul2(D0, x0), xs1 = mul2(D1, x1);              // D x, times s for dbeta
      float2 dx0 = mul2(D0, both(bt_r)), dx1 = mul2(D1, both(bt_r));
      if constexpr (kNorm) {
        auto slope = [](float2 a, float2 s) {  // ds/dg = -a^2 / s
          return make_float2(__fdividef(-a.x * a.x, s.x), __fdividef(-a.y * a.y, s.y));
        };
        dg0 = fma2(mul2(xs0, both(bt_r)), slope(a0[r], q0[r]), dg0);
        dg1 = fma2(mul2(xs1, both(bt_r)), slope(a1[r], q1[r]), dg1);
        xs0 = mul2(xs0, q0[r]);
        xs1 = mul2(xs1, q1[r]);
        dx0 = mul2(dx0, q0[r]);
        dx1 = mul2(dx1, q1[r]);
      }
      // clamped gates pass no gradient; an infinite gate (its decay and dg are 0) counts as finite
      auto passed = [&](float dg, float g) { return g > gate.lb2 || gate.lb2 == -INFINITY ? dg : 0.f; };
      dg0 = make_float2(passed(dg0.x, g0[r].x), passed(dg0.y, g0[r].y));
      dg1 = make_float2(passed(dg1.x, g1[r].x), passed(dg1.y, g1[r].y));
      const float2 lim = both(-3.0e38f);
      sum_log = fma2(dg0, make_float2(fmaxf(g0[r].x, lim.x), fmaxf(g0[r].y, lim.y)), sum_log);
      sum_log = fma2(dg1, make_float2(fmaxf(g1[r].x, lim.x), fmaxf(g1[r].y, lim.y)), sum_log);
      z0 = pre_log2(z0, bias0);
      z1 = pre_log2(z1, bias1);
      auto sigmoid = [](float z) {  // e / (1 + e) or 1 / (1 + e) with e = exp(-|z|), z being in units of log2
        const float e = ex2(-fabsf(z));
        return (z >= 0.f ? 1.f : e) * rcp(1.f + e);
      };
      const float2 dr0 = mul2(mul2(dg0, both(gate.c)), make_float2(sigmoid(z0.x), sigmoid(z0.y)));
      const float2 dr1 = mul2(mul2(dg1, both(gate.c)), make_float2(sigmoid(z1.x), sigmoid(z1.y)));
      sum_bias0 = add2(sum_bias0, dr0);
      sum_bias1 = add2(sum_bias1, dr1);
      const int c = 4 * lane;
      dots[r] = (c < d ? xs0.x : 0.f) + (c + 1 < d ? xs0.y : 0.f) + (c + 2 < d ? xs1.x : 0.f) + (c + 3 < d ? xs1.y : 0.f);
      const size_t at = first + (size_t)(t0 + r) * row;
      put4(reinterpret_cast<TX*>(p.dx) + at, d, lane, dx0, dx1, vec_grad);
      put4(reinterpret_cast<TR*>(p.draw) + at, d, lane, dr0, dr1, vec_grad);
    }
    // ---- dbeta of the warp's tokens
#pragma unroll
    for (int r = 0; r < kBwdRows; ++r) {
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) dots[r] += __shfl_xor_sync(0xffffffffu, dots[r], o);
    }
#pragma unroll
    for (int r = 0; r < kBwdRows; ++r)
      if (lane == r && t0 + r < n)
        p.dbeta[(size_t)(s0 + t0 + r) * p.H + h] = prob ? dots[r] : dots[r] * bt * (1.f - bt);
  }
  if (rank == 0 && warp == 0) put4(p.d_initial + ((size_t)b * p.H + h) * d, d, lane, c0, c1, false);

  // ---- the CTA's share of the parameters' gradients, summed over the warps in order
  __syncthreads();
  float* red = &sm.rev_b[0][0];  // [warps][kRow]
  *reinterpret_cast<float4*>(red + warp * kRow + 4 * lane) = make_float4(sum_bias0.x, sum_bias0.y, sum_bias1.x, sum_bias1.y);
  float lg = sum_log.x + sum_log.y;
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) lg += __shfl_xor_sync(0xffffffffu, lg, o);
  float* red_log = &sm.fwd_map[0].a[0];
  if (lane == 0) red_log[warp] = lg;
  __syncthreads();
  for (int i = threadIdx.x; i <= d; i += kBwdThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kBwdWarps; ++w) s += i < d ? red[w * kRow + i] : red_log[w];
    part_bias[i] = i < d ? s : s * kLn2;  // the last one: dg g, g having been kept times log2 e
  }
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
    const float2 a = make_float2(ex2(g.x), ex2(g.y));
    float2 in = mul2(xv, both(bt));
    if (p.flags & KDA_INPUT_NORM) {
      const float2 u = one_minus_sq(g, a);
      in = mul2(in, mul2(u, rsq2(u)));
    }
    return fma2(a, s, in);
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

// CTAs per (sequence, head): the smallest power of two that gives every SM two of them, as long as
// the average sequence has a tile for each.
int cluster_size(int32_t batch, int64_t T, int32_t H, int most) {
  int dev = 0, sms = 148;
  if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const int64_t tiles = (T / batch + kTile - 1) / kTile;
  int c = 1;
  while (c < most && (int64_t)batch * H * c * 8 < 6 * sms && 2 * c <= tiles) c *= 2;
  return c;
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
  return launch_cluster(kernel, (unsigned)grid, kFwdThreads, smem, ranks, stream, a, maps, how, out_map, vec_out);
}

template <typename TX, typename TR, typename TO>
cudaError_t bwd(const GlrBwdArgs& a, cudaStream_t stream) {
  const Access how =
      worse(worse(access_of<TX>(a.x, a.d), access_of<TR>(a.raw_gate, a.d)), access_of<TO>(a.dout, a.d));
  const bool vec_grad = a.d % 4 == 0 && aligned(a.dx, 4 * sizeof(TX)) && aligned(a.draw, 4 * sizeof(TR));
  const int ranks = cluster_size(a.batch, a.total_tokens, a.H, BwdSmem<TX, TR, TO>::kMaxRanks);
  const int64_t grid = (int64_t)a.batch * a.H * ranks;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const size_t smem = sizeof(BwdSmem<TX, TR, TO>);
  const auto kernel = a.flags & KDA_INPUT_NORM ? glr_bwd_kernel<TX, TR, TO, true> : glr_bwd_kernel<TX, TR, TO, false>;
  cudaError_t e = launch_cluster(kernel, (unsigned)grid, kBwdThreads, smem, ranks, stream, a, how, vec_grad);
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
