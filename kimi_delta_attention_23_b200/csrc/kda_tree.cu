// kda_tree.cu -- KDA over a tree of drafted tokens against a state that is only read, and the
// accepted path of a tree written into that state.
//
// Let G_i be the sum of the gates on the path from the root to node i (its own included), S the
// slot's state, and j a proper ancestor of i.  Unrolling the recurrence along the path gives, with
// o for the product over key channels,
//     u_i = beta_i (v_i - (k_i o e^{G_i})^T S - sum_j A_ij u_j),   A_ij = sum_c k_ic k_jc e^{G_ic - G_jc}
//     o_i = (q_i o e^{G_i})^T S + sum_j B_ij u_j + (q_i . k_i) u_i, B_ij = sum_c q_ic k_jc e^{G_ic - G_jc}
// so no node's own state is ever formed: S is read once, all nodes' products with it are one small
// matrix product, and what the nodes do to one another is a triangular solve along the tree.
//
// One CTA per (sequence, value head):
//  1. scores: a group of lanes per node walks from the node to the root.  The decay from the ancestor
//     to the node is a running product of the tokens' decays (never an exponential of a sum, so
//     nothing over- or underflows early), which at the root is e^{G_i} itself.
//  2. P = [K o e^G; Q o e^G] S on mma.sync, S in the B fragments.  kda_tree_commit writes what comes of
//     this into fp32 states, and a good prediction k^T S all but cancels v, so the products must be as good
//     as fp32's whatever the types of the inputs and outputs: every factor is split into two tf32 parts
//     (at most 2^-22 of it is lost) and three of the four partial products are summed.
//  3. blocks of 16 nodes down the tree: a product with the deltas of the blocks before, then a thread per
//     value column substitutes within the block; a last product gives the outputs.
// The state's 4 dk dv bytes are the floor (64 requests x 16 nodes x 32 heads: 26 us; 32 x 64 nodes: 27 us).
// Measured 59 and 197 us: a small tree is a chain of short phases, and four CTAs per SM are what the
// registers allow to overlap; a 64-node tree runs as one CTA per SM, whose phases follow one another, and
// its products take 6 mma.sync of tf32 where unsplit ones would take 2.
//
// The commit is S' = e^{G_a} o S + sum over the path (k_j o e^{G_a - G_j}) u_j^T, one pass over the
// state, bound by its 8 dk dv bytes: 49 us for 64 states of 32 heads, 88 % of the copy rate.
#include "kda_glr_math.cuh"
#include "kda_ops_internal.h"
#include "kda_sm100.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256;     // of the commit
constexpr int kPitch = 132;    // floats of a node's row in shared memory
constexpr uint64_t kWaitNs = 1000000000ull;  // limit of the wait for a copy
constexpr int kPitchH = 144;   // floats of a factor's row: 64 bytes past a whole line

// Offsets and slot of a sequence; false where one is out of range.
__device__ __forceinline__ bool tree_at(const TreeArgs& a, int b, int32_t& m0, int32_t& n, int32_t& slot) {
  m0 = a.cu[b];
  n = a.cu[b + 1] - m0;
  slot = a.slots[b];
  return m0 >= 0 && n >= 0 && n <= a.max_nodes && (int64_t)m0 + n <= a.total_nodes && slot >= 0 && slot < a.max_slots;
}

// The same with the parents, which go to shared memory.  All threads call it.
__device__ __forceinline__ bool tree_of(const TreeArgs& a, int b, int32_t& m0, int32_t& n, int32_t& slot, int32_t* s_par) {
  bool ok = tree_at(a, b, m0, n, slot);
  if (ok && (int)threadIdx.x < n) {
    const int32_t par = a.parents[m0 + threadIdx.x];
    s_par[threadIdx.x] = par;
    ok = par >= -1 && par < (int)threadIdx.x;
  }
  ok = __syncthreads_and(ok);
  if (!ok && threadIdx.x == 0) report(a.status, KDA_ERR_DEVICE_CHECK);
  return ok;
}

__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// x = hi + lo up to 2^-22 of x: hi rounded to tf32's 10 bits of mantissa, which leaves at most 2^-11 of x to
// lo, of which the hardware drops what is below its own 10 bits.  In integers: the conversion instruction
// does the same for finite values and took 64 x 16 drafted tokens from 61 to 66 us, 32 x 64 from 197 to 215.
// (An x that is not a number leaves one in lo.)
__device__ __forceinline__ uint32_t round_tf32(float x) { return (__float_as_uint(x) + 0x1000u) & 0xffffe000u; }
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = round_tf32(x);
  lo = __float_as_uint(x - __uint_as_float(hi));
}

// Up to 16 nodes, four CTAs of four warps share an SM, and each reads the state straight from L2: the
// phases of so small a tree are all latency, and other CTAs are what fills it.  Beyond, the products
// carry the time: eight warps, with the state staged in shared memory.
template <int kNodes>
constexpr int kTreeThreads = kNodes <= 16 ? 128 : 256;
template <int kNodes>
constexpr bool kStaged = kNodes > 16;

template <int kNodes>
struct TreeSmem {
  // the state if it is staged (1), then (K o e^G) S and (Q o e^G) S (2), the former becoming the deltas (3)
  union {
    alignas(128) float state[kStaged<kNodes> ? 128 * 128 : 4];
    struct {
      float u[kNodes < 16 ? 16 : kNodes][128], qs[kNodes < 16 ? 16 : kNodes][128];
    };
  };
  // keys and decays (1), then the factors of the product with the state (2).  Factor rows 16 t + r:
  // key row 8 t + r for r < 8, query row 8 t + r - 8 for the others
  union {
    struct {
      float k[kNodes][kPitch], al[kNodes][kPitch];
    };
    float factor[2 * kNodes][kPitchH];
  };
  // scores, zero where j is no ancestor of i; the pitch keeps 16-byte reads of neighbouring rows apart
  static constexpr int kRows = kNodes < 16 ? 16 : kNodes;
  static constexpr int kPitchS = kRows + (kNodes == 64 ? 16 : 4);
  float a[kRows][kPitchS], b[kRows][kPitchS];
  float beta[kNodes];
  int32_t par[kNodes];
  uint64_t full;
};

// four channels of an input row of d, zero past its end.  No branches: a load whose value is converted
// inside one is waited for there, and the loads of a thread then come one after the other.
template <bool kWide, typename T>
__device__ __forceinline__ float4 load_quad(const T* row, int c, int d) {
  if constexpr (kWide) {
    float2 lo, hi;
    glr::unpack4(row + c, lo, hi);
    return make_float4(lo.x, lo.y, hi.x, hi.y);
  } else {
    float v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = glr::to_f32(row[min(c + e, d - 1)]);
    return make_float4(c < d ? v[0] : 0.f, c + 1 < d ? v[1] : 0.f, c + 2 < d ? v[2] : 0.f, c + 3 < d ? v[3] : 0.f);
  }
}

// 16 of the summed index times 8 columns of the right factor: a lane's four elements, 4 (lane % 4) .. + 3 of
// the summed index.
struct Right {
  float w[4];
  __device__ __forceinline__ void set(float s0, float s1, float s2, float s3) { w[0] = s0, w[1] = s1, w[2] = s2, w[3] = s3; }
};
// 16 rows of the left factor: rows lane / 4 and 8 further, the same four of the summed index
struct Left {
  uint32_t hi[8], lo[8];
  __device__ __forceinline__ void set(float4 x, float4 y) {
    split_tf32(x.x, hi[0], lo[0]), split_tf32(y.x, hi[1], lo[1]), split_tf32(x.y, hi[2], lo[2]), split_tf32(y.y, hi[3], lo[3]);
    split_tf32(x.z, hi[4], lo[4]), split_tf32(y.z, hi[5], lo[5]), split_tf32(x.w, hi[6], lo[6]), split_tf32(y.w, hi[7], lo[7]);
  }
};
// big + small += left right, the large and the small partial products apart
__device__ __forceinline__ void multiply(float (&big)[4], float (&small)[4], const Left& a, const Right& b) {
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const uint32_t ah[4] = {a.hi[4 * s], a.hi[4 * s + 1], a.hi[4 * s + 2], a.hi[4 * s + 3]};
    const uint32_t al[4] = {a.lo[4 * s], a.lo[4 * s + 1], a.lo[4 * s + 2], a.lo[4 * s + 3]};
    uint32_t h0, h1;
    // (volatile: split anew for every tile of rows; the parts of a whole state do not fit the registers)
    asm volatile("add.u32 %0, %1, 0x1000;" : "=r"(h0) : "r"(__float_as_uint(b.w[2 * s])));
    asm volatile("add.u32 %0, %1, 0x1000;" : "=r"(h1) : "r"(__float_as_uint(b.w[2 * s + 1])));
    h0 &= 0xffffe000u, h1 &= 0xffffe000u;
    const uint32_t l0 = __float_as_uint(b.w[2 * s] - __uint_as_float(h0));
    const uint32_t l1 = __float_as_uint(b.w[2 * s + 1] - __uint_as_float(h1));
    mma_tf32(big, ah, h0, h1);
    mma_tf32(small, al, h0, h1);
    mma_tf32(small, ah, l0, l1);
  }
}

template <int kNodes, bool kVFirst, bool kFull, typename T>
__global__ void __launch_bounds__(kTreeThreads<kNodes>, kNodes <= 16 ? 4 : kNodes <= 32 ? 2 : 1)
    tree_kernel(const TreeArgs p, const bool wide_out) {
  constexpr int kThreads = kTreeThreads<kNodes>, kWarps = kThreads / 32;
  constexpr int kCols = 8 / kWarps;  // groups of 16 value columns per warp: warp, warp + kWarps, ..
  extern __shared__ __align__(128) unsigned char smem_raw[];
  TreeSmem<kNodes>& sm = *reinterpret_cast<TreeSmem<kNodes>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / p.Hv, h = blockIdx.x - b * p.Hv, kh = h / (p.Hv / p.Hk);
  const int dk = kFull ? 128 : p.dk, dv = kFull ? 128 : p.dv;
  // every load of the nodes is on its way before the first one is waited for
  const int c4 = 4 * lane;
  const float a_log = p.a_log[h];
  const float4 bias = load_quad<kFull>(p.dt_bias + (size_t)h * dk, c4, dk);
  int32_t m0, n, slot;
  const bool there = tree_at(p, b, m0, n, slot);
  if (!there) {
    if (tid == 0) report(p.status, KDA_ERR_DEVICE_CHECK);
    return;
  }
  if (n == 0) return;
  const float* state = p.pool + ((size_t)slot * p.Hv + h) * (size_t)dk * dv;
  if constexpr (kFull && !kStaged<kNodes>) {  // the state comes while the scores are worked out
    if (tid == 0)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(state), "r"(128 * 128 * 4) : "memory");
  } else if constexpr (kFull) {
    if (tid == 0) {
      const uint32_t bar = sm100::smem_addr(&sm.full);
      sm100::mbar_init(bar, 1);
      sm100::fence_mbar_init();
      if (!(p.flags & KDA_DEBUG_WITHHOLD_HANDOFF)) {
        sm100::mbar_arrive_expect_tx(bar, sizeof(sm.state));
        sm100::bulk_g2s(sm100::smem_addr(sm.state), state, sizeof(sm.state), bar);
      }
    }
  }
  const T* qs = reinterpret_cast<const T*>(p.q) + ((size_t)m0 * p.Hk + kh) * dk;
  const T* ks = reinterpret_cast<const T*>(p.k) + ((size_t)m0 * p.Hk + kh) * dk;
  const float* raws = p.raw_gate + ((size_t)m0 * p.Hv + h) * dk;
  const size_t k_row = (size_t)p.Hk * dk, raw_row = (size_t)p.Hv * dk;
  constexpr int kGroup = kThreads / kNodes;  // lanes per node
  constexpr int kQuads = 32 / kGroup;        // float4's of channels per lane
  static_assert(kGroup <= 32 && kQuads >= 1, "");
  constexpr int kAtOnce = kNodes == 64 ? 8 : kNodes >= 32 ? 4 : kNodes / kWarps;  // rows of a warp with their loads in flight together
  const int node = tid / kGroup, g = tid % kGroup;
  const int mine = min(tid, n - 1);
  const int32_t parent = p.parents[m0 + mine];
  const float beta = p.beta[(size_t)(m0 + mine) * p.Hv + h];
  float4 kv[kAtOnce], raw[kAtOnce], qq[kQuads];
  auto load_rows = [&](int m1) {
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int m = min(m1 + kWarps * j, n - 1);
      kv[j] = load_quad<kFull>(ks + m * k_row, c4, dk);
      raw[j] = load_quad<kFull>(raws + m * raw_row, c4, dk);
    }
  };
  load_rows(warp);
#pragma unroll
  for (int j = 0; j < kQuads; ++j) {
    qq[j] = load_quad<kFull>(qs + min(node, n - 1) * k_row, 4 * (g + kGroup * j), dk);
    if (node >= n) qq[j] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int i = tid; i < (int)(sizeof(sm.a) + sizeof(sm.b)) / 16; i += kThreads)
    reinterpret_cast<float4*>(sm.a)[i] = make_float4(0.f, 0.f, 0.f, 0.f);

  // ---- keys, decays and beta of all nodes (zero keys past dk); no scores yet
  if (tid < kNodes) {
    sm.par[tid] = parent;
    sm.beta[tid] = tid < n ? beta_f32(beta, p.flags & KDA_BETA_PROB) : 0.f;
  }
  {
    const glr::HeadGate gate = glr::head_gate(a_log, p.flags & KDA_GATE_SAFE, p.lb);
    const float2 bias0 = glr::mul2(make_float2(bias.x, bias.y), glr::both(glr::kLog2e));
    const float2 bias1 = glr::mul2(make_float2(bias.z, bias.w), glr::both(glr::kLog2e));
#pragma unroll 1
    for (int m1 = warp; m1 < n; m1 += kWarps * kAtOnce) {
      if (m1 != warp) load_rows(m1);
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int m = m1 + kWarps * j;
        const float2 z0 = glr::pre_log2(make_float2(raw[j].x, raw[j].y), bias0);
        const float2 z1 = glr::pre_log2(make_float2(raw[j].z, raw[j].w), bias1);
        const float2 g0 = glr::clamp2(glr::gate_log2(z0, glr::exp_neg_abs(z0), gate.c), gate.lb2);
        const float2 g1 = glr::clamp2(glr::gate_log2(z1, glr::exp_neg_abs(z1), gate.c), gate.lb2);
        if (m < n) {
          *reinterpret_cast<float4*>(&sm.k[m][c4]) = kv[j];
          const float2 a0 = glr::decay_of(g0).a, a1 = glr::decay_of(g1).a;
          *reinterpret_cast<float4*>(&sm.al[m][c4]) = make_float4(a0.x, a0.y, a1.x, a1.y);
        }
      }
    }
  }
  auto state_there = [&] { return sm100::mbar_wait_bounded(sm100::smem_addr(&sm.full), 0, kWaitNs); };
  if (!__syncthreads_and(parent >= -1 && parent < mine)) {
    if constexpr (kFull && kStaged<kNodes>) {  // the copy in flight writes to this CTA's memory
      if (!state_there()) report(p.status, KDA_ERR_DEVICE_TIMEOUT);
    }
    if (tid == 0) report(p.status, KDA_ERR_DEVICE_CHECK);
    return;
  }

  // ---- 1. scores, and the factors of the product with the state
  {
    float4 kq[kQuads], w[kQuads];
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      w[j] = make_float4(1.f, 1.f, 1.f, 1.f);
      kq[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (node < n) kq[j] = *reinterpret_cast<const float4*>(&sm.k[node][4 * (g + kGroup * j)]);
    }
    int anc = node < n ? node : -1;
    while (__any_sync(0xffffffffu, anc >= 0)) {
      float sa = 0.f, sb = 0.f;
      if (anc >= 0) {
#pragma unroll
        for (int j = 0; j < kQuads; ++j) {
          const int c = 4 * (g + kGroup * j);
          const float4 ka = *reinterpret_cast<const float4*>(&sm.k[anc][c]);
          const float4 al = *reinterpret_cast<const float4*>(&sm.al[anc][c]);
          const float wx = w[j].x * ka.x, wy = w[j].y * ka.y, wz = w[j].z * ka.z, ww = w[j].w * ka.w;
          sa = fmaf(kq[j].x, wx, fmaf(kq[j].y, wy, fmaf(kq[j].z, wz, fmaf(kq[j].w, ww, sa))));
          sb = fmaf(qq[j].x, wx, fmaf(qq[j].y, wy, fmaf(qq[j].z, wz, fmaf(qq[j].w, ww, sb))));
          w[j] = make_float4(w[j].x * al.x, w[j].y * al.y, w[j].z * al.z, w[j].w * al.w);
        }
      }
#pragma unroll
      for (int o = kGroup / 2; o >= 1; o >>= 1) {
        sa += __shfl_xor_sync(0xffffffffu, sa, o);
        sb += __shfl_xor_sync(0xffffffffu, sb, o);
      }
      if (anc >= 0) {
        if (g == 0) {
          if (anc != node) sm.a[node][anc] = sa;
          sm.b[node][anc] = sb;
        }
        anc = sm.par[anc];
      }
    }
    __syncthreads();  // keys and decays have been read: the factors take their place
    // rows past the last node are zero: they share 16-row tiles with others
    const int rk = 16 * (node >> 3) + (node & 7);
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      const int c = 4 * (g + kGroup * j);
      const float4 kf = make_float4(kq[j].x * w[j].x, kq[j].y * w[j].y, kq[j].z * w[j].z, kq[j].w * w[j].w);
      const float4 qf = make_float4(qq[j].x * w[j].x, qq[j].y * w[j].y, qq[j].z * w[j].z, qq[j].w * w[j].w);
      *reinterpret_cast<float4*>(&sm.factor[rk][c]) = kf;
      *reinterpret_cast<float4*>(&sm.factor[rk + 8][c]) = qf;
    }
  }

  // ---- 2. the product with the state.  A warp owns 16 value columns (two n-tiles: columns
  // 16 warp + 2 (lane / 4) + {0, 1}) over all key channels.  Within each 16 channels a lane's four
  // are 4 (lane % 4) .. + 3 in both operands (the order of the summed index is free), so that its
  // share of V_FIRST states and of the factors is one wide access.
  bool late = false;
  if constexpr (kFull && kStaged<kNodes>) late = !state_there();
  const float* from = kFull && kStaged<kNodes> ? sm.state : state;
  const int q = lane & 3, gr = lane >> 2;
  auto c0 = [&](int g) { return 16 * (warp + kWarps * g) + 4 * q; };  // a lane's columns of the products
  const size_t row = (size_t)p.Hv * dv;
  const T* vs = reinterpret_cast<const T*>(p.v) + ((size_t)m0 * p.Hv + h) * dv;
  float4 v0[kCols], v8[kCols];
  auto load_values = [&](int i0) {
#pragma unroll
    for (int g = 0; g < kCols; ++g) {
      v0[g] = load_quad<kFull>(vs + min(i0 + gr, n - 1) * row, c0(g), dv);
      v8[g] = load_quad<kFull>(vs + min(i0 + gr + 8, n - 1) * row, c0(g), dv);
    }
  };
  if constexpr (kNodes == 64) load_values(0);  // where the registers allow it, ahead of the products
  // a lane's elements of the state: channels 16 ks + 4 q .. + 3 of columns 16 group + 2 gr and the next
  auto load_state = [&](int group, int ks, float (&s)[2][4]) {
    const int c = 16 * ks + 4 * q, col = 16 * group + 2 * gr;
    if constexpr (kFull && kVFirst) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const float4 v = *reinterpret_cast<const float4*>(from + (col + t) * 128 + c);
        s[t][0] = v.x, s[t][1] = v.y, s[t][2] = v.z, s[t][3] = v.w;
      }
    } else if constexpr (kFull) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = *reinterpret_cast<const float2*>(from + (c + e) * 128 + col);
        s[0][e] = v.x, s[1][e] = v.y;
      }
    } else {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          s[t][e] = c + e < dk && col + t < dv ? state[state_off(c + e, col + t, dk, dv, kVFirst)] : 0.f;
    }
  };
  auto load_factors = [&](int tile, int ks, Left& left) {
    const int c = 16 * ks + 4 * q, r = 16 * tile + gr;
    left.set(*reinterpret_cast<const float4*>(&sm.factor[r][c]), *reinterpret_cast<const float4*>(&sm.factor[r + 8][c]));
  };
  // accumulator n = 2 (lane % 4) + {0, 1} of n-tile nt is column 16 group + 2 n + nt
  auto put = [&](int tile, int group, const float (&big)[2][4], const float (&small)[2][4]) {
    const int at = 16 * group + 4 * q, i = 8 * tile + gr;
    *reinterpret_cast<float4*>(&sm.u[i][at]) =
        make_float4(big[0][0] + small[0][0], big[1][0] + small[1][0], big[0][1] + small[0][1], big[1][1] + small[1][1]);
    *reinterpret_cast<float4*>(&sm.qs[i][at]) =
        make_float4(big[0][2] + small[0][2], big[1][2] + small[1][2], big[0][3] + small[0][3], big[1][3] + small[1][3]);
  };
  if constexpr (kStaged<kNodes>) {
    static_assert(kCols == 1, "a warp takes one group");
    Right right[8][2];  // [k-step][n-tile]
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      float s[2][4];
      load_state(warp, ks, s);
#pragma unroll
      for (int t = 0; t < 2; ++t) right[ks][t].set(s[t][0], s[t][1], s[t][2], s[t][3]);
    }
    // the factors are there, and the state has been read: u and qs take its place
    if (__syncthreads_or(late)) {  // not the whole state: no results, and no end while it may still arrive
      if (tid == 0) {
        state_there();
        report(p.status, KDA_ERR_DEVICE_TIMEOUT);
      }
      return;
    }
    const int tiles = (n + 7) >> 3;
    for (int t = 0; t < tiles; ++t) {
      float big[2][4] = {}, small[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        Left left;
        load_factors(t, ks, left);
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) multiply(big[nt], small[nt], left, right[ks][nt]);
      }
      put(t, warp, big, small);
    }
  } else {
    // few rows: all of them are accumulated while the state streams by, a k-step ahead
    constexpr int kTiles = kNodes / 8, kAhead = 1;
    float s[kAhead + 1][kCols][2][4], big[kTiles][kCols][2][4] = {}, small[kTiles][kCols][2][4] = {};
#pragma unroll
    for (int ks = 0; ks < kAhead; ++ks)
#pragma unroll
      for (int g = 0; g < kCols; ++g) load_state(warp + kWarps * g, ks, s[ks][g]);
    __syncthreads();  // the factors are there
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      if (ks + kAhead < 8) {
#pragma unroll
        for (int g = 0; g < kCols; ++g) load_state(warp + kWarps * g, ks + kAhead, s[(ks + kAhead) % (kAhead + 1)][g]);
      }
      Left left[kTiles];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) load_factors(t, ks, left[t]);
#pragma unroll
      for (int g = 0; g < kCols; ++g)
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          const float(&w)[4] = s[ks % (kAhead + 1)][g][nt];
          Right right;
          right.set(w[0], w[1], w[2], w[3]);
#pragma unroll
          for (int t = 0; t < kTiles; ++t) multiply(big[t][g][nt], small[t][g][nt], left[t], right);
        }
    }
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int g = 0; g < kCols; ++g) put(t, warp + kWarps * g, big[t][g], small[t][g]);
  }
  __syncthreads();

  // ---- 3. down the tree, 16 nodes at a time: what earlier blocks contribute is a matrix product (split
  // as above), the rest a substitution with a thread per value column.  The products run over all
  // nodes, weights being zero where one is no ancestor; a delta that is not finite must not reach
  // other branches through such a zero, so from the first one on, ancestors are walked instead.
  const int blocks = (n + 15) >> 4, col = tid & 127;
  float* deltas = p.deltas + ((size_t)m0 * p.Hv + h) * dv;
  bool walk = false;
  constexpr int kBlocks = (kNodes + 15) / 16;
  Right solved[kCols][kBlocks][2];  // solved blocks as fragments: [.][block][n-tile]
  if constexpr (kNodes < 64) load_values(0);
#pragma unroll
  for (int blk = 0; blk < kBlocks; ++blk) {
    if (blk >= blocks) break;
    const int i0 = 16 * blk;
#pragma unroll
    for (int g = 0; g < kCols; ++g) {
      float big[2][4] = {}, small[2][4] = {};
#pragma unroll
      for (int kb = 0; kb < blk; ++kb) {
        Left left;
        left.set(*reinterpret_cast<const float4*>(&sm.a[i0 + gr][16 * kb + 4 * q]),
                 *reinterpret_cast<const float4*>(&sm.a[i0 + gr + 8][16 * kb + 4 * q]));
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) multiply(big[nt], small[nt], left, solved[g][kb][nt]);
      }
      float4* r0 = reinterpret_cast<float4*>(&sm.u[i0 + gr][c0(g)]);
      float4* r8 = reinterpret_cast<float4*>(&sm.u[i0 + gr + 8][c0(g)]);
      const float4 x = *r0, y = *r8;
      auto part = [&](int nt, int e) { return walk ? 0.f : big[nt][e] + small[nt][e]; };
      *r0 = make_float4(v0[g].x - x.x - part(0, 0), v0[g].y - x.y - part(1, 0), v0[g].z - x.z - part(0, 1), v0[g].w - x.w - part(1, 1));
      if (kNodes >= 16)
        *r8 = make_float4(v8[g].x - y.x - part(0, 2), v8[g].y - y.y - part(1, 2), v8[g].z - y.z - part(0, 3), v8[g].w - y.w - part(1, 3));
    }
    if (blk + 1 < blocks) load_values(i0 + 16);
    __syncthreads();
    bool odd = false;
    constexpr int kIn = kNodes < 16 ? kNodes : 16;
    float r[kIn];
    if (tid < 128) {
#pragma unroll
      for (int i = 0; i < kIn; ++i) r[i] = i0 + i < n ? sm.u[i0 + i][col] : 0.f;
#pragma unroll
      for (int i = 0; i < kIn; ++i) {
        float s = r[i];
#pragma unroll
        for (int j = 0; j < i; j += 4) {
          const float4 w = *reinterpret_cast<const float4*>(&sm.a[i0 + i][i0 + j]);
          s = fmaf(-w.x, r[j], s);
          if (j + 1 < i) s = fmaf(-w.y, r[j + 1], s);
          if (j + 2 < i) s = fmaf(-w.z, r[j + 2], s);
          if (j + 3 < i) s = fmaf(-w.w, r[j + 3], s);
        }
        r[i] = s * sm.beta[i0 + i];
        odd |= !isfinite(r[i]);
      }
    }
    // (what other columns of a row past dv hold is nobody's)
    const bool before = walk;
    walk |= __syncthreads_or(odd && col < dv) != 0;
    if (tid < 128) {
      if (!walk) {
#pragma unroll
        for (int i = 0; i < kIn; ++i) {
          sm.u[i0 + i][col] = r[i];
        }
      } else {
        for (int i = i0; i < min(i0 + 16, n); ++i) {
          float s = sm.u[i][col];
          for (int j = sm.par[i]; j >= (before ? 0 : i0); j = sm.par[j]) s = fmaf(-sm.a[i][j], sm.u[j][col], s);
          s *= sm.beta[i];
          sm.u[i][col] = s;
        }
      }
    }
    __syncthreads();
    if (!walk) {
#pragma unroll
      for (int g = 0; g < kCols; ++g) {
        const int i = i0 + 4 * q, cc = 16 * (warp + kWarps * g) + 2 * gr;
        float2 w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = kNodes >= 16 || 4 * q + e < kNodes ? *reinterpret_cast<const float2*>(&sm.u[i + e][cc]) : make_float2(0.f, 0.f);
        solved[g][blk][0].set(w[0].x, w[1].x, w[2].x, w[3].x);
        solved[g][blk][1].set(w[0].y, w[1].y, w[2].y, w[3].y);
      }
    }
  }
  // ---- the deltas, and the outputs: (Q o e^G) S plus the scores' product with them
  for (int i = warp; i < n; i += kWarps) {
    const float4 x = *reinterpret_cast<const float4*>(&sm.u[i][c4]);
    float* to = deltas + i * row + c4;
    if (kFull && wide_out) {
      *reinterpret_cast<float4*>(to) = x;
    } else {
      if (c4 < dv) to[0] = x.x;
      if (c4 + 1 < dv) to[1] = x.y;
      if (c4 + 2 < dv) to[2] = x.z;
      if (c4 + 3 < dv) to[3] = x.w;
    }
  }
  if (!walk) {
#pragma unroll
    for (int blk = 0; blk < kBlocks; ++blk) {
      if (blk >= blocks) break;
      const int i0 = 16 * blk;
#pragma unroll
      for (int g = 0; g < kCols; ++g) {
        float big[2][4] = {}, small[2][4] = {};
#pragma unroll
        for (int kb = 0; kb <= blk; ++kb) {
          Left left;
          left.set(*reinterpret_cast<const float4*>(&sm.b[i0 + gr][16 * kb + 4 * q]),
                   *reinterpret_cast<const float4*>(&sm.b[i0 + gr + 8][16 * kb + 4 * q]));
#pragma unroll
          for (int nt = 0; nt < 2; ++nt) multiply(big[nt], small[nt], left, solved[g][kb][nt]);
        }
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int i = i0 + gr + 8 * half;
          if (i < n) {
            const float4 x = *reinterpret_cast<const float4*>(&sm.qs[i][c0(g)]);
            const float o[4] = {x.x + big[0][2 * half] + small[0][2 * half], x.y + big[1][2 * half] + small[1][2 * half],
                                x.z + big[0][2 * half + 1] + small[0][2 * half + 1],
                                x.w + big[1][2 * half + 1] + small[1][2 * half + 1]};
            const size_t at = ((size_t)(m0 + i) * p.Hv + h) * dv + c0(g);
            if (kFull && wide_out) {
              if (p.out_bf16) glr::store4(reinterpret_cast<__nv_bfloat16*>(p.out) + at, make_float2(o[0], o[1]), make_float2(o[2], o[3]));
              else glr::store4(reinterpret_cast<float*>(p.out) + at, make_float2(o[0], o[1]), make_float2(o[2], o[3]));
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (c0(g) + e < dv) store_out(p.out, at + e, o[e], p.out_bf16);
            }
          }
        }
      }
    }
  } else if (col < dv) {
    for (int i = tid >> 7; i < n; i += kThreads / 128) {
      float s = sm.qs[i][col];
      for (int j = i; j >= 0; j = sm.par[j]) s = fmaf(sm.b[i][j], sm.u[j][col], s);
      store_out(p.out, ((size_t)(m0 + i) * p.Hv + h) * dv + col, s, p.out_bf16);
    }
  }
}

// ------------------------------------------------------------------------------------ commit

template <int kNodes>
struct CommitSmem {
  float kw[kNodes][128];  // k_j o e^{G_a - G_j} of the path's nodes, the accepted one first
  float u[kNodes][128];
  float total[128];       // e^{G_a}
  int32_t par[kNodes], path[kNodes];
  int32_t length;
};

// Thread mapping as the single-token step's: warp w takes the stored rows w + 8 m, a lane four columns.
template <int kNodes, bool kVFirst, bool kFull>
__global__ void __launch_bounds__(kThreads, 2) commit_kernel(const TreeArgs p) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  CommitSmem<kNodes>& sm = *reinterpret_cast<CommitSmem<kNodes>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / p.Hv, h = blockIdx.x - b * p.Hv, kh = h / (p.Hv / p.Hk);
  const int dk = kFull ? 128 : p.dk, dv = kFull ? 128 : p.dv;
  int32_t m0, n, slot;
  if (!tree_of(p, b, m0, n, slot, sm.par)) return;
  const int32_t acc = p.accepted[b];
  if (acc < 0 || acc >= n) {
    if (acc != -1 && tid == 0) report(p.status, KDA_ERR_DEVICE_CHECK);
    return;
  }
  float* blk = p.pool + ((size_t)slot * p.Hv + h) * (size_t)dk * dv;
  const int rows = kVFirst ? dv : dk, cols = kVFirst ? dk : dv;
  auto col = [&](int c) { return kFull ? 4 * lane + c : lane + 32 * c; };

  float s[16][4];
#pragma unroll
  for (int m = 0; m < 16; ++m) {
    const int r = warp + 8 * m;
    if constexpr (kFull) {
      const float4 v = *reinterpret_cast<const float4*>(blk + (size_t)r * 128 + 4 * lane);
      s[m][0] = v.x, s[m][1] = v.y, s[m][2] = v.z, s[m][3] = v.w;
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) s[m][c] = r < rows && col(c) < cols ? blk[(size_t)r * cols + col(c)] : 0.f;
    }
  }

  if (tid == 0) {
    int l = 0;
    for (int j = acc; j >= 0; j = sm.par[j]) sm.path[l++] = j;
    sm.length = l;
  }
  __syncthreads();
  const int length = sm.length;
  if (tid < 128) {
    float w = 1.f;
    if (tid < dk) {
      const float a_log = p.a_log[h], bias = p.dt_bias[(size_t)h * dk + tid];
      for (int l = 0; l < length; ++l) {
        const size_t m = m0 + sm.path[l];
        sm.kw[l][tid] = w * load_in(p.k, (m * p.Hk + kh) * dk + tid, p.in_bf16);
        const float g = gate_f32(p.raw_gate[(m * p.Hv + h) * dk + tid], a_log, bias, false, 0.f);
        w *= expf(p.flags & KDA_GATE_SAFE ? glr::max_nan(g, p.lb) : g);  // as in the tree, not a number stays one
      }
    } else {
      for (int l = 0; l < length; ++l) sm.kw[l][tid] = 0.f;
    }
    sm.total[tid] = w;
  } else {
    const int j = tid - 128;
    for (int l = 0; l < length; ++l)
      sm.u[l][j] = j < dv ? p.deltas[((size_t)(m0 + sm.path[l]) * p.Hv + h) * dv + j] : 0.f;
  }
  __syncthreads();

  // the stored row's factor and the lane's columns' factors: key channels are rows with K_FIRST and
  // columns with V_FIRST
#pragma unroll
  for (int m = 0; m < 16; ++m)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[m][c] *= sm.total[kVFirst ? col(c) & 127 : (warp + 8 * m) & 127];
  for (int l = 0; l < length; ++l) {
    const float* rv = kVFirst ? sm.u[l] : sm.kw[l];
    const float* cv = kVFirst ? sm.kw[l] : sm.u[l];
    float x[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) x[c] = cv[col(c) & 127];
#pragma unroll
    for (int m = 0; m < 16; ++m) {
      const float y = rv[warp + 8 * m];
#pragma unroll
      for (int c = 0; c < 4; ++c) s[m][c] = fmaf(y, x[c], s[m][c]);
    }
  }
#pragma unroll
  for (int m = 0; m < 16; ++m) {
    const int r = warp + 8 * m;
    if constexpr (kFull) {
      *reinterpret_cast<float4*>(blk + (size_t)r * 128 + 4 * lane) = make_float4(s[m][0], s[m][1], s[m][2], s[m][3]);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (r < rows && col(c) < cols) blk[(size_t)r * cols + col(c)] = s[m][c];
    }
  }
}

template <typename Kernel, typename... More>
cudaError_t launch(Kernel kernel, const TreeArgs& a, int threads, size_t smem, cudaStream_t stream, More... more) {
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)((int64_t)a.batch * a.Hv), threads, smem, stream>>>(a, more...);
  return cudaGetLastError();
}

template <int kNodes, bool kCommit>
cudaError_t pick(const TreeArgs& a, cudaStream_t stream) {
  auto on = [](const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  const bool full = a.dk == 128 && a.dv == 128 && on(a.pool, 16);
  const size_t smem = kCommit ? sizeof(CommitSmem<kNodes>) : sizeof(TreeSmem<kNodes>);
  if constexpr (kCommit) {
    auto go = [&](auto kernel) { return launch(kernel, a, kThreads, smem, stream); };
    if (a.v_first) return full ? go(commit_kernel<kNodes, true, true>) : go(commit_kernel<kNodes, true, false>);
    return full ? go(commit_kernel<kNodes, false, true>) : go(commit_kernel<kNodes, false, false>);
  } else {
    const bool wide_out = on(a.out, a.out_bf16 ? 8 : 16) && on(a.deltas, 16);
    auto go = [&](auto kernel) { return launch(kernel, a, kTreeThreads<kNodes>, smem, stream, wide_out); };
    // the form for 128 x 128 states reads rows in wide accesses: all of them start on 16 bytes (bf16: 8)
    const size_t in = a.in_bf16 ? 8 : 16;
    const bool wide = full && on(a.q, in) && on(a.k, in) && on(a.v, in) && on(a.raw_gate, 16) && on(a.dt_bias, 16);
    auto layout = [&](auto type) {
      using T = decltype(type);
      if (a.v_first) return wide ? go(tree_kernel<kNodes, true, true, T>) : go(tree_kernel<kNodes, true, false, T>);
      return wide ? go(tree_kernel<kNodes, false, true, T>) : go(tree_kernel<kNodes, false, false, T>);
    };
    return a.in_bf16 ? layout(__nv_bfloat16{}) : layout(float{});
  }
}

}  // namespace

cudaError_t launch_tree_decode(const TreeArgs& a, cudaStream_t stream) {
  if (a.max_nodes <= 8) return pick<8, false>(a, stream);
  if (a.max_nodes <= 16) return pick<16, false>(a, stream);
  if (a.max_nodes <= 32) return pick<32, false>(a, stream);
  return pick<64, false>(a, stream);
}

cudaError_t launch_tree_commit(const TreeArgs& a, cudaStream_t stream) {
  if (a.max_nodes <= 16) return pick<16, true>(a, stream);
  return pick<64, true>(a, stream);
}

}  // namespace kda
