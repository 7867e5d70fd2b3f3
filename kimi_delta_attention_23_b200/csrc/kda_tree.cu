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
//  2. P = [K o e^G; Q o e^G] S on mma.sync: S comes from global memory straight into the B
//     fragments.  Every fp32 factor is split into two bf16 parts and three of the four partial
//     products are summed (2^-18 of the factors is lost): kda_tree_commit writes the results of this
//     into fp32 states, which one bf16 product would spoil.
//  3. each value column's thread solves down the tree, then the outputs follow.
// It is bound by the state's 4 dk dv bytes for drafts of about 16 nodes and fewer.  tcgen05 is not
// used: with 2 N <= 128 rows against a 128 x 128 state read once, staging S through shared memory
// for it costs more than the whole product does here.
//
// The commit is S' = e^{G_a} o S + sum over the path (k_j o e^{G_a - G_j}) u_j^T, one pass over the
// state, bound by its 8 dk dv bytes.
#include "kda_common.cuh"
#include "kda_ops_internal.h"

namespace kda {
namespace {

constexpr int kThreads = 256;
constexpr int kPitch = 132;    // floats of a node's row in shared memory
constexpr int kPitchH = 144;   // bf16 of a row of the split factors (32 bytes past 256: no conflicts)

// Offsets, slot and parents of a sequence; false where one is out of range.  All threads call it.
__device__ __forceinline__ bool tree_of(const TreeArgs& a, int b, int32_t& m0, int32_t& n, int32_t& slot, int32_t* s_par) {
  m0 = a.cu[b];
  n = a.cu[b + 1] - m0;
  slot = a.slots[b];
  bool ok = m0 >= 0 && n >= 0 && n <= a.max_nodes && (int64_t)m0 + n <= a.total_nodes && slot >= 0 && slot < a.max_slots;
  if (ok && (int)threadIdx.x < n) {
    const int32_t par = a.parents[m0 + threadIdx.x];
    s_par[threadIdx.x] = par;
    ok = par >= -1 && par < (int)threadIdx.x;
  }
  ok = __syncthreads_and(ok);
  if (!ok && threadIdx.x == 0) report(a.status, KDA_ERR_DEVICE_CHECK);
  return ok;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// x = hi + lo up to 2^-18 of x; two values to a word, the first in the low half
__device__ __forceinline__ void split2(float x, float y, uint32_t& hi, uint32_t& lo) {
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(y), "f"(x));
  const float rx = x - __uint_as_float(hi << 16), ry = y - __uint_as_float(hi & 0xffff0000u);
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(ry), "f"(rx));
}

template <int kNodes>
struct TreeSmem {
  union {
    float k[kNodes][kPitch];   // keys (1)
    float u[kNodes][kPitch];   // (K o e^G) S (2), then the deltas (3)
  };
  union {
    float al[kNodes][kPitch];  // decays (1)
    float qs[kNodes][kPitch];  // (Q o e^G) S (2)
  };
  // rows 16 t + r: key row 8 t + r for r < 8, query row 8 t + r - 8 for the others
  __nv_bfloat16 hi[2 * kNodes][kPitchH], lo[2 * kNodes][kPitchH];
  float a[kNodes][kNodes + 1], b[kNodes][kNodes + 1];
  float beta[kNodes];
  int32_t par[kNodes];
};

template <int kNodes, bool kVFirst, bool kFull>
__global__ void __launch_bounds__(kThreads, 2) tree_kernel(const TreeArgs p) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  TreeSmem<kNodes>& sm = *reinterpret_cast<TreeSmem<kNodes>*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / p.Hv, h = blockIdx.x - b * p.Hv, kh = h / (p.Hv / p.Hk);
  const int dk = kFull ? 128 : p.dk, dv = kFull ? 128 : p.dv;
  int32_t m0, n, slot;
  if (!tree_of(p, b, m0, n, slot, sm.par)) return;
  if (n == 0) return;
  const float* state = p.pool + ((size_t)slot * p.Hv + h) * (size_t)dk * dv;
  if constexpr (kFull) {  // the state is wanted after the scores: bring it to L2 meanwhile
    if (tid == 0)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(state), "r"(128 * 128 * 4) : "memory");
  }

  // ---- keys, decays and beta of all nodes; zero keys past dk
  const bool safe = p.flags & KDA_GATE_SAFE, prob = p.flags & KDA_BETA_PROB;
  {
    const float a_log = p.a_log[h];
    for (int i = tid; i < n * 128; i += kThreads) {
      const int m = i >> 7, c = i & 127;
      float kv = 0.f, al = 1.f;
      if (c < dk) {
        kv = load_in(p.k, ((size_t)(m0 + m) * p.Hk + kh) * dk + c, p.in_bf16);
        al = expf(gate_f32(p.raw_gate[((size_t)(m0 + m) * p.Hv + h) * dk + c], a_log, p.dt_bias[(size_t)h * dk + c], safe, p.lb));
      }
      sm.k[m][c] = kv;
      sm.al[m][c] = al;
    }
    for (int m = tid; m < n; m += kThreads) sm.beta[m] = beta_f32(p.beta[(size_t)(m0 + m) * p.Hv + h], prob);
  }
  __syncthreads();

  // ---- 1. scores, and the factors of the product with the state
  {
    constexpr int kGroup = kThreads / kNodes;  // lanes per node
    constexpr int kQuads = 32 / kGroup;        // float4's of channels per lane
    static_assert(kGroup <= 32 && kQuads >= 1, "");
    const int i = tid / kGroup, g = tid % kGroup;
    const bool mine = i < n;
    float4 kq[kQuads], qq[kQuads], w[kQuads];
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      const int c = 4 * (g + kGroup * j);
      w[j] = make_float4(1.f, 1.f, 1.f, 1.f);
      kq[j] = qq[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (mine) {
        kq[j] = *reinterpret_cast<const float4*>(&sm.k[i][c]);
        const size_t at = ((size_t)(m0 + i) * p.Hk + kh) * dk + c;
        qq[j] = make_float4(c < dk ? load_in(p.q, at, p.in_bf16) : 0.f, c + 1 < dk ? load_in(p.q, at + 1, p.in_bf16) : 0.f,
                            c + 2 < dk ? load_in(p.q, at + 2, p.in_bf16) : 0.f, c + 3 < dk ? load_in(p.q, at + 3, p.in_bf16) : 0.f);
      }
    }
    int anc = mine ? i : -1;
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
          sm.a[i][anc] = sa;  // for anc == i: not used
          sm.b[i][anc] = sb;
        }
        anc = sm.par[anc];
      }
    }
    // rows past the last node are zero: they share 16-row tiles with others
    const int rk = 16 * (i >> 3) + (i & 7);
#pragma unroll
    for (int j = 0; j < kQuads; ++j) {
      const int c = 4 * (g + kGroup * j);
      uint2 hi, lo;
      split2(kq[j].x * w[j].x, kq[j].y * w[j].y, hi.x, lo.x);
      split2(kq[j].z * w[j].z, kq[j].w * w[j].w, hi.y, lo.y);
      *reinterpret_cast<uint2*>(&sm.hi[rk][c]) = hi;
      *reinterpret_cast<uint2*>(&sm.lo[rk][c]) = lo;
      split2(qq[j].x * w[j].x, qq[j].y * w[j].y, hi.x, lo.x);
      split2(qq[j].z * w[j].z, qq[j].w * w[j].w, hi.y, lo.y);
      *reinterpret_cast<uint2*>(&sm.hi[rk + 8][c]) = hi;
      *reinterpret_cast<uint2*>(&sm.lo[rk + 8][c]) = lo;
    }
  }
  __syncthreads();

  // ---- 2. the product with the state.  A warp owns 16 value columns (two n-tiles: columns
  // 16 warp + 2 (lane / 4) + {0, 1}) over all key channels.  Within each 16 channels a lane's four
  // are 4 (lane % 4) .. + 3 in both operands (the order of the summed index is free), so that its
  // share of V_FIRST states and of the factors is one wide access.
  {
    const int q = lane & 3, g = lane >> 2, col = 16 * warp + 2 * g;
    uint32_t bh[8][2][2], bl[8][2][2];  // [k-step][n-tile][register]
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const int c = 16 * ks + 4 * q;
      float s[2][4];
      if constexpr (kFull && kVFirst) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float4 v = __ldg(reinterpret_cast<const float4*>(state + (size_t)(col + t) * 128 + c));
          s[t][0] = v.x, s[t][1] = v.y, s[t][2] = v.z, s[t][3] = v.w;
        }
      } else if constexpr (kFull) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 v = __ldg(reinterpret_cast<const float2*>(state + (size_t)(c + e) * 128 + col));
          s[0][e] = v.x, s[1][e] = v.y;
        }
      } else {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[t][e] = c + e < dk && col + t < dv ? state[state_off(c + e, col + t, dk, dv, kVFirst)] : 0.f;
      }
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        split2(s[t][0], s[t][1], bh[ks][t][0], bl[ks][t][0]);
        split2(s[t][2], s[t][3], bh[ks][t][1], bl[ks][t][1]);
      }
    }
    const int tiles = (n + 7) >> 3;
    for (int t = 0; t < tiles; ++t) {
      float acc[2][4] = {};
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        const int c = 16 * ks + 4 * q;
        const uint2 h0 = *reinterpret_cast<const uint2*>(&sm.hi[16 * t + g][c]);
        const uint2 h1 = *reinterpret_cast<const uint2*>(&sm.hi[16 * t + g + 8][c]);
        const uint2 l0 = *reinterpret_cast<const uint2*>(&sm.lo[16 * t + g][c]);
        const uint2 l1 = *reinterpret_cast<const uint2*>(&sm.lo[16 * t + g + 8][c]);
        const uint32_t ah[4] = {h0.x, h1.x, h0.y, h1.y}, al[4] = {l0.x, l1.x, l0.y, l1.y};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt) {
          mma_bf16(acc[nt], al, bh[ks][nt][0], bh[ks][nt][1]);
          mma_bf16(acc[nt], ah, bl[ks][nt][0], bl[ks][nt][1]);
          mma_bf16(acc[nt], ah, bh[ks][nt][0], bh[ks][nt][1]);
        }
      }
      // accumulator n = 2 (lane % 4) + {0, 1} of tile nt is column 16 warp + 2 n + nt
      const int c0 = 16 * warp + 4 * q, i = 8 * t + g;
      *reinterpret_cast<float4*>(&sm.u[i][c0]) = make_float4(acc[0][0], acc[1][0], acc[0][1], acc[1][1]);
      *reinterpret_cast<float4*>(&sm.qs[i][c0]) = make_float4(acc[0][2], acc[1][2], acc[0][3], acc[1][3]);
    }
  }
  __syncthreads();

  // ---- 3. down the tree, a thread per value column; its own column is all it reads
  if (tid < dv) {
    for (int i = 0; i < n; ++i) {
      const size_t at = ((size_t)(m0 + i) * p.Hv + h) * dv + tid;
      float r = load_in(p.v, at, p.in_bf16) - sm.u[i][tid];
      for (int j = sm.par[i]; j >= 0; j = sm.par[j]) r = fmaf(-sm.a[i][j], sm.u[j][tid], r);
      r *= sm.beta[i];
      sm.u[i][tid] = r;
      p.deltas[at] = r;
    }
  }
  __syncthreads();
  const int col = tid & 127;
  if (col < dv) {
    for (int i = tid >> 7; i < n; i += kThreads / 128) {
      float r = sm.qs[i][col];
      for (int j = i; j >= 0; j = sm.par[j]) r = fmaf(sm.b[i][j], sm.u[j][col], r);
      store_out(p.out, ((size_t)(m0 + i) * p.Hv + h) * dv + col, r, p.out_bf16);
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
  extern __shared__ __align__(16) unsigned char smem_raw[];
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
        w *= expf(gate_f32(p.raw_gate[(m * p.Hv + h) * dk + tid], a_log, bias, p.flags & KDA_GATE_SAFE, p.lb));
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

template <typename Kernel>
cudaError_t launch(Kernel kernel, const TreeArgs& a, size_t smem, cudaStream_t stream) {
  if (smem > 48 * 1024) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  kernel<<<(unsigned)((int64_t)a.batch * a.Hv), kThreads, smem, stream>>>(a);
  return cudaGetLastError();
}

template <int kNodes, bool kCommit>
cudaError_t pick(const TreeArgs& a, cudaStream_t stream) {
  const bool full = a.dk == 128 && a.dv == 128 && (reinterpret_cast<uintptr_t>(a.pool) & 15u) == 0;
  const size_t smem = kCommit ? sizeof(CommitSmem<kNodes>) : sizeof(TreeSmem<kNodes>);
  auto go = [&](auto kernel) { return launch(kernel, a, smem, stream); };
  if constexpr (kCommit) {
    if (a.v_first) return full ? go(commit_kernel<kNodes, true, true>) : go(commit_kernel<kNodes, true, false>);
    return full ? go(commit_kernel<kNodes, false, true>) : go(commit_kernel<kNodes, false, false>);
  } else {
    if (a.v_first) return full ? go(tree_kernel<kNodes, true, true>) : go(tree_kernel<kNodes, true, false>);
    return full ? go(tree_kernel<kNodes, false, true>) : go(tree_kernel<kNodes, false, false>);
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
