// kda_ops_internal.h -- launch arguments and launchers of the operators around the state pools: the
// gated linear recurrence, drafted trees, and slots moved within a pool.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

// Tokens between the states the recurrence's forward pass keeps for its backward pass.
constexpr int kGlrBlock = 64;

struct GlrArgs {
  const void* x;         // [T,H,d]
  const void* raw_gate;  // [T,H,d]
  int32_t x_bf16, raw_bf16;
  const float* beta;     // [T,H]
  const float* a_log;    // [H]
  const float* dt_bias;  // [H,d]
  const int32_t* cu;     // [batch+1]; NULL: one token per sequence (decode)
  int32_t batch;
  int64_t total_tokens;
  int32_t H, d;
  float* pool;           // [max_slots][H][d]
  int32_t max_slots;
  const int32_t* slots;  // [batch]
  void* out;             // [T,H,d]
  int32_t out_bf16;
  float* checkpoints;    // nullable: [T/64 + batch][H][d]
  uint32_t flags;
  float lb;
  int32_t* status;
};

struct GlrBwdArgs {
  const void* dout;      // [T,H,d]
  int32_t dout_bf16;
  const void* x;
  const void* raw_gate;
  int32_t x_bf16, raw_bf16;
  const float* beta;
  const float* a_log;
  const float* dt_bias;
  const int32_t* cu;
  int32_t batch;
  int64_t total_tokens;
  int32_t H, d;
  const float* checkpoints;  // [T/64 + batch][H][d]
  const float* d_final;      // nullable: [batch][H][d]
  void* dx;                  // [T,H,d] as x
  void* draw;                // [T,H,d] as raw_gate
  float* dbeta;              // [T,H]
  float* da_log;             // [H]
  float* ddt_bias;           // [H,d]
  float* d_initial;          // [batch][H][d]
  float* partial;            // glr_bwd_partials() x [H][d + 1]: a head's sums over its channels' bias and gate
  uint32_t flags;
  float lb;
  int32_t* status;
};

struct TreeArgs {
  const void* q;           // [M,Hk,dk]
  const void* k;           // [M,Hk,dk]
  const void* v;           // [M,Hv,dv]
  int32_t in_bf16;
  const float* raw_gate;   // [M,Hv,dk]
  const float* beta;       // [M,Hv]
  const float* a_log;      // [Hv]
  const float* dt_bias;    // [Hv,dk]
  const int32_t* cu;       // [batch+1]
  const int32_t* parents;  // [M] local to the sequence, -1: the slot's state
  int32_t batch;
  int64_t total_nodes;
  int32_t max_nodes;
  int32_t Hk, Hv, dk, dv;
  float* pool;             // read (tree), written in place (commit)
  int32_t max_slots;
  const int32_t* slots;
  int32_t v_first;
  void* out;               // [M,Hv,dv]
  int32_t out_bf16;
  float* deltas;           // [M,Hv,dv] written by the tree, read by the commit
  const int32_t* accepted; // commit: [batch] local node or -1
  uint32_t flags;
  float lb;
  int32_t* status;
};

struct PoolArgs {
  float* pool;             // [layers][max_slots][slot_elems]
  int64_t slot_elems;
  int32_t layers, max_slots;
  int32_t* live;           // [max_slots] (fork, free, compact)
  const int32_t* src;      // [n]
  const int32_t* dst;      // [n]  (copy)
  int32_t* dst_out;        // [n]  (fork)
  int32_t* indices;        // [n]  (compact: state_indices, rewritten)
  int32_t* num_live;       // [1]  (compact)
  int32_t n;
  int32_t* work;           // pool_work_ints(n, max_slots)
  int32_t* status;
};
enum PoolOp { kPoolCopy = 0, kPoolFork = 1, kPoolFree = 2, kPoolCompact = 3 };

int glr_bwd_partials(int32_t batch, int64_t total_tokens, int32_t H);
cudaError_t launch_glr_fwd(const GlrArgs& a, cudaStream_t stream);
cudaError_t launch_glr_bwd(const GlrBwdArgs& a, cudaStream_t stream);
cudaError_t launch_glr_decode(const GlrArgs& a, cudaStream_t stream);
cudaError_t launch_tree_decode(const TreeArgs& a, cudaStream_t stream);
cudaError_t launch_tree_commit(const TreeArgs& a, cudaStream_t stream);
size_t pool_work_ints(int32_t n, int32_t max_slots);
bool pool_needs_work(PoolOp op, int32_t n);
cudaError_t launch_pool(const PoolArgs& a, PoolOp op, cudaStream_t stream);

}  // namespace kda
