// kda_ops_api.cu -- the C ABI of the operators around the state pools (include/kda.h): host-side
// validation and dispatch.  As everywhere, every check is always on and comes before any launch.
#include <cuda_runtime.h>

#include "../../include/kda.h"
#include "kda_ops_internal.h"

namespace {

constexpr uint32_t kGlrDecodeFlags = KDA_GATE_SAFE | KDA_BETA_PROB | KDA_INPUT_NORM;
constexpr uint32_t kGlrFlags = kGlrDecodeFlags | KDA_DEBUG_WITHHOLD_HANDOFF;
constexpr uint32_t kTreeFlags = KDA_GATE_SAFE | KDA_BETA_PROB | KDA_STATE_V_FIRST | KDA_DEBUG_WITHHOLD_HANDOFF;
constexpr int64_t kMaxTokens = INT32_MAX - 1024;  // the recurrence counts in whole tiles past the end
constexpr int32_t kMaxNodes = 64;
constexpr int32_t kMaxEntries = INT32_MAX - 1024;  // of a list or a pool that a plan's 1024 threads walk
constexpr int32_t kMaxCopies = 8192;  // pairs of one simultaneous copy: 16 bytes of each fit shared memory

bool dtype_ok(kda_dtype_t t) { return t == KDA_F32 || t == KDA_BF16; }
// a failed launch is told by the status alone: the runtime's record of it would be found by whoever asks next
kda_status_t done(cudaError_t e) {
  if (e == cudaSuccess) return KDA_OK;
  cudaGetLastError();
  return KDA_ERR_CUDA;
}
cudaStream_t as_stream(void* s) { return reinterpret_cast<cudaStream_t>(s); }
bool work_ok(const void* p, size_t have, size_t need) {
  return need == 0 || (p && have >= need && !(reinterpret_cast<uintptr_t>(p) & 255u));
}
// A safe gate's bound is a logarithm of a decay: the kernels' exponential is made for gates of at most 0.
bool bound_ok(uint32_t flags, float lb) { return !(flags & KDA_GATE_SAFE) || lb <= 0.f; }
// grid sizes and per-call element counts of the kernels
bool fits(int64_t batch, int64_t heads, int64_t each) { return batch * heads <= INT32_MAX / each; }

kda_status_t glr_types(kda_dtype_t x, kda_dtype_t gate, kda_dtype_t out) {
  if (!dtype_ok(x) || !dtype_ok(gate) || !dtype_ok(out)) return KDA_ERR_UNSUPPORTED;
  if (x == KDA_F32 && (gate != KDA_F32 || out != KDA_F32)) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

size_t glr_partial_bytes(int64_t T, int32_t batch, int32_t H, int32_t d) {
  if (T < 0 || T > kMaxTokens || batch <= 0 || H <= 0 || d <= 0 || d > 128 || !fits(batch, H, 16)) return 0;
  return (size_t)kda::glr_bwd_partials(batch, T, H) * H * (d + 1) * sizeof(float);
}

}  // namespace

extern "C" int64_t kda_glr_checkpoints(int64_t total_tokens, int32_t batch) {
  return total_tokens < 0 || batch < 0 ? 0 : total_tokens / kda::kGlrBlock + batch;
}

extern "C" kda_status_t kda_glr_fwd(const void* x, kda_dtype_t x_dtype, const void* raw_gate, kda_dtype_t gate_dtype,
                                    const float* beta_logits, const float* a_log, const float* dt_bias,
                                    const int32_t* cu_seqlens, int32_t batch, int64_t total_tokens,
                                    int32_t num_heads, int32_t d, float* state_pool, int32_t max_slots,
                                    const int32_t* state_indices, void* out, kda_dtype_t out_dtype,
                                    float* checkpoints, uint32_t flags, float gate_lower_bound,
                                    int32_t* device_status, void* stream) {
  if (batch < 0 || total_tokens < 0 || total_tokens > kMaxTokens || num_heads <= 0 || d <= 0 || max_slots <= 0)
    return KDA_ERR_INVALID_ARG;
  if ((flags & ~kGlrFlags) != 0 || !bound_ok(flags, gate_lower_bound)) return KDA_ERR_INVALID_ARG;
  if (!cu_seqlens || !state_pool || !state_indices || !a_log || !dt_bias) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!x || !raw_gate || !beta_logits || !out)) return KDA_ERR_INVALID_ARG;
  if (kda_status_t s = glr_types(x_dtype, gate_dtype, out_dtype); s != KDA_OK) return s;
  if (d > 128) return KDA_ERR_UNSUPPORTED;
  if (!fits(batch, num_heads, 16)) return KDA_ERR_INVALID_ARG;
  if (batch == 0) return KDA_OK;
  kda::GlrArgs a{};
  a.x = x;
  a.raw_gate = raw_gate;
  a.x_bf16 = x_dtype == KDA_BF16;
  a.raw_bf16 = gate_dtype == KDA_BF16;
  a.beta = beta_logits;
  a.a_log = a_log;
  a.dt_bias = dt_bias;
  a.cu = cu_seqlens;
  a.batch = batch;
  a.total_tokens = total_tokens;
  a.H = num_heads;
  a.d = d;
  a.pool = state_pool;
  a.max_slots = max_slots;
  a.slots = state_indices;
  a.out = out;
  a.out_bf16 = out_dtype == KDA_BF16;
  a.checkpoints = checkpoints;
  a.flags = flags;
  a.lb = gate_lower_bound;
  a.status = device_status;
  return done(kda::launch_glr_fwd(a, as_stream(stream)));
}

extern "C" kda_status_t kda_glr_decode(const void* x, kda_dtype_t x_dtype, const void* raw_gate,
                                       kda_dtype_t gate_dtype, const float* beta_logits, const float* a_log,
                                       const float* dt_bias, int32_t batch, int32_t num_heads, int32_t d,
                                       float* state_pool, int32_t max_slots, const int32_t* state_indices, void* out,
                                       kda_dtype_t out_dtype, uint32_t flags, float gate_lower_bound,
                                       int32_t* device_status, void* stream) {
  if (batch < 0 || num_heads <= 0 || d <= 0 || max_slots <= 0) return KDA_ERR_INVALID_ARG;
  if ((flags & ~kGlrDecodeFlags) != 0 || !bound_ok(flags, gate_lower_bound)) return KDA_ERR_INVALID_ARG;
  if (!state_pool || !state_indices || !a_log || !dt_bias) return KDA_ERR_INVALID_ARG;
  if (batch > 0 && (!x || !raw_gate || !beta_logits || !out)) return KDA_ERR_INVALID_ARG;
  if (kda_status_t s = glr_types(x_dtype, gate_dtype, out_dtype); s != KDA_OK) return s;
  if (d > 128) return KDA_ERR_UNSUPPORTED;
  if (!fits(batch, num_heads, 16)) return KDA_ERR_INVALID_ARG;
  if (batch == 0) return KDA_OK;
  kda::GlrArgs a{};
  a.x = x;
  a.raw_gate = raw_gate;
  a.x_bf16 = x_dtype == KDA_BF16;
  a.raw_bf16 = gate_dtype == KDA_BF16;
  a.beta = beta_logits;
  a.a_log = a_log;
  a.dt_bias = dt_bias;
  a.batch = batch;
  a.total_tokens = batch;
  a.H = num_heads;
  a.d = d;
  a.pool = state_pool;
  a.max_slots = max_slots;
  a.slots = state_indices;
  a.out = out;
  a.out_bf16 = out_dtype == KDA_BF16;
  a.flags = flags;
  a.lb = gate_lower_bound;
  a.status = device_status;
  return done(kda::launch_glr_decode(a, as_stream(stream)));
}

extern "C" size_t kda_glr_bwd_workspace_size(int64_t total_tokens, int32_t batch, int32_t num_heads, int32_t d) {
  return glr_partial_bytes(total_tokens, batch, num_heads, d);
}

extern "C" kda_status_t kda_glr_bwd(const void* dout, kda_dtype_t out_dtype, const void* x, kda_dtype_t x_dtype,
                                    const void* raw_gate, kda_dtype_t gate_dtype, const float* beta_logits,
                                    const float* a_log, const float* dt_bias, const int32_t* cu_seqlens,
                                    int32_t batch, int64_t total_tokens, int32_t num_heads, int32_t d,
                                    const float* checkpoints, const float* d_final, void* dx, void* draw_gate,
                                    float* dbeta, float* da_log, float* ddt_bias, float* d_initial, uint32_t flags,
                                    float gate_lower_bound, void* workspace, size_t workspace_bytes,
                                    int32_t* device_status, void* stream) {
  if (batch < 0 || total_tokens < 0 || total_tokens > kMaxTokens || num_heads <= 0 || d <= 0) return KDA_ERR_INVALID_ARG;
  if ((flags & ~kGlrFlags) != 0 || !bound_ok(flags, gate_lower_bound)) return KDA_ERR_INVALID_ARG;
  if (!cu_seqlens || !a_log || !dt_bias || !da_log || !ddt_bias) return KDA_ERR_INVALID_ARG;
  if (batch > 0 && (!d_initial || !checkpoints)) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0 && (!dout || !x || !raw_gate || !beta_logits || !dx || !draw_gate || !dbeta))
    return KDA_ERR_INVALID_ARG;
  if (kda_status_t s = glr_types(x_dtype, gate_dtype, out_dtype); s != KDA_OK) return s;
  if (d > 128) return KDA_ERR_UNSUPPORTED;
  if (!fits(batch, num_heads, 16)) return KDA_ERR_INVALID_ARG;
  cudaStream_t s = as_stream(stream);
  if (batch == 0) {
    cudaError_t e = cudaMemsetAsync(da_log, 0, (size_t)num_heads * sizeof(float), s);
    if (e == cudaSuccess) e = cudaMemsetAsync(ddt_bias, 0, (size_t)num_heads * d * sizeof(float), s);
    return done(e);
  }
  if (!work_ok(workspace, workspace_bytes, glr_partial_bytes(total_tokens, batch, num_heads, d)))
    return KDA_ERR_WORKSPACE;
  kda::GlrBwdArgs a{};
  a.dout = dout;
  a.dout_bf16 = out_dtype == KDA_BF16;
  a.x = x;
  a.raw_gate = raw_gate;
  a.x_bf16 = x_dtype == KDA_BF16;
  a.raw_bf16 = gate_dtype == KDA_BF16;
  a.beta = beta_logits;
  a.a_log = a_log;
  a.dt_bias = dt_bias;
  a.cu = cu_seqlens;
  a.batch = batch;
  a.total_tokens = total_tokens;
  a.H = num_heads;
  a.d = d;
  a.checkpoints = checkpoints;
  a.d_final = d_final;
  a.dx = dx;
  a.draw = draw_gate;
  a.dbeta = dbeta;
  a.da_log = da_log;
  a.ddt_bias = ddt_bias;
  a.d_initial = d_initial;
  a.partial = reinterpret_cast<float*>(workspace);
  a.flags = flags;
  a.lb = gate_lower_bound;
  a.status = device_status;
  return done(kda::launch_glr_bwd(a, s));
}

namespace {

// what the two calls on trees check alike
kda_status_t tree_checks(int32_t batch, int64_t total_nodes, int32_t max_nodes, int32_t Hk, int32_t Hv, int32_t dk,
                         int32_t dv, int32_t max_slots, uint32_t flags, float lb) {
  if (batch < 0 || total_nodes < 0 || total_nodes > INT32_MAX || max_nodes <= 0 || Hk <= 0 || Hv <= 0 || dk <= 0 ||
      dv <= 0 || max_slots <= 0)
    return KDA_ERR_INVALID_ARG;
  if (Hv % Hk != 0 || (flags & ~kTreeFlags) != 0 || !bound_ok(flags, lb)) return KDA_ERR_INVALID_ARG;
  if (!fits(batch, Hv, 1)) return KDA_ERR_INVALID_ARG;
  if (dk > 128 || dv > 128 || max_nodes > kMaxNodes) return KDA_ERR_UNSUPPORTED;
  return KDA_OK;
}

}  // namespace

extern "C" kda_status_t kda_tree_decode(const void* q, const void* k, const void* v, kda_dtype_t qkv_dtype,
                                        const float* raw_gate, const float* beta_logits, const float* a_log,
                                        const float* dt_bias, const int32_t* cu_nodes, const int32_t* parents,
                                        int32_t batch, int64_t total_nodes, int32_t max_nodes, int32_t num_k_heads,
                                        int32_t num_v_heads, int32_t dk, int32_t dv, const float* state_pool,
                                        int32_t max_slots, const int32_t* state_indices, void* out,
                                        kda_dtype_t out_dtype, float* deltas, uint32_t flags, float gate_lower_bound,
                                        int32_t* device_status, void* stream) {
  const kda_status_t st = tree_checks(batch, total_nodes, max_nodes, num_k_heads, num_v_heads, dk, dv, max_slots, flags,
                                      gate_lower_bound);
  if (st == KDA_ERR_INVALID_ARG) return st;
  if (!cu_nodes || !state_pool || !state_indices || !a_log || !dt_bias) return KDA_ERR_INVALID_ARG;
  if (total_nodes > 0 && (!q || !k || !v || !raw_gate || !beta_logits || !parents || !out || !deltas))
    return KDA_ERR_INVALID_ARG;
  if (st != KDA_OK) return st;
  if (!dtype_ok(qkv_dtype) || !dtype_ok(out_dtype)) return KDA_ERR_UNSUPPORTED;
  if (qkv_dtype == KDA_F32 && out_dtype != KDA_F32) return KDA_ERR_UNSUPPORTED;
  if (batch == 0 || total_nodes == 0) return KDA_OK;
  kda::TreeArgs a{};
  a.q = q;
  a.k = k;
  a.v = v;
  a.in_bf16 = qkv_dtype == KDA_BF16;
  a.raw_gate = raw_gate;
  a.beta = beta_logits;
  a.a_log = a_log;
  a.dt_bias = dt_bias;
  a.cu = cu_nodes;
  a.parents = parents;
  a.batch = batch;
  a.total_nodes = total_nodes;
  a.max_nodes = max_nodes;
  a.Hk = num_k_heads;
  a.Hv = num_v_heads;
  a.dk = dk;
  a.dv = dv;
  a.pool = const_cast<float*>(state_pool);
  a.max_slots = max_slots;
  a.slots = state_indices;
  a.v_first = (flags & KDA_STATE_V_FIRST) ? 1 : 0;
  a.out = out;
  a.out_bf16 = out_dtype == KDA_BF16;
  a.deltas = deltas;
  a.flags = flags;
  a.lb = gate_lower_bound;
  a.status = device_status;
  return done(kda::launch_tree_decode(a, as_stream(stream)));
}

extern "C" kda_status_t kda_tree_commit(const void* k, kda_dtype_t k_dtype, const float* raw_gate, const float* a_log,
                                        const float* dt_bias, const float* deltas, const int32_t* cu_nodes,
                                        const int32_t* parents, const int32_t* accepted, int32_t batch,
                                        int64_t total_nodes, int32_t max_nodes, int32_t num_k_heads,
                                        int32_t num_v_heads, int32_t dk, int32_t dv, float* state_pool,
                                        int32_t max_slots, const int32_t* state_indices, uint32_t flags,
                                        float gate_lower_bound, int32_t* device_status, void* stream) {
  const kda_status_t st = tree_checks(batch, total_nodes, max_nodes, num_k_heads, num_v_heads, dk, dv, max_slots, flags,
                                      gate_lower_bound);
  if (st == KDA_ERR_INVALID_ARG) return st;
  if (!cu_nodes || !state_pool || !state_indices || !a_log || !dt_bias || !accepted) return KDA_ERR_INVALID_ARG;
  if (total_nodes > 0 && (!k || !raw_gate || !parents || !deltas)) return KDA_ERR_INVALID_ARG;
  if (st != KDA_OK) return st;
  if (!dtype_ok(k_dtype)) return KDA_ERR_UNSUPPORTED;
  if (batch == 0) return KDA_OK;
  kda::TreeArgs a{};
  a.k = k;
  a.in_bf16 = k_dtype == KDA_BF16;
  a.raw_gate = raw_gate;
  a.a_log = a_log;
  a.dt_bias = dt_bias;
  a.cu = cu_nodes;
  a.parents = parents;
  a.batch = batch;
  a.total_nodes = total_nodes;
  a.max_nodes = max_nodes;
  a.Hk = num_k_heads;
  a.Hv = num_v_heads;
  a.dk = dk;
  a.dv = dv;
  a.pool = state_pool;
  a.max_slots = max_slots;
  a.slots = state_indices;
  a.v_first = (flags & KDA_STATE_V_FIRST) ? 1 : 0;
  a.deltas = const_cast<float*>(deltas);
  a.accepted = accepted;
  a.flags = flags;
  a.lb = gate_lower_bound;
  a.status = device_status;
  return done(kda::launch_tree_commit(a, as_stream(stream)));
}

extern "C" size_t kda_pool_workspace_size(int32_t n, int32_t max_slots) {
  return n < 0 || max_slots <= 0 ? 0 : kda::pool_work_ints(n, max_slots) * sizeof(int32_t);
}

namespace {

kda_status_t pool_call(kda::PoolArgs& a, kda::PoolOp op, void* workspace, size_t workspace_bytes, void* stream) {
  if (!a.pool || a.layers <= 0 || a.max_slots <= 0 || a.slot_elems <= 0 || a.n < 0) return KDA_ERR_INVALID_ARG;
  if (a.n > kMaxEntries || (op != kda::kPoolCopy && a.max_slots > kMaxEntries)) return KDA_ERR_INVALID_ARG;
  // element offsets within the stack are 64-bit; their product must be one too
  if (a.slot_elems > INT64_MAX / 4 / a.layers / a.max_slots) return KDA_ERR_INVALID_ARG;
  if (kda::pool_needs_work(op, a.n) &&
      !work_ok(workspace, workspace_bytes, kda_pool_workspace_size(a.n, a.max_slots)))
    return KDA_ERR_WORKSPACE;
  a.work = reinterpret_cast<int32_t*>(workspace);
  return done(kda::launch_pool(a, op, as_stream(stream)));
}

kda::PoolArgs pool_args(float* pool, int32_t layers, int32_t max_slots, int64_t slot_elems, int32_t n, int32_t* status) {
  kda::PoolArgs a{};
  a.pool = pool;
  a.slot_elems = slot_elems;
  a.layers = layers;
  a.max_slots = max_slots;
  a.n = n;
  a.status = status;
  return a;
}

}  // namespace

extern "C" kda_status_t kda_pool_copy(float* state_pool, int32_t layers, int32_t max_slots, int64_t slot_elems,
                                      const int32_t* src, const int32_t* dst, int32_t n, void* workspace,
                                      size_t workspace_bytes, int32_t* device_status, void* stream) {
  kda::PoolArgs a = pool_args(state_pool, layers, max_slots, slot_elems, n, device_status);
  if (n > 0 && (!src || !dst)) return KDA_ERR_INVALID_ARG;
  if (n > kMaxCopies) return KDA_ERR_UNSUPPORTED;
  if (n == 0 && state_pool && layers > 0 && max_slots > 0 && slot_elems > 0) return KDA_OK;
  a.src = src;
  a.dst = dst;
  return pool_call(a, kda::kPoolCopy, workspace, workspace_bytes, stream);
}

extern "C" kda_status_t kda_pool_fork(float* state_pool, int32_t layers, int32_t max_slots, int64_t slot_elems,
                                      int32_t* live, const int32_t* src, int32_t* dst, int32_t n, void* workspace,
                                      size_t workspace_bytes, int32_t* device_status, void* stream) {
  kda::PoolArgs a = pool_args(state_pool, layers, max_slots, slot_elems, n, device_status);
  if (!live || (n > 0 && (!src || !dst))) return KDA_ERR_INVALID_ARG;
  if (n == 0 && state_pool && layers > 0 && max_slots > 0 && slot_elems > 0) return KDA_OK;
  a.live = live;
  a.src = src;
  a.dst_out = dst;
  return pool_call(a, kda::kPoolFork, workspace, workspace_bytes, stream);
}

extern "C" kda_status_t kda_pool_free(float* state_pool, int32_t layers, int32_t max_slots, int64_t slot_elems,
                                      int32_t* live, const int32_t* slots, int32_t n, void* workspace,
                                      size_t workspace_bytes, int32_t* device_status, void* stream) {
  kda::PoolArgs a = pool_args(state_pool, layers, max_slots, slot_elems, n, device_status);
  if (!live || (n > 0 && !slots)) return KDA_ERR_INVALID_ARG;
  if (n == 0 && state_pool && layers > 0 && max_slots > 0 && slot_elems > 0) return KDA_OK;
  a.live = live;
  a.src = slots;
  return pool_call(a, kda::kPoolFree, workspace, workspace_bytes, stream);
}

extern "C" kda_status_t kda_pool_compact(float* state_pool, int32_t layers, int32_t max_slots, int64_t slot_elems,
                                         int32_t* live, int32_t* state_indices, int32_t n, int32_t* num_live,
                                         void* workspace, size_t workspace_bytes, int32_t* device_status,
                                         void* stream) {
  kda::PoolArgs a = pool_args(state_pool, layers, max_slots, slot_elems, n, device_status);
  if (!live || !num_live || (n > 0 && !state_indices)) return KDA_ERR_INVALID_ARG;
  a.live = live;
  a.indices = state_indices;
  a.num_live = num_live;
  return pool_call(a, kda::kPoolCompact, workspace, workspace_bytes, stream);
}
