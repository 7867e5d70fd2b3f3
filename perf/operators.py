"""The serving and training operators around the state pools, as measured workloads.

Kinds of case:
  glr_fwd     the gated linear recurrence over a varlen batch, states read from and written to a pool
  glr_train   one training step of it: the forward pass, then the gradients of everything it read
  glr_decode  one token of each sequence
  tree        a tree of drafted tokens of each sequence, read against that sequence's KDA state
  commit      the accepted path of each tree written into the sequence's state
  copy, fork, free, compact   slots of a state pool moved, duplicated, cleared, packed

``run`` computes a case in its plain form (elementary torch operations in 32 bits, 64 for sums of
gates along a path), or through the package where ``own`` is true.
"""
import math

import torch

own = False

DEV = "cuda"
LOWER = -5.0  # the safe gate's bound
BLOCK = 64    # tokens between the states that training keeps
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def _glr(kind, **kw):
    base = dict(kind=kind, tokens=64, seqs=1, heads=32, d=128, x="bf16", raw="bf16", out="bf16",
                gate="original", beta="logits", input="norm")
    return {**base, **kw}


def _tree(kind, **kw):
    base = dict(kind=kind, seqs=1, nodes=8, ragged=False, shape="tree", kheads=32, heads=32, dk=128, dv=128,
                x="bf16", out="bf16", gate="original", beta="logits", layout="K_FIRST")
    return {**base, **kw}


def _pool(kind, **kw):
    base = dict(kind=kind, layers=1, slots=8, heads=16, dk=128, dv=128, moved=1)
    return {**base, **kw}


def listed():
    return [
        # the prefill of one very long document through a recurrent layer
        _glr("glr_fwd", name="glr_prefill_long", tokens=131072),
        # a training step on a packed batch of documents, fp32 gates as the projections give them
        _glr("glr_train", name="glr_train_packed", tokens=32768, seqs=8, raw="f32", input="unit"),
        # a small fp32 model on short ragged texts: odd head size, clamped gate
        _glr("glr_train", name="glr_train_odd_f32", tokens=1531, seqs=7, heads=5, d=37, x="f32", raw="f32", out="f32",
             gate="safe", beta="probability"),
        # a full decode batch, one token of each request
        _glr("glr_decode", name="glr_decode_batch", tokens=256, seqs=256),
        # one interactive request with a short draft: latency
        _tree("tree", name="tree_one_request"),
        # a serving batch with drafts of up to 16 tokens, some of them shorter or missing
        _tree("tree", name="tree_serving", seqs=64, nodes=16, ragged=True),
        # wide drafts for every request of a batch, fewer key than value heads
        _tree("tree", name="tree_wide", seqs=32, nodes=64, kheads=8, layout="V_FIRST"),
        # plain drafted chains on a small fp32 model with odd head sizes
        _tree("tree", name="tree_chain_odd_f32", seqs=3, nodes=21, shape="chain", kheads=2, heads=6, dk=72, dv=45,
              x="f32", out="f32", gate="safe", beta="probability"),
        # the serving batch's accepted paths written into the states
        _tree("commit", name="commit_serving", seqs=64, nodes=16, ragged=True),
        # one prompt's state kept aside before a risky continuation: latency
        _pool("copy", name="pool_copy_one"),
        # several samples from each prompt of a batch
        _pool("fork", name="pool_fork_samples", slots=256, heads=32, moved=64),
        # a pool of small states, of an odd size, packed after most requests have ended
        _pool("compact", name="pool_compact_small", slots=4096, heads=5, dk=37, dv=1, moved=1100),
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    kind = rng.choice(["glr_fwd", "glr_train", "glr_decode", "tree", "tree", "commit", "copy", "fork", "free", "compact"])
    if kind.startswith("glr"):
        x, raw = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
        out = "f32" if x == "f32" else rng.choice(["bf16", "bf16", "f32"])
        if kind == "glr_decode":
            seqs = tokens = _log(rng, 1, 512)
        else:
            tokens = _log(rng, 1, 32768 if kind == "glr_fwd" else 12000)
            seqs = min(_log(rng, 1, 64), tokens)
        return _glr(kind, tokens=tokens, seqs=seqs, heads=_log(rng, 1, 32),
                    d=rng.choice([128, 128, 128, 64, 96, rng.randint(1, 128)]), x=x, raw=raw, out=out,
                    gate=rng.choice(["original", "safe"]), beta=rng.choice(["logits", "probability"]),
                    input=rng.choice(["unit", "norm"]))
    if kind in ("tree", "commit"):
        kheads = _log(rng, 1, 16)
        x = rng.choice(["bf16", "bf16", "f32"])
        dk, dv = rng.choice([(128, 128), (128, 128), (128, 128), (64, 64), (rng.randint(1, 128), rng.randint(1, 128))])
        nodes = _log(rng, 1, 64)
        return _tree(kind, seqs=_log(rng, 1, 32), nodes=nodes, ragged=rng.random() < 0.5,
                     shape=rng.choice(["tree", "chain"]), kheads=kheads, heads=kheads * rng.choice([1, 1, 2]),
                     dk=dk, dv=dv, x=x, out="f32" if x == "f32" else rng.choice(["bf16", "bf16", "f32"]),
                     gate=rng.choice(["original", "safe"]), beta=rng.choice(["logits", "probability"]),
                     layout=rng.choice(["K_FIRST", "V_FIRST"]))
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (rng.randint(1, 128), rng.randint(1, 128)), (128, 1)])
    slots = _log(rng, 2, 200 if dv > 1 else 3000)
    return _pool(kind, layers=rng.choice([1, 1, 2]), slots=slots, heads=_log(rng, 1, 32), dk=dk, dv=dv,
                 moved=rng.randint(1, max(1, slots // 2)))


# ---------------------------------------------------------------------------------- inputs

def _counts(case):
    """Drafted tokens of each sequence; in a ragged batch some sequences have few or none."""
    n = case["nodes"]
    return [37 * b % (n + 1) if case["ragged"] and b else n for b in range(case["seqs"])]


def _offsets(lengths):
    cu = torch.zeros(len(lengths) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(lengths, dtype=torch.int32).cumsum(0)
    return cu


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    h = torch.Generator()
    h.manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        return (torch.randn(*shape, device=DEV, generator=g) * std + mean).to(dtype)

    s = {"case": dict(case)}
    kind = case["kind"]
    if kind.startswith("glr"):
        T, B, H, d = case["tokens"], case["seqs"], case["heads"], case["d"]
        xt, rt = TYPES[case["x"]], TYPES[case["raw"]]
        s["x"] = normal(T, H, d, dtype=xt)
        s["raw"] = normal(T, H, d, dtype=rt)
        beta = normal(T, H, mean=1.0)
        s["beta"] = beta.sigmoid() if case["beta"] == "probability" else beta
        s["a_log"] = torch.rand(H, device=DEV, generator=g) * math.log(16.0)
        s["dt_bias"] = normal(H, d, mean=-4.0)  # decays from a few to thousands of tokens
        slots = B + B // 4 + 1
        s["pool"] = normal(slots, H, d)
        s["idx"] = torch.randperm(slots, generator=h)[:B].to(torch.int32).to(DEV)
        if kind != "glr_decode":
            cuts = sorted(torch.randint(0, T + 1, (B - 1,), generator=h).tolist())
            lengths = [b - a for a, b in zip([0] + cuts, cuts + [T])]
            s["longest"] = max(lengths)
            s["cu"] = _offsets(lengths).to(DEV)
        if kind == "glr_train":
            s["carried"] = s["pool"].clone()
            s["dout"] = normal(T, H, d, dtype=TYPES[case["out"]])
            s["dfinal"] = normal(B, H, d)
        return s
    if kind in ("tree", "commit"):
        B, Hk, Hv, dk, dv = case["seqs"], case["kheads"], case["heads"], case["dk"], case["dv"]
        counts = _counts(case)
        M = sum(counts)
        s["cu"] = _offsets(counts).to(DEV)
        if case["shape"] == "chain":
            parents = [i - 1 for n in counts for i in range(n)]
        else:
            r = torch.rand(max(1, M), generator=h).tolist()
            at = [i for n in counts for i in range(n)]
            parents = [int(u * (i + 1)) - 1 for u, i in zip(r, at)]
        s["parents"] = torch.tensor(parents, dtype=torch.int32).to(DEV)
        xt = TYPES[case["x"]]
        unit = lambda x: x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)  # noqa: E731
        s["q"] = unit(normal(M, Hk, dk)).to(xt)
        s["k"] = unit(normal(M, Hk, dk)).to(xt)
        s["v"] = normal(M, Hv, dv, dtype=xt)
        s["raw"] = normal(M, Hv, dk)
        beta = normal(M, Hv)
        s["beta"] = beta.sigmoid() if case["beta"] == "probability" else beta
        s["a_log"] = torch.rand(Hv, device=DEV, generator=g) * math.log(16.0)
        s["dt_bias"] = normal(Hv, dk, mean=-2.0)
        slots = B + B // 4 + 1
        s["pool"] = normal(slots, Hv, *((dk, dv) if case["layout"] == "K_FIRST" else (dv, dk)), std=0.3)
        s["idx"] = torch.randperm(slots, generator=h)[:B].to(torch.int32).to(DEV)
        if kind == "commit":
            s["deltas"] = normal(M, Hv, dv, std=0.7)
            u = torch.rand(B, generator=h).tolist()
            s["accepted"] = torch.tensor([int(r * (n + 1)) - 1 for r, n in zip(u, counts)], dtype=torch.int32).to(DEV)
        return s
    L, S, n = case["layers"], case["slots"], case["moved"]
    s["pool"] = normal(L, S, case["heads"], case["dk"], case["dv"])
    order = torch.randperm(S, generator=h)
    if kind == "copy":
        s["src"] = torch.randint(0, S, (n,), generator=h).to(torch.int32).to(DEV)
        s["dst"] = order[:n].to(torch.int32).to(DEV)
        return s
    # fork and compact keep `moved` slots free; free takes `moved` of the live ones
    live = torch.ones(S, dtype=torch.int32)
    if kind != "free":
        live[order[:n]] = 0
    used = order[n:] if kind != "free" else order
    s["live0"] = live.to(DEV)
    s["live"] = live.to(DEV)
    if kind == "compact":
        s["idx0"] = used.to(torch.int32).to(DEV)
        s["idx"] = s["idx0"].clone()
    elif kind == "fork":
        s["src"] = used[torch.randint(0, used.numel(), (n,), generator=h)].to(torch.int32).to(DEV)
    else:
        s["gone"] = used[:n].to(torch.int32).to(DEV)
    return s


# ---------------------------------------------------------------------------------- the package's calls

def _run_own(s):
    import kimi_delta_attention_23_b200 as kda
    c = s["case"]
    kind = c["kind"]
    if kind.startswith("glr"):
        kw = dict(gate_mode=c["gate"], beta_mode=c["beta"], input_mode=c["input"], gate_lower_bound=LOWER)
        params = (s["raw"], s["beta"], s["a_log"], s["dt_bias"])
        out_type = TYPES[c["out"]]
        if kind == "glr_decode":
            out = kda.kda_glr_decode(s["x"], *params, s["pool"], s["idx"], output_dtype=out_type, **kw)
            return {"out": out, "pool": s["pool"]}
        if kind == "glr_fwd":
            out = kda.kda_glr_fwd(s["x"], *params, s["cu"], s["pool"], s["idx"], output_dtype=out_type, **kw)
            return {"out": out, "pool": s["pool"]}
        s["pool"].copy_(s["carried"])
        kept = torch.empty(kda.kda_glr_checkpoint_shape(c["tokens"], c["seqs"], c["heads"], c["d"]), device=DEV)
        out = kda.kda_glr_fwd(s["x"], *params, s["cu"], s["pool"], s["idx"], output_dtype=out_type, checkpoints=kept, **kw)
        grads = kda.kda_glr_bwd(s["dout"], s["x"], *params, s["cu"], kept, s["dfinal"], **kw)
        if c["out"] == "f32":
            # the plain form adds the final states' gradients into an fp32 dout, where the next pass on the
            # same state finds them; the two go on from the same dout only if this does so too, every pass anew
            first, end = s["cu"][:-1], s["cu"][1:]
            s["dout"].index_add_(0, (end - 1).clamp_min(0), s["dfinal"] * (end > first)[:, None, None])
        return {"out": out, "pool": s["pool"], **grads}
    if kind == "tree":
        out, deltas = kda.kda_tree_decode(
            s["q"], s["k"], s["v"], s["raw"], s["beta"], s["a_log"], s["dt_bias"], s["cu"], s["parents"], s["pool"],
            s["idx"], max_nodes=c["nodes"], output_dtype=TYPES[c["out"]], gate_mode=c["gate"], beta_mode=c["beta"],
            state_layout=c["layout"], gate_lower_bound=LOWER)
        return {"out": out, "deltas": deltas}
    if kind == "commit":
        kda.kda_tree_commit(s["k"], s["raw"], s["a_log"], s["dt_bias"], s["deltas"], s["cu"], s["parents"], s["accepted"],
                            s["pool"], s["idx"], max_nodes=c["nodes"], gate_mode=c["gate"], state_layout=c["layout"],
                            gate_lower_bound=LOWER)
        return {"pool": s["pool"]}
    pool = s["pool"]
    if kind == "copy":
        kda.kda_pool_copy(pool, s["src"], s["dst"], stacked=True)
        return {"pool": pool}
    s["live"].copy_(s["live0"])
    if kind == "fork":
        dst = kda.kda_pool_fork(pool, s["live"], s["src"], stacked=True)
        return {"pool": pool, "live": s["live"], "dst": dst}
    if kind == "free":
        kda.kda_pool_free(pool, s["live"], s["gone"], stacked=True)
        return {"pool": pool, "live": s["live"]}
    s["idx"].copy_(s["idx0"])
    count = kda.kda_pool_compact(pool, s["live"], s["idx"], stacked=True)
    return {"pool": pool, "live": s["live"], "idx": s["idx"], "count": count}


# ---------------------------------------------------------------------------------- the plain forms

def _softplus(z):
    return z.clamp_min(0) + torch.log1p(torch.exp(-z.abs()))


def _sigmoid(z):
    e = torch.exp(-z.abs())
    return torch.where(z >= 0, 1 / (1 + e), e / (1 + e))


def _gate(case, raw, a_log, dt_bias):
    """(g, whether the clamp left it alone) of every token, head and channel."""
    g = -torch.exp(a_log)[:, None] * _softplus(raw.float() + dt_bias)
    return (g.clamp_min(LOWER), g > LOWER) if case["gate"] == "safe" else (g, None)


def _scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t along the first axis, by doubling; a is zero where a sequence starts."""
    step = 1
    while step < longest:
        b = torch.cat([b[:step], b[step:] + a[step:] * b[:-step]])
        a = torch.cat([a[:step], a[step:] * a[:-step]])
        step *= 2
    return b


def _glr_plain(s):
    c = s["case"]
    decode = c["kind"] == "glr_decode"
    T = c["tokens"]
    x = s["x"].float()
    g, free = _gate(c, s["raw"], s["a_log"], s["dt_bias"])
    a = torch.exp(g)
    beta = (_sigmoid(s["beta"]) if c["beta"] == "logits" else s["beta"])[..., None]
    scale = torch.sqrt(-torch.expm1(2 * g)) if c["input"] == "norm" else torch.ones_like(g)
    b = beta * scale * x
    if c["kind"] == "glr_train":
        s["pool"].copy_(s["carried"])
    start = s["pool"][s["idx"]]
    if decode:
        h = a * start + b
        s["pool"][s["idx"]] = h
        return {"out": h.to(TYPES[c["out"]]), "pool": s["pool"]}
    cu = s["cu"].long()
    some = cu[1:] > cu[:-1]
    first, last = cu[:-1][some], cu[1:][some] - 1
    before = torch.zeros_like(b)  # the state before each sequence's first token
    before[first] = start[some]
    inner = a.clone()
    inner[first] = 0
    h = _scan(inner, b + a * before, s["longest"])
    slots = s["idx"].long()[some]
    s["pool"][slots] = h[last]
    res = {"out": h.to(TYPES[c["out"]]), "pool": s["pool"]}
    if c["kind"] == "glr_fwd":
        return res
    before[1:] += h[:-1] * (inner[1:] != 0)
    dh = s["dout"].float()
    dh[last] += s["dfinal"][some]
    following = torch.cat([inner[1:], torch.zeros_like(inner[:1])])
    dh = _scan(following.flip(0), dh.flip(0), s["longest"]).flip(0)
    dg = dh * a * before
    if c["input"] == "norm":
        dg = dg - dh * beta * x * torch.where(scale > 0, a * a / scale, 0.0)
    if free is not None:
        dg = dg * free
    z = s["raw"].float() + s["dt_bias"]
    draw_gate = -dg * torch.exp(s["a_log"])[:, None] * _sigmoid(z)
    dbeta = (dh * scale * x).sum(-1)
    if c["beta"] == "logits":
        dbeta = dbeta * beta[..., 0] * (1 - beta[..., 0])
    dinit = s["dfinal"].clone()
    dinit[some] = a[first] * dh[first]
    return {**res, "dx": (dh * beta * scale).to(s["x"].dtype), "draw_gate": draw_gate.to(s["raw"].dtype), "dbeta": dbeta,
            "da_log": (dg * g).double().sum((0, 2)).float(), "ddt_bias": draw_gate.double().sum(0).float(), "d_initial": dinit}


def _tree_parts(s):
    """The trees padded to one size: node numbers, which of them exist, who is whose ancestor, and the
    gates summed along each node's path (in 64 bits: differences of long sums are taken)."""
    c = s["case"]
    B, N, M = c["seqs"], c["nodes"], s["parents"].numel()
    cu = s["cu"].long()
    at = torch.arange(N, device=DEV)
    there = at < (cu[1:] - cu[:-1])[:, None]
    node = (cu[:-1, None] + at).clamp_max(max(0, M - 1))
    parent = torch.where(there, s["parents"].long()[node], -1)
    above = (parent[..., None] == at) | torch.eye(N, dtype=torch.bool, device=DEV)
    step = 1
    while step < N:  # ancestors twice as far up with each product
        above = (above.float() @ above.float()) > 0
        step *= 2
    above = above & there[:, :, None] & there[:, None, :]
    g, _ = _gate(c, s["raw"], s["a_log"], s["dt_bias"])
    path = torch.einsum("bij,bjhc->bhic", above.double(), g[node].double())
    return node, there, above, path


def _tree_plain(s):
    c = s["case"]
    N, heads, group = c["nodes"], c["heads"], c["heads"] // c["kheads"]
    if s["parents"].numel() == 0:
        return {"out": s["v"].to(TYPES[c["out"]]), "deltas": s["v"].float()}
    node, there, above, path = _tree_parts(s)
    rows = lambda x, n: x.float().repeat_interleave(n, 1)[node].transpose(1, 2)  # noqa: E731
    q, k, v = rows(s["q"], group), rows(s["k"], group), rows(s["v"], 1)
    beta = (_sigmoid(s["beta"]) if c["beta"] == "logits" else s["beta"])[node].transpose(1, 2)[..., None]
    state = s["pool"][s["idx"]]
    if c["layout"] == "V_FIRST":
        state = state.transpose(2, 3)
    down = path.exp().float()
    between = (path[:, :, :, None] - path[:, :, None]).masked_fill_(~above[:, None, :, :, None], -math.inf).float().exp_()
    between = between * k[:, :, None]
    strict = above & ~torch.eye(N, dtype=torch.bool, device=DEV)
    low = -beta * (between @ k[..., None])[..., 0] * strict[:, None]
    score = (between @ q[..., None])[..., 0] * above[:, None]
    u = beta * (v - (k * down) @ state)
    step = 1
    while step < N:  # (I - low)^-1 u, low being nilpotent: (I + low)(I + low^2)(I + low^4) ... u
        u = u + low @ u
        low = low @ low
        step *= 2
    out = (q * down) @ state + score @ u
    flat = lambda x: x.transpose(1, 2)[there]  # noqa: E731
    return {"out": flat(out).to(TYPES[c["out"]]), "deltas": flat(u)}


def _commit_plain(s):
    c = s["case"]
    group = c["heads"] // c["kheads"]
    if s["parents"].numel() == 0:
        return {"pool": s["pool"]}
    node, there, above, path = _tree_parts(s)
    taken = s["accepted"].long()
    some = taken >= 0
    last = taken.clamp_min(0)
    rows = torch.arange(c["seqs"], device=DEV)
    on = above[rows, last][:, None, :, None]
    total = path[rows, :, last][:, :, None]
    k = s["k"].float().repeat_interleave(group, 1)[node].transpose(1, 2)
    k = k * (total - path).masked_fill(~on, -math.inf).float().exp()
    u = s["deltas"][node].transpose(1, 2) * on
    slots = s["idx"].long()
    state = s["pool"][slots]
    if c["layout"] == "V_FIRST":
        state = state.transpose(2, 3)
    new = total.exp().float().transpose(2, 3) * state + k.transpose(2, 3) @ u
    new = torch.where(some[:, None, None, None], new, state)
    s["pool"][slots] = new if c["layout"] == "K_FIRST" else new.transpose(2, 3)
    return {"pool": s["pool"]}


def _pool_plain(s):
    kind, pool = s["case"]["kind"], s["pool"]
    if kind == "copy":
        pool[:, s["dst"].long()] = pool[:, s["src"].long()]
        return {"pool": pool}
    live = s["live"].copy_(s["live0"])
    if kind == "free":
        gone = s["gone"].long()
        pool[:, gone] = 0
        live[gone] = 0
        return {"pool": pool, "live": live}
    if kind == "fork":
        dst = torch.sort(live, stable=True).indices[: s["src"].numel()]
        pool[:, dst] = pool[:, s["src"].long()]
        live[dst] = 1
        return {"pool": pool, "live": live, "dst": dst.int()}
    idx = s["idx"].copy_(s["idx0"])
    at = torch.arange(live.numel(), device=DEV)
    count = (live != 0).sum()
    holes = ((live == 0) & (at < count)).nonzero()[:, 0]
    movers = ((live != 0) & (at >= count)).nonzero()[:, 0]
    pool[:, holes] = pool[:, movers]
    at[movers] = holes
    idx.copy_(at[idx.long()])
    live.copy_(torch.arange(live.numel(), device=DEV) < count)
    return {"pool": pool, "live": live, "idx": idx, "count": count.int().reshape(1)}


def run(state):
    if own:
        return _run_own(state)
    kind = state["case"]["kind"]
    if kind.startswith("glr"):
        return _glr_plain(state)
    if kind == "tree":
        return _tree_plain(state)
    return _commit_plain(state) if kind == "commit" else _pool_plain(state)


# ---------------------------------------------------------------------------------- work

def work(case):
    kind = case["kind"]
    if kind.startswith("glr"):
        n, rows = case["tokens"] * case["heads"] * case["d"], case["tokens"] * case["heads"] * 4
        x, raw, out = BYTES[case["x"]], BYTES[case["raw"]], BYTES[case["out"]]
        states = 2 * 4 * case["seqs"] * case["heads"] * case["d"]
        if kind != "glr_train":
            return {"bytes": n * (x + raw + out) + rows + states, "flops": 12 * n}
        return {"bytes": n * (2 * x + 2 * raw + 2 * out) + 2 * rows + 2 * states, "flops": 50 * n}
    if kind in ("tree", "commit"):
        M, B = sum(_counts(case)), case["seqs"]
        Hk, Hv, dk, dv = case["kheads"], case["heads"], case["dk"], case["dv"]
        x = BYTES[case["x"]]
        state = 4 * B * Hv * dk * dv
        if kind == "tree":
            token = M * (2 * Hk * dk * x + Hv * (dv * x + 4 * dk + 4 + dv * (BYTES[case["out"]] + 4) + 4))
            return {"bytes": state + token, "flops": 4 * M * Hv * dk * dv}
        return {"bytes": 2 * state + M * (Hk * dk * x + Hv * 4 * (dk + dv)) // 2, "flops": 2 * B * Hv * dk * dv + M * Hv * dk * dv}
    slot = 4 * case["layers"] * case["heads"] * case["dk"] * case["dv"]
    if kind == "compact":  # about the share of the kept slots that lie behind the packed part
        moved = case["moved"] * (case["slots"] - case["moved"]) / case["slots"]
        return {"bytes": 2 * slot * moved + 8 * case["slots"], "flops": 0}
    return {"bytes": (1 if kind == "free" else 2) * slot * case["moved"] + 4 * case["slots"], "flops": 0}


# ---------------------------------------------------------------------------------- exact values

def _exact_gate(case, raw, a_log, dt_bias):
    z = raw.double() + dt_bias.double()
    raw_g = -a_log.double().exp()[:, None] * torch.logaddexp(z, torch.zeros_like(z))
    return z, raw_g, raw_g.clamp_min(LOWER) if case["gate"] == "safe" else raw_g


def _exact_beta(case, beta):
    return 1 / (1 + (-beta.double()).exp()) if case["beta"] == "logits" else beta.double()


def _exact_glr(case, s):
    z, raw_g, g = _exact_gate(case, s["raw"], s["a_log"], s["dt_bias"])
    a, beta = g.exp(), _exact_beta(case, s["beta"])[..., None]
    scale = (-(2 * g).expm1()).sqrt() if case["input"] == "norm" else torch.ones_like(g)
    w = beta * scale * s["x"].double()
    pool, idx = s["pool"].double(), s["idx"].tolist()
    if case["kind"] == "glr_decode":
        h = a * pool[idx] + w
        pool[idx] = h
        return {"out": h, "pool": pool}
    cu, h = s["cu"].tolist(), torch.empty_like(a)
    before = torch.empty_like(a) if case["kind"] == "glr_train" else None
    for b, slot in enumerate(idx):
        now = pool[slot].clone()
        for t in range(cu[b], cu[b + 1]):
            if before is not None:
                before[t] = now
            now = torch.addcmul(w[t], a[t], now, out=h[t])
        pool[slot] = now
    res = {"out": h, "pool": pool}
    if case["kind"] == "glr_fwd":
        return res
    dh, dinit = s["dout"].double(), s["dfinal"].double()
    for b in range(len(idx)):
        now = dinit[b]
        for t in range(cu[b + 1] - 1, cu[b] - 1, -1):
            dh[t] += now
            now = a[t] * dh[t]
        dinit[b] = now
    x = s["x"].double()
    dg = dh * a * before
    if case["input"] == "norm":
        dg += dh * beta * x * torch.where(scale > 0, -(2 * g).exp() / scale, 0.0)
    if case["gate"] == "safe":
        dg *= raw_g > LOWER
    draw_gate = -dg * s["a_log"].double().exp()[:, None] / (1 + (-z).exp())
    dbeta = (dh * scale * x).sum(-1)
    if case["beta"] == "logits":
        dbeta *= (beta * (1 - beta))[..., 0]
    return {**res, "dx": dh * beta * scale, "draw_gate": draw_gate, "dbeta": dbeta, "da_log": (dg * g).sum((0, 2)),
            "ddt_bias": draw_gate.sum(0), "d_initial": dinit}


def _exact_tree(case, s):
    """Token by token: every node's own state from its parent's."""
    group, dk, dv = case["heads"] // case["kheads"], case["dk"], case["dv"]
    _, _, g = _exact_gate(case, s["raw"], s["a_log"], s["dt_bias"])
    k = s["k"].double().repeat_interleave(group, 1)
    cu, parents, counts = s["cu"].tolist(), s["parents"].tolist(), _counts(case)
    start = s["pool"].double()
    start = start if case["layout"] == "K_FIRST" else start.transpose(2, 3)
    start = start[s["idx"].long()].clone()
    M = len(parents)
    if case["kind"] == "commit":
        for b, last in enumerate(s["accepted"].tolist()):
            path = []
            while last >= 0:
                path.insert(0, cu[b] + last)
                last = parents[cu[b] + last]
            for m in path:
                start[b] = g[m].exp()[..., None] * start[b] + k[m][..., None] * s["deltas"][m].double()[:, None]
        pool = s["pool"].double()
        pool[s["idx"].long()] = start if case["layout"] == "K_FIRST" else start.transpose(2, 3)
        return {"pool": pool}
    q, v, beta = s["q"].double().repeat_interleave(group, 1), s["v"].double(), _exact_beta(case, s["beta"])
    kept = torch.empty(M + 1, case["heads"], dk, dv, dtype=torch.float64, device=DEV)
    out, deltas = torch.empty(2, M, case["heads"], dv, dtype=torch.float64, device=DEV)
    for i in range(case["nodes"]):  # the i-th nodes of all trees at once
        seqs = [b for b, n in enumerate(counts) if n > i]
        if not seqs:
            break
        m = [cu[b] + i for b in seqs]
        up = torch.tensor([parents[x] for x in m], device=DEV)
        base = torch.tensor([cu[b] for b in seqs], device=DEV)
        S = torch.where((up < 0)[:, None, None, None], start[seqs], kept[base + up.clamp_min(0)])
        S = g[m].exp()[..., None] * S
        u = beta[m][..., None] * (v[m] - torch.einsum("mhc,mhcv->mhv", k[m], S))
        S = S + k[m][..., None] * u[:, :, None]
        kept[m], deltas[m] = S, u
        out[m] = torch.einsum("mhc,mhcv->mhv", q[m], S)
    return {"out": out, "deltas": deltas}


def exact(case, seed):
    """The definitions, one token after the other, in 64 bits; slots that only move have no computed value."""
    if case["kind"] in ("copy", "fork", "free", "compact"):
        return None
    s = prepare(case, seed)
    return _exact_glr(case, s) if case["kind"].startswith("glr") else _exact_tree(case, s)
