"""Plain 64-bit forms of the operators around the state pools, one token after the other, on the CPU.

Nothing here calls the package.  Everything is written in torch with gradients, so the reference
gradients of the recurrence come from differentiating its definition.
"""
import torch


def rel(x, ref):
    """Relative L2 distance; infinite where one is finite and the other is not."""
    x, ref = torch.as_tensor(x).double().cpu(), torch.as_tensor(ref).double().cpu()
    assert x.shape == ref.shape
    if not torch.equal(torch.isfinite(x), torch.isfinite(ref)):
        return float("inf")
    n = float(ref.norm())
    return float((x - ref).norm()) / (n if n > 0 else 1.0)


def gate(raw, a_log, dt_bias, mode, lower):
    z = raw + dt_bias
    g = -a_log.exp()[:, None] * torch.logaddexp(z, torch.zeros_like(z))
    # the clamp passes no gradient where it acts
    return torch.where(g > lower, g, torch.full_like(g, lower)) if mode == "safe" else g


def beta_of(logits, mode):
    return torch.sigmoid(logits) if mode == "logits" else logits


def glr(x, raw, beta_logits, a_log, dt_bias, lengths, initial, *, gate_mode="original", beta_mode="logits",
        input_mode="unit", lower=-5.0):
    """(out [T,H,d], final states [B,H,d]) of the recurrence from ``initial`` [B,H,d], in 64 bits."""
    g = gate(raw, a_log, dt_bias, gate_mode, lower)
    a = g.exp()
    w = beta_of(beta_logits, beta_mode)[..., None] * x
    if input_mode == "norm":
        w = w * torch.sqrt(-torch.expm1(2 * g))
    out, final, t = [], [], 0
    for b, n in enumerate(lengths):
        h = initial[b]
        for _ in range(n):
            h = a[t] * h + w[t]
            out.append(h)
            t += 1
        final.append(h)
    return (torch.stack(out) if out else torch.zeros_like(x)), torch.stack(final)


def kda_step(S, q, k, v, g, beta):
    """One token of one head set: S [H,dk,dv] -> (S', o [H,dv], delta [H,dv])."""
    S = g.exp()[..., None] * S
    delta = beta[..., None] * (v - torch.einsum("hc,hcv->hv", k, S))
    S = S + k[..., None] * delta[:, None]
    return S, torch.einsum("hc,hcv->hv", q, S), delta


def tree(q, k, v, raw, beta_logits, a_log, dt_bias, counts, parents, states, *, gate_mode="original",
         beta_mode="logits", lower=-5.0):
    """(out, deltas, every node's state as a list per sequence); states [B,Hv,dk,dv], all in 64 bits."""
    Hv = v.shape[1]
    q, k = (t.repeat_interleave(Hv // t.shape[1], 1) for t in (q, k))
    g, beta = gate(raw, a_log, dt_bias, gate_mode, lower), beta_of(beta_logits, beta_mode)
    out, deltas = torch.zeros(v.shape, dtype=torch.float64), torch.zeros(v.shape, dtype=torch.float64)
    kept, m = [], 0
    for b, n in enumerate(counts):
        nodes = []
        for i in range(n):
            p = int(parents[m])
            S, out[m], deltas[m] = kda_step(states[b] if p < 0 else nodes[p], q[m], k[m], v[m], g[m], beta[m])
            nodes.append(S)
            m += 1
        kept.append(nodes)
    return out, deltas, kept
