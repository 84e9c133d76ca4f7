"""The state scan's recurrence (General recurrence form, without the quantizer) in 64 bits, one token after
another, for packed sequences; gradients come from differentiating it."""
import torch


def scan64(q, k, v, log_alpha, beta, offsets, state, delta):
    """o [T, H, d_v] and last states [N, H, d_v, d_k] in fp64 (differentiable)."""
    H = v.shape[1]
    share = H // q.shape[1]
    q, k = q.repeat_interleave(share, 1), k.repeat_interleave(share, 1)
    outs, states = {}, []
    for i in range(len(offsets) - 1):
        S = state[i]
        for t in range(offsets[i], offsets[i + 1]):
            S = S * torch.exp(log_alpha[t])[:, None, None]
            u = torch.einsum("hvk,hk->hv", S, k[t]) if delta else 0.0
            w = beta[t][:, None] * (v[t] - u)
            S = S + w[:, :, None] * k[t][:, None, :]
            outs[t] = torch.einsum("hvk,hk->hv", S, q[t])
        states.append(S)
    zero = torch.zeros_like(v[0]) if len(v) else None
    o = torch.stack([outs.get(t, zero) for t in range(len(v))]) if len(v) else v * 1.0
    return o, torch.stack(states)


def inputs(lens, H, Hq, dk, dv, dtype, seed=0, lead=0, trail=0, decay=1.0, device="cuda"):
    """Tensors of a call in fp64 that `dtype` holds exactly: tokens of no sequence in front and behind."""
    g = torch.Generator().manual_seed(seed)
    T, N = lead + sum(lens) + trail, len(lens)
    r = lambda *s: torch.randn(*s, generator=g, dtype=torch.float64)  # noqa: E731
    unit = torch.nn.functional.normalize
    x = {"q": unit(r(T, Hq, dk), dim=-1), "k": unit(r(T, Hq, dk), dim=-1), "v": r(T, H, dv)}
    x = {n: t.to(dtype).double() for n, t in x.items()}
    x["log_alpha"] = (-torch.nn.functional.softplus(r(T, H) - 1.0) * decay).float().double()
    x["beta"] = torch.sigmoid(r(T, H)).float().double()
    x["state"] = (0.5 * r(N, H, dv, dk)).float().double()
    offsets = [lead]
    for n in lens:
        offsets.append(offsets[-1] + n)
    return {n: t.to(device) for n, t in x.items()}, offsets


def rel(a, b):
    """|a - b| / |b| in the 2-norm (|a| where b is zero)."""
    a, b = a.double(), b.double()
    n = float(b.norm())
    return float((a - b).norm()) / n if n else float(a.norm())
