"""What is measured of the state scan, its backward pass and the state pool's write and read.

Every case is one of four kinds:
  scan    a run of new tokens of every sequence through the gated linear recurrence
          S_t = S_{t-1} a_t (I - d b_t k_t k_t^T) + b_t v_t k_t^T,  o_t = S_t q_t
          (the decode step's recurrence without the quantizer), packed sequences, fp32 state
          carried in and out
  grad    the backward pass of the same call
  store   states of some sequences quantized into the slots of a layer's pool and read back
          (prefill -> decode handoff, a paused sequence that comes back)
  fetch   states of some slots read back alone

`run` computes them from elementary torch operations in 32 bits, or, with `own`, through the
library's calls; `exact` computes them token by token in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
CHUNK = 64                          # tokens that the plain form takes at a time, at most


# -------------------------------------------------------------------------------------
# the cases
# -------------------------------------------------------------------------------------
def _scan(name, kind, seqs, longest, shortest, heads, heads_qk, d_k, d_v, delta, dtype, decay):
    return {"name": name, "kind": kind, "seqs": seqs, "longest": longest, "shortest": shortest,
            "heads": heads, "heads_qk": heads_qk, "d_k": d_k, "d_v": d_v, "delta": delta,
            "dtype": dtype, "decay": decay}


def _pool(name, kind, slots, taken, heads, d_k, d_v, group, bits, stochastic, dtype):
    return {"name": name, "kind": kind, "slots": slots, "taken": taken, "heads": heads,
            "d_k": d_k, "d_v": d_v, "group": group, "bits": bits, "stochastic": stochastic,
            "dtype": dtype}


def listed():
    return [
        # one token of one sequence, state kept in fp32: the latency of a single step
        _scan("scan_1x1", "scan", 1, 1, 1, 32, 32, 128, 128, 1, "bf16", "tau"),
        # a few drafted tokens of a decoding batch, checked in one call
        _scan("scan_64x5", "scan", 64, 5, 2, 32, 16, 128, 128, 1, "bf16", "tau"),
        # a scheduler's ragged prefill batch
        _scan("scan_ragged", "scan", 12, 700, 17, 16, 16, 128, 128, 1, "bf16", "softplus"),
        # one long prompt, layer of 32 heads of 128 x 128
        _scan("scan_8k", "scan", 1, 8192, 8192, 32, 32, 128, 128, 1, "bf16", "tau"),
        # no delta rule, 128 heads that share 8 pairs of q and k
        _scan("scan_nodelta", "scan", 4, 2048, 1900, 128, 8, 128, 64, 0, "bf16", "tau"),
        # fp32 activations and a value width that is no power of two
        _scan("scan_fp32", "scan", 6, 530, 300, 8, 8, 64, 100, 1, "fp32", "softplus"),
        # training: a toy layer in fp32
        _scan("grad_small", "grad", 2, 130, 61, 4, 4, 64, 64, 1, "fp32", "softplus"),
        # training: a layer of 16 heads on 8 pairs of q and k
        _scan("grad_4k", "grad", 2, 4096, 4096, 16, 8, 128, 128, 1, "bf16", "tau"),
        # training without the delta rule, one pair of q and k for 16 heads each, ragged
        _scan("grad_nodelta", "grad", 3, 3000, 1700, 64, 4, 128, 64, 0, "bf16", "tau"),
        # handoff of a prefilled batch into the int8 pool of a layer, one scale per row
        _pool("store_64", "store", 256, 64, 32, 128, 128, 128, 8, 1, "fp32"),
        # one sequence of an int4 layer with a scale per 32 keys
        _pool("store_1", "store", 16, 1, 32, 128, 128, 32, 4, 1, "fp32"),
        # states of a batch read back in 16 bits
        _pool("fetch_96", "fetch", 128, 96, 32, 128, 128, 128, 8, 1, "bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["scan", "scan", "grad", "grad", "store", "fetch"])
    d_k = rng.choice([16, 32, 64, 128, 128])
    if kind in ("store", "fetch"):
        slots = _log_int(rng, 1, 160)
        return {"kind": kind, "slots": slots, "taken": rng.randint(1, slots),
                "heads": rng.randint(1, 32), "d_k": d_k, "d_v": 4 * rng.randint(1, 32),
                "group": rng.choice([g for g in (16, 32, 64, 128) if g <= d_k]),
                "bits": rng.choice([4, 8]), "stochastic": rng.choice([0, 1]),
                "dtype": rng.choice(["fp32", "bf16"]) if kind == "fetch" else "fp32"}
    heads_qk = rng.choice([1, 2, 3, 4, 8])
    heads = heads_qk * rng.choice([1, 1, 2, 4])
    d_v = 4 * rng.randint(2, 32)
    most = 8192 * 32 * 128 * 128 / (heads * d_k * d_v) / (1 if kind == "scan" else 4)
    seqs = _log_int(rng, 1, 24)
    longest = _log_int(rng, 1, max(1, min(8192, int(most / seqs))))
    return {"kind": kind, "seqs": seqs, "longest": longest, "shortest": rng.randint(0, longest),
            "heads": heads, "heads_qk": heads_qk, "d_k": d_k, "d_v": d_v,
            "delta": rng.choice([0, 1, 1]), "dtype": rng.choice(["bf16", "bf16", "fp32", "fp16"]),
            "decay": rng.choice(["tau", "softplus"])}


def _lengths(case):
    """Sequence lengths of a case: the longest first, the shortest last, spread between."""
    n, a, b = case["seqs"], case["longest"], case["shortest"]
    if n == 1:
        return [a]
    return [a - (a - b) * ((i * 5) % n if 0 < i < n - 1 else i) // (n - 1) for i in range(n)]


def work(case):
    H, dk, dv = case["heads"], case["d_k"], case["d_v"]
    if case["kind"] in ("store", "fetch"):
        entries = case["taken"] * H * dk * dv
        code = entries * case["bits"] // 8 + entries // case["group"] * 4
        wide = entries * DTYPES[case["dtype"]].itemsize
        if case["kind"] == "store":       # states in, codes and scales out, and back again
            return {"bytes": 2 * (wide + code), "flops": 4 * entries}
        return {"bytes": wide + code, "flops": entries}
    T, w = sum(_lengths(case)), DTYPES[case["dtype"]].itemsize
    hq = case["heads_qk"]
    states = case["seqs"] * H * dk * dv * 4
    tokens = T * (2 * hq * dk + 2 * H * dv) * w + T * H * 8
    # token by token: a decay, (S'k,) w k^T and S q are 1 + 2 (+ 2) + 2 operations per entry
    flops = T * H * dk * dv * (7 if case["delta"] else 5)
    if case["kind"] == "scan":
        return {"bytes": tokens + 2 * states, "flops": flops}
    # the inputs and d_o and d_state in; dq, dk, dv, the gates' and the state's gradients out
    return {"bytes": T * (4 * hq * dk + 3 * H * dv) * w + T * H * 16 + 3 * states,
            "flops": 3 * flops}


# -------------------------------------------------------------------------------------
# inputs
# -------------------------------------------------------------------------------------
class _Handle:
    """A layer's state pool in the library, released with the state that holds it."""

    def __init__(self, L, case):
        self.L = L
        self.h = L.lores_create(case["slots"], case["heads"], case["d_k"], case["d_v"],
                                group_size=case["group"], head_bits=[case["bits"]] * case["heads"],
                                stochastic=case["stochastic"], seed=POOL_SEED)

    def __del__(self):
        if self.h:
            self.L.lores_destroy(self.h)
            self.h = None


POOL_SEED = 11                      # key of the pool's dither
STEP = 7                            # its rounding counter at the call


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    H, dk, dv = case["heads"], case["d_k"], case["d_v"]
    st = {"case": dict(case)}
    if case["kind"] in ("store", "fetch"):
        n = case["taken"]
        st["slots"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:n].to(torch.int32)
        # states as a layer leaves them: rows of very different sizes
        st["states"] = normal(n, H, dv, dk) * torch.exp(normal(n, H, dv, 1))
        if case["kind"] == "fetch":
            st["codes"], st["scales"] = _quantize(st["states"], st["slots"], case)
            st["out"] = torch.empty(n, H, dv, dk, device="cuda", dtype=DTYPES[case["dtype"]])
            del st["states"]
        else:
            st["out"] = torch.empty(n, H, dv, dk, device="cuda")
        if own:
            from bit_recurrent_state_lores_b200 import lores as L
            st["L"], st["pool"] = L, _Handle(L, case)
            if case["kind"] == "fetch":
                back = st["codes"].float() * st["scales"].repeat_interleave(case["group"], -1)
                L.lores_write_states(st["pool"].h, n, st["slots"], back, STEP)
        return st

    lens = _lengths(case)
    T, N, hq, dt = sum(lens), case["seqs"], case["heads_qk"], DTYPES[case["dtype"]]
    offs = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32)
    unit = torch.nn.functional.normalize
    st["q"] = unit(normal(T, hq, dk), dim=-1).to(dt)
    st["k"] = unit(normal(T, hq, dk), dim=-1).to(dt)
    st["v"] = normal(T, H, dv).to(dt)
    if case["decay"] == "tau":        # time constants log-uniform in [1, 1000] tokens
        tau = torch.exp(torch.rand(H, generator=gen, device="cuda") * math.log(1000.0))
        st["log_alpha"] = (-(0.5 + torch.rand(T, H, generator=gen, device="cuda")) / tau)
    else:
        st["log_alpha"] = -torch.nn.functional.softplus(normal(T, H) - 2.0)
    st["beta"] = torch.sigmoid(normal(T, H))
    st["state"] = normal(N, H, dv, dk) * 0.3
    st["offsets"] = offs.cuda()
    st["longest"] = max(lens)
    st["out"] = torch.empty(T, H, dv, device="cuda", dtype=dt)
    st["state_out"] = torch.empty_like(st["state"])
    if case["kind"] == "grad":
        st["d_out"] = normal(T, H, dv).to(dt)
        st["d_state"] = normal(N, H, dv, dk) * 0.3
        st["grads"] = [torch.empty_like(st[n]) for n in ("q", "k", "v", "log_alpha", "beta",
                                                          "state")]
    if own:
        from bit_recurrent_state_lores_b200 import lores as L
        st["L"] = L
        st["cfg"] = L.make_scan_config(N, T, H, dk, dv, heads_qk=hq, delta=case["delta"],
                                       dtype=dt, max_len=st["longest"])
        size = L.lores_scan_workspace(st["cfg"], backward=case["kind"] == "grad")
        st["work"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return st


# -------------------------------------------------------------------------------------
# the plain forms
# -------------------------------------------------------------------------------------
def _unit_lower_inverse(A):
    """(I + A)^-1 of strictly lower triangular matrices, by halves."""
    n = A.shape[-1]
    if n == 1:
        return torch.ones_like(A)
    m = n // 2
    a, c = _unit_lower_inverse(A[..., :m, :m]), _unit_lower_inverse(A[..., m:, m:])
    low = -(c @ (A[..., m:, :m] @ a))
    top = torch.cat([a, torch.zeros_like(A[..., :m, m:])], -1)
    return torch.cat([top, torch.cat([low, c], -1)], -2)


def _plain_scan(q, k, v, log_alpha, beta, state, offsets, longest, delta):
    """o [T, H, d_v] and the last state, in fp32; up to CHUNK tokens of every sequence at a time."""
    T, H = log_alpha.shape
    N = state.shape[0]
    C = min(CHUNK, 1 << (longest - 1).bit_length())
    share = H // q.shape[1]
    M = -(-longest // C)
    at = offsets[:-1, None].long() + torch.arange(M * C, device=q.device)
    there = at < offsets[1:, None].long()
    at = torch.where(there, at, torch.zeros_like(at))

    def grid(x):                               # [T, h, ...] -> [N, M, h, C, ...]
        y = x[at]
        y = torch.where(there.reshape(N, -1, *[1] * (x.dim() - 1)), y, torch.zeros_like(y))
        return y.reshape(N, M, C, *x.shape[1:]).transpose(2, 3)

    Q, K = (grid(x.repeat_interleave(share, 1)) for x in (q, k))
    V, g, b = grid(v), grid(log_alpha), grid(beta)
    G = torch.cumsum(g.double(), -1)           # sums of logarithms and their differences
    low = torch.ones(C, C, device=q.device, dtype=torch.bool).tril()
    gap = torch.where(low, G[..., :, None] - G[..., None, :], torch.zeros((), device=q.device,
                                                                          dtype=torch.float64))
    decay = torch.where(low, torch.exp(gap).float(), torch.zeros((), device=q.device))
    to_start = torch.exp(G).float()
    to_end = torch.exp(G[..., -1:] - G).float()
    P = (Q @ K.transpose(-1, -2)) * decay * b[..., None, :]
    Qs = Q * to_start[..., None]
    if delta:
        A = ((K @ K.transpose(-1, -2)) * decay * b[..., None, :]).tril(-1)
        inv = _unit_lower_inverse(A)
        Ks = K * to_start[..., None]
    wk = b * to_end
    S, out = state, []
    for m in range(M):
        St = S.transpose(-1, -2)
        E = inv[:, m] @ (V[:, m] - Ks[:, m] @ St) if delta else V[:, m]
        out.append(Qs[:, m] @ St + P[:, m] @ E)
        S = S * to_start[:, m, :, -1, None, None] + (E * wk[:, m, ..., None]).transpose(-1, -2) @ K[:, m]
    o = torch.stack(out, 1).transpose(2, 3).reshape(N, M * C, H, -1)
    return o[there], S


def _mulfold(a, m):
    p = a * m                                  # 64-bit product, low and high halves folded
    return (p ^ (p >> 32)) & 0xFFFFFFFF


def _splitmix64(z):
    m = (1 << 64) - 1
    z = (z + 0x9E3779B97F4A7C15) & m
    z = ((z ^ (z >> 30)) * 0xBF58476D1CE4E5B9) & m
    z = ((z ^ (z >> 27)) * 0x94D049BB133111EB) & m
    return z ^ (z >> 31)


def _fmix32(h):
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & 0xFFFFFFFF
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & 0xFFFFFFFF
    return h ^ (h >> 16)


def _dither(slots, case):
    """The pool's dither bytes [n, H, d_v, d_k] of the slots' entries, 128 without it."""
    n, H, dv, dk = len(slots), case["heads"], case["d_v"], case["d_k"]
    if not case["stochastic"]:
        return torch.full((1, 1, 1, dk), 128, device="cuda", dtype=torch.int64)
    z = _splitmix64(POOL_SEED ^ _splitmix64(STEP))
    key = (z & 0xFFFFFFFF) ^ (z >> 32)
    tile = slots.long()[:, None] * H + torch.arange(H, device="cuda")
    tile = _fmix32((key + 0x85EBCA77 * (tile + 1)) & 0xFFFFFFFF)
    block = (torch.arange(dv, device="cuda")[:, None] * (dk // 16)
             + torch.arange(dk // 16, device="cuda"))
    c = (tile[:, :, None, None] + 0x9E3779B9 * (4 * block + 1)) & 0xFFFFFFFF
    w = _mulfold(c, 0x7FEB352D)
    words = torch.stack([_mulfold(w, m) for m in (0x846CA68B, 0xCC9E2D51, 0x1B873593,
                                                  0xE6546B65)], -1)
    d = torch.stack([(words >> (8 * i)) & 255 for i in range(4)], -1)
    return d.reshape(n, H, dv, dk)


def _scale_of(m, r):
    """The quantizer's scale and inverse scale of a group's largest magnitude m (fp32): the
    state format names every rounding, so each product and fused step is formed in 64 bits
    (exact, or far finer than fp32) and rounded to fp32 once."""
    y = (0x7F000000 - m.view(torch.int32)).view(torch.float32).double()
    md = m.double()
    for _ in range(3):
        e = (1.0 - md * y).float().double()
        y = (y * e + y).float().double()
    inv = (r * y).float()
    return (md * torch.tensor(1.0 / r, dtype=torch.float32).double().item()).float(), inv


def _quantize(states, slots, case):
    """Codes (int8) and scales of the states, by the pool's format."""
    n, H, dv, dk = states.shape
    r = float(2 ** (case["bits"] - 1) - 1)
    x = states.float().reshape(n, H, dv, dk // case["group"], case["group"])
    m = x.abs().amax(-1)
    keep = m >= 2.0 ** -100
    s, inv = _scale_of(torch.where(keep, m, torch.ones_like(m)), r)
    d = _dither(slots, case).reshape(-1, H if case["stochastic"] else 1,
                                     dv if case["stochastic"] else 1, *x.shape[3:])
    t = x.double() * inv[..., None].double() + (49152.0 + d.double() / 256.0)
    code = torch.floor(t.float() - 49152.0)
    code = torch.where(keep[..., None], code, torch.zeros_like(code))
    s = torch.where(keep, s, torch.zeros_like(s))
    return code.to(torch.int8).reshape(n, H, dv, dk), s


def run(st):
    case = st["case"]
    if own:
        return _run_own(st)
    if case["kind"] in ("store", "fetch"):
        if case["kind"] == "store":
            codes, scales = _quantize(st["states"], st["slots"], case)
        else:
            codes, scales = st["codes"], st["scales"]
        back = codes.float() * scales.repeat_interleave(case["group"], -1)
        return back.to(DTYPES[case["dtype"]])
    names = ("q", "k", "v", "log_alpha", "beta", "state")
    x = [st[n].float() for n in names]
    if case["kind"] == "scan":
        o, S = _plain_scan(*x, st["offsets"], st["longest"], case["delta"])
        return {"o": o.to(st["v"].dtype), "state": S}
    x = [t.detach().requires_grad_(True) for t in x]
    o, S = _plain_scan(*x, st["offsets"], st["longest"], case["delta"])
    grads = torch.autograd.grad([o, S], x, [st["d_out"].float(), st["d_state"]],
                                allow_unused=True)
    return {"d_" + n: (torch.zeros_like(st[n]) if g is None else g.to(st[n].dtype))
            for n, g in zip(names, grads)}


def _run_own(st):
    case, L = st["case"], st["L"]
    if case["kind"] == "store":
        L.lores_write_states(st["pool"].h, case["taken"], st["slots"], st["states"], STEP)
        L.lores_read_states(st["pool"].h, case["taken"], st["slots"], st["out"])
        return st["out"]
    if case["kind"] == "fetch":
        L.lores_read_states(st["pool"].h, case["taken"], st["slots"], st["out"])
        return st["out"]
    args = [st[n] for n in ("q", "k", "v", "log_alpha", "beta", "offsets", "state")]
    if case["kind"] == "scan":
        L.lores_scan_forward(st["cfg"], *args, st["out"], st["state_out"], st["work"])
        return {"o": st["out"], "state": st["state_out"]}
    L.lores_scan_backward(st["cfg"], *args, st["d_out"], st["d_state"], *st["grads"], st["work"])
    return dict(zip(("d_q", "d_k", "d_v", "d_log_alpha", "d_beta", "d_state"), st["grads"]))


# -------------------------------------------------------------------------------------
# the definition in 64 bits, one token after another
# -------------------------------------------------------------------------------------
def _tokens(x, offs, longest, fill=0.0):
    """[T, ...] -> [longest, N, ...] in 64 bits, `fill` behind a sequence's end."""
    y = torch.full((longest, len(offs) - 1, *x.shape[1:]), fill, device=x.device,
                   dtype=torch.float64)
    for i in range(len(offs) - 1):
        y[:offs[i + 1] - offs[i], i] = x[offs[i]:offs[i + 1]].double()
    return y


def _packed(y, offs):
    return torch.cat([y[:offs[i + 1] - offs[i], i] for i in range(len(offs) - 1)])


def _step(S, kt, vt, at, bt, delta):
    """(S', E, S_t) of one token: S' = a S, E = v - d S'k, S_t = S' + b E k^T."""
    Sd = S * at[..., None, None]
    E = vt - torch.einsum("nhvk,nhk->nhv", Sd, kt) if delta else vt
    return Sd, E, Sd + torch.einsum("nhv,nhk->nhvk", E * bt[..., None], kt)


def exact(case, seed):
    st = prepare(case, seed)
    if case["kind"] in ("store", "fetch"):
        return _exact_pool(st, case)
    H, offs, L = case["heads"], st["offsets"].tolist(), st["longest"]
    share, delta = H // case["heads_qk"], case["delta"]
    steps = L * (1 if case["kind"] == "scan" else 4)
    if steps * max(1.0, case["seqs"] * H * case["d_k"] * case["d_v"] / 2e6) > 2e5:
        return None
    q, k = (_tokens(st[n], offs, L).repeat_interleave(share, 2) for n in ("q", "k"))
    v, b = _tokens(st["v"], offs, L), _tokens(st["beta"], offs, L)
    a = torch.exp(_tokens(st["log_alpha"], offs, L))
    S = st["state"].double()
    if case["kind"] == "scan":
        o = torch.zeros_like(v)
        for t in range(L):
            S = _step(S, k[t], v[t], a[t], b[t], delta)[2]
            o[t] = torch.einsum("nhvk,nhk->nhv", S, q[t])
        return {"o": _packed(o, offs), "state": S}
    span = max(1, min(128, int(8e9 / (S.numel() * 8))))     # tokens between kept states
    kept = {}
    for t in range(L):
        if t % span == 0:
            kept[t] = S
        S = _step(S, k[t], v[t], a[t], b[t], delta)[2]
    do = _tokens(st["d_out"], offs, L)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(b), torch.zeros_like(b)
    D = st["d_state"].double()
    for t0 in sorted(kept, reverse=True):
        inside, S = [], kept[t0]
        for t in range(t0, min(L, t0 + span)):
            S = _step(S, k[t], v[t], a[t], b[t], delta)[2]
            inside.append(S)
        for t in reversed(range(t0, min(L, t0 + span))):
            S_t, S_p = inside[t - t0], inside[t - t0 - 1] if t > t0 else kept[t0]
            Sd, E, _ = _step(S_p, k[t], v[t], a[t], b[t], delta)
            dq[t] = torch.einsum("nhvk,nhv->nhk", S_t, do[t])
            D = D + torch.einsum("nhv,nhk->nhvk", do[t], q[t])
            dw = torch.einsum("nhvk,nhk->nhv", D, k[t])
            dk[t] = torch.einsum("nhvk,nhv->nhk", D, E * b[t][..., None])
            db[t] = (dw * E).sum(-1)
            dE = dw * b[t][..., None]
            dv[t] = dE
            if delta:
                dk[t] -= torch.einsum("nhvk,nhv->nhk", Sd, dE)
                D = D - torch.einsum("nhv,nhk->nhvk", dE, k[t])
            dg[t] = (D * Sd).sum((-1, -2))
            D = D * a[t][..., None, None]
    shared = lambda x: x.reshape(*x.shape[:2], -1, share, x.shape[-1]).sum(3)  # noqa: E731
    return {"d_q": _packed(shared(dq), offs), "d_k": _packed(shared(dk), offs),
            "d_v": _packed(dv, offs), "d_log_alpha": _packed(dg, offs),
            "d_beta": _packed(db, offs), "d_state": D}


def _exact_pool(st, case):
    """code * scale entry by entry in 64 bits.  The codes belong to the format, which fixes the
    roundings of scale and grid, so those are made here too (to 24 bits of significand)."""
    if case["kind"] == "fetch":
        s = st["scales"].double()[..., None].expand(*st["scales"].shape, case["group"])
        return st["codes"].double() * s.reshape(st["codes"].shape)

    def r24(x):
        f, e = torch.frexp(x)
        return torch.ldexp(torch.round(f * 2.0 ** 24), e - 24)

    x = st["states"].double()
    n, H, dv, dk = x.shape
    r = 2 ** (case["bits"] - 1) - 1
    x = x.reshape(n, H, dv, -1, case["group"])
    m = x.abs().amax(-1, keepdim=True)
    zero = m < 2.0 ** -100
    m = torch.where(zero, torch.ones_like(m), m)
    f, e = torch.frexp(m)                       # m = f 2^e, f in [1/2, 1)
    y = torch.ldexp(3.0 - 2.0 * f, -e)          # exponent and mantissa fields reflected
    for _ in range(3):
        y = r24(y + y * r24(1.0 - m * y))
    d = _dither(st["slots"], case).double()
    d = d.expand(n, H, dv, dk).reshape(x.shape)
    t = torch.round((x * r24(r * y) + 49152.0) * 256.0 + d) / 256.0 - 49152.0
    code = torch.where(zero, torch.zeros_like(t), torch.floor(t))
    s = torch.where(zero, torch.zeros_like(m), r24(m * r24(torch.full_like(m, 1.0 / r))))
    return (code * s).reshape(n, H, dv, dk)
