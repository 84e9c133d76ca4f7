"""The state scan (lores_scan_forward, lores_scan_backward) against its recurrence in 64 bits.

Tolerances (relative 2-norm).  fp32 results: operands carry 22 bits (2^-22 relative to their scale) and a product drops
a term of the same size, so a product is off by at most 3 * 2^-22; no result is more than about a dozen
products deep, and the norms of what is added are of the result's size: 12 * 3 * 2^-22 = 8.6e-6.
16-bit results add their own rounding, eps/2, and o's two products of one fp16 plane each, whose operands
are off by 2^-11 at most.
"""
import pytest
import torch

from .scan_reference import inputs, rel, scan64

pytestmark = pytest.mark.gpu

FP32 = 12 * 3 * 2.0 ** -22
NAMES = ("q", "k", "v", "log_alpha", "beta", "state")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def lib():
    from bit_recurrent_state_lores_b200 import lores
    return lores


def tol(dtype, planes=False):
    if dtype == torch.float32:
        return FP32
    return torch.finfo(dtype).eps / 2 + (2 * 2.0 ** -11 if planes else FP32)


def strided(x, stride, dtype):
    """x [T, h, d] as rows of `stride` elements (the rest holds NaN)."""
    T, h, d = x.shape
    buf = torch.full((T, stride), float("nan"), device=x.device, dtype=dtype)
    buf[:, :h * d] = x.reshape(T, h * d).to(dtype)
    return buf


class Call:
    """One call's buffers; forward() and backward() run it."""

    def __init__(self, x, offsets, delta, dtype, pad=0, max_len=0, with_offsets=True, device_offsets=None):
        L = self.L = lib()
        self.x, self.offs, self.dtype, self.pad = x, offsets, dtype, pad
        (self.T, self.Hq, self.dk), (_, self.H, self.dv) = x["q"].shape, x["v"].shape
        self.N = x["state"].shape[0]
        self.wq, self.wv = self.Hq * self.dk + pad, self.H * self.dv + pad
        self.cfg = L.make_scan_config(self.N, self.T, self.H, self.dk, self.dv, heads_qk=self.Hq,
                                      delta=delta, dtype=dtype, max_len=max_len, q_stride=self.wq,
                                      k_stride=self.wq, v_stride=self.wv, o_stride=self.wv)
        self.q, self.k = (strided(x[n], self.wq, dtype) for n in "qk")
        self.v = strided(x["v"], self.wv, dtype)
        self.la, self.be = x["log_alpha"].float().contiguous(), x["beta"].float().contiguous()
        self.state = x["state"].float().contiguous()
        o = torch.tensor(offsets if device_offsets is None else device_offsets, dtype=torch.int32)
        self.offsets = o.cuda() if with_offsets else None
        self.o = torch.full((self.T, self.wv), 777.0, device="cuda", dtype=dtype)
        self.state_out = torch.full_like(self.state, 777.0)
        self.work = None

    def workspace(self, backward):
        n = self.L.lores_scan_workspace(self.cfg, backward)
        if self.work is None or self.work.numel() < n:
            # filled with NaN patterns: nothing may be read that was not written
            self.work = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
        return self.work

    def rows(self, buf, h, d):
        return buf[:, :h * d].reshape(self.T, h, d)

    def forward(self, state_in=True, state_out=True, stream=None):
        self.L.lores_scan_forward(self.cfg, self.q, self.k, self.v, self.la, self.be, self.offsets,
                                  self.state if state_in else None, self.o,
                                  self.state_out if state_out else None, self.workspace(False), stream=stream)
        return self.rows(self.o, self.H, self.dv), self.state_out

    def backward(self, d_o, d_state, state_in=True, d_state_in=True):
        self.d_o = strided(d_o, self.wv, self.dtype)
        self.d_state_out = None if d_state is None else d_state.float().contiguous()
        f = lambda *s, t=self.dtype: torch.full(s, 777.0, device="cuda", dtype=t)  # noqa: E731
        self.dq, self.dk_, self.dv_ = f(self.T, self.wq), f(self.T, self.wq), f(self.T, self.wv)
        self.dla, self.dbe = f(self.T, self.H, t=torch.float32), f(self.T, self.H, t=torch.float32)
        self.ds = f(*self.state.shape, t=torch.float32)
        self.L.lores_scan_backward(self.cfg, self.q, self.k, self.v, self.la, self.be, self.offsets,
                                   self.state if state_in else None, self.d_o, self.d_state_out,
                                   self.dq, self.dk_, self.dv_, self.dla, self.dbe,
                                   self.ds if d_state_in else None, self.workspace(True))
        return {"q": self.rows(self.dq, self.Hq, self.dk), "k": self.rows(self.dk_, self.Hq, self.dk),
                "v": self.rows(self.dv_, self.H, self.dv), "log_alpha": self.dla, "beta": self.dbe,
                "state": self.ds}

    def check(self):
        return self.L.lores_scan_check_errors(self.cfg, self.work)


# lens, H, Hq, d_k, d_v, delta, dtype, pad
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
SHAPES = [
    ([1], 1, 1, 16, 4, 1, F32, 0),
    ([64], 2, 2, 128, 128, 1, BF16, 0),
    ([65], 2, 1, 128, 128, 1, BF16, 0),
    ([63, 1, 64, 0, 130], 3, 3, 64, 20, 1, F32, 0),
    ([17, 200, 5], 4, 2, 128, 100, 1, BF16, 0),
    ([33, 128, 129], 4, 1, 32, 36, 1, F16, 8),
    ([90, 0, 70], 2, 2, 16, 128, 1, F32, 4),
    ([130], 6, 2, 64, 132, 1, BF16, 4),
    ([70, 257], 4, 4, 128, 64, 0, BF16, 0),
    ([100, 31], 8, 1, 128, 12, 0, F32, 0),
    ([66, 66], 2, 2, 16, 16, 0, F16, 12),
    ([320], 2, 2, 32, 260, 0, BF16, 8),
    ([128], 2, 2, 128, 16, 1, F32, 0),
]
IDS = ["%s-H%d/%d-%dx%d-d%d-%s-p%d" % ("_".join(map(str, s[0])), s[1], s[2], s[3], s[4], s[5],
                                       str(s[6])[6:], s[7]) for s in SHAPES]


@pytest.mark.parametrize("lens,H,Hq,dk,dv,delta,dtype,pad", SHAPES, ids=IDS)
def test_forward(lens, H, Hq, dk, dv, delta, dtype, pad):
    x, offs = inputs(lens, H, Hq, dk, dv, dtype, seed=dk + dv, lead=3, trail=2)
    c = Call(x, offs, delta, dtype, pad)
    o, S = c.forward()
    ro, rS = scan64(*(x[n] for n in NAMES[:5]), offs, x["state"], delta)
    a, b = offs[0], offs[-1]
    assert rel(o[a:b], ro[a:b]) <= tol(dtype, planes=True)
    assert rel(S, rS) <= FP32
    # tokens of no sequence and what lies between the rows stay as they were
    assert (o[:a] == 777).all() and (o[b:] == 777).all()
    assert (c.o[:, H * dv:] == 777).all()
    assert c.check() == c.L.LORES_OK
    # no first state: zeros; no last state wanted
    o0, S0 = c.forward(state_in=False)
    ro0, rS0 = scan64(*(x[n] for n in NAMES[:5]), offs, torch.zeros_like(x["state"]), delta)
    assert rel(o0[a:b], ro0[a:b]) <= tol(dtype, planes=True) and rel(S0, rS0) <= FP32
    S0 = S0.clone()
    c.state_out.fill_(777)
    c.forward(state_in=False, state_out=False)
    assert (c.state_out == 777).all()


@pytest.mark.parametrize("lens,H,Hq,dk,dv,delta,dtype,pad", SHAPES, ids=IDS)
def test_backward(lens, H, Hq, dk, dv, delta, dtype, pad):
    x, offs = inputs(lens, H, Hq, dk, dv, dtype, seed=dk + dv + 1, lead=2, trail=3)
    c = Call(x, offs, delta, dtype, pad)
    g = torch.Generator().manual_seed(5)
    d_o = torch.randn(x["v"].shape, generator=g).to(dtype).double().cuda()
    d_S = torch.randn(x["state"].shape, generator=g).double().cuda()
    got = c.backward(d_o, d_S)
    leaves = [x[n].clone().requires_grad_(True) for n in NAMES]
    o, S = scan64(*leaves[:5], offs, leaves[5], delta)
    a, b = offs[0], offs[-1]
    want = dict(zip(NAMES, torch.autograd.grad((o[a:b] * d_o[a:b]).sum() + (S * d_S).sum(), leaves,
                                               allow_unused=True)))
    for n in NAMES:
        # a gate's gradient sums terms of either sign: its error is measured against the terms, which are
        # of the size of the gradients of the tensors it multiplies (at most 4 times it here)
        t = tol(dtype) if n in "qkv" else 4 * FP32 if n in ("log_alpha", "beta") else FP32
        if n == "state":
            assert rel(got[n], want[n]) <= t, n
        else:
            assert rel(got[n][a:b], want[n][a:b]) <= t, n
            assert (got[n][:a] == 777).all() and (got[n][b:] == 777).all(), n
    for buf, w in ((c.dq, Hq * dk), (c.dk_, Hq * dk), (c.dv_, H * dv)):
        assert (buf[:, w:] == 777).all()
    assert c.check() == c.L.LORES_OK


def test_gradient_against_differences():
    # the directional derivative of the kernel's own loss along a random direction, by central differences.
    # The loss is a sum of 1e4 fp32 terms of relative error FP32; over a step h its difference is
    # off by FP32 |loss terms| / h plus h^2 of third derivatives
    x, offs = inputs([70, 40], 2, 1, 32, 24, F32, seed=3)
    g = torch.Generator().manual_seed(9)
    rnd = lambda t: torch.randn(t.shape, generator=g).double().cuda()  # noqa: E731
    d_o, d_S = rnd(x["v"]), rnd(x["state"])
    got = Call(x, offs, 1, F32).backward(d_o, d_S)
    for n in NAMES:
        way = rnd(x[n]) * (0.1 if n in ("log_alpha", "beta") else 1.0)
        h = 2.0 ** -8
        loss = []
        for s in (1, -1):
            y = dict(x)
            y[n] = x[n] + s * h * way
            o, S = Call(y, offs, 1, F32).forward()
            loss.append(float((o.double() * d_o).sum() + (S.double() * d_S).sum()))
        slope = (loss[0] - loss[1]) / (2 * h)
        want = float((got[n].double() * way).sum())
        size = float((got[n].double().norm() * way.norm()))
        assert abs(slope - want) <= 2e-2 * size, n


def test_no_gradient_of_the_last_state_and_none_for_the_first():
    x, offs = inputs([100], 2, 2, 64, 32, F32, seed=4)
    d_o = torch.randn(x["v"].shape, generator=torch.Generator().manual_seed(1)).double().cuda()
    c = Call(x, offs, 1, F32)
    got = {n: t.clone() for n, t in c.backward(d_o, torch.zeros_like(x["state"])).items()}
    again = c.backward(d_o, None)
    for n in NAMES:
        assert torch.equal(got[n], again[n]), n
    none = c.backward(d_o, None, d_state_in=False)
    assert (c.ds == 777).all()
    for n in NAMES[:5]:
        assert torch.equal(got[n], none[n]), n


@pytest.mark.parametrize("dk,dv,delta,dtype", [(128, 128, 1, BF16), (256, 64, 1, F32), (16, 12, 0, F16),
                                               (64, 100, 1, F32)])
def test_token_by_token_kernel(dk, dv, delta, dtype):
    """Short sequences (and d_k = 256) take another kernel: same results."""
    lens = [1, 16, 0, 5] if dk < 256 else [1, 40, 0, 9]
    x, offs = inputs(lens, 4, 2, dk, dv, dtype, seed=dk, lead=1, trail=1)
    c = Call(x, offs, delta, dtype, pad=4, max_len=max(lens))
    o, S = c.forward()
    ro, rS = scan64(*(x[n] for n in NAMES[:5]), offs, x["state"], delta)
    a, b = offs[0], offs[-1]
    assert rel(o[a:b], ro[a:b]) <= tol(dtype)
    assert rel(S, rS) <= FP32
    assert (o[:a] == 777).all() and (o[b:] == 777).all()
    if dk < 256:
        d = Call(x, offs, delta, dtype, pad=4)               # the chunk kernels on the same call
        o2, S2 = d.forward()
        assert rel(o2[a:b], o[a:b]) <= 2 * tol(dtype, planes=True) and rel(S2, S) <= 2 * FP32


def test_one_token_at_a_time_equals_one_call():
    x, offs = inputs([90], 2, 2, 64, 64, F32, seed=8)
    whole = Call(x, offs, 1, F32)
    o, S = whole.forward()
    state = x["state"].clone()
    for t in range(90):
        y = {n: (v[t:t + 1] if n != "state" else state) for n, v in x.items()}
        c = Call(y, [0, 1], 1, F32, max_len=1)
        ot, st = c.forward()
        assert rel(ot[0], o[t]) <= 2 * FP32 * 4
        state = st.double()
    assert rel(state, S) <= 2 * FP32


def test_equals_the_decode_steps_of_an_fp32_handle():
    L = lib()
    H, dk, dv, T = 4, 64, 32, 70
    x, offs = inputs([T, T], H, H, dk, dv, F32, seed=12)
    o, S = Call(x, offs, 1, F32).forward()
    h = L.lores_create(2, H, dk, dv, head_bits=[32] * H)
    try:
        L.lores_load_state(h, x["state"].float().contiguous(), 0)
        tm = lambda n: torch.stack([x[n][:T], x[n][T:]], 1).float().contiguous()  # noqa: E731
        out = torch.empty(T, 2, H, dv, device="cuda")
        L.lores_decode_steps(h, T, tm("q"), tm("k"), tm("v"), torch.exp(tm("log_alpha")), tm("beta"), out, 0)
        back = torch.empty(2, H, dv, dk, device="cuda")
        L.lores_dequant_state(h, back)
        assert rel(o, torch.cat([out[:, 0], out[:, 1]])) <= 2 * FP32
        assert rel(S, back) <= 2 * FP32
    finally:
        L.lores_destroy(h)


@pytest.mark.parametrize("delta", [0, 1])
def test_decays_that_drop_or_keep_the_state(delta):
    """log_alpha of -infinity, of -1e4 and of 0; beta of 0; k of 0."""
    x, offs = inputs([150], 2, 2, 32, 16, F32, seed=21)
    la = x["log_alpha"]
    la[10], la[64], la[65], la[100] = -float("inf"), -float("inf"), -float("inf"), -1e4
    la[20:30] = 0.0
    x["beta"][5] = 0.0
    x["beta"][70] = 0.0
    x["k"][40] = 0.0
    c = Call(x, offs, delta, F32)
    o, S = c.forward()
    ro, rS = scan64(*(x[n] for n in NAMES[:5]), offs, x["state"], delta)
    assert rel(o, ro) <= FP32 and rel(S, rS) <= FP32
    g = torch.Generator().manual_seed(2)
    d_o = torch.randn(x["v"].shape, generator=g).double().cuda()
    d_S = torch.randn(x["state"].shape, generator=g).double().cuda()
    got = c.backward(d_o, d_S)
    leaves = [x[n].clone().requires_grad_(True) for n in NAMES]
    leaves[3] = torch.where(la < -1000, torch.full_like(la, -1000.0), la).requires_grad_(True)
    o, S = scan64(*leaves[:5], offs, leaves[5], delta)
    want = dict(zip(NAMES, torch.autograd.grad((o * d_o).sum() + (S * d_S).sum(), leaves)))
    for n in NAMES:
        t = 4 * FP32 if n in ("log_alpha", "beta") else FP32
        assert rel(got[n], want[n]) <= t, n
    assert (got["log_alpha"][[10, 64, 65, 100]].abs() <= 1e-30).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("vs,ss,ds", [(1e8, 1.0, 1e-9), (1e-8, 1e-8, 1e7), (1.0, 1e6, 1.0), (0.0, 1.0, 1.0),
                                      (1e-6, 0.0, 0.0)])
def test_magnitudes(dtype, vs, ss, ds):
    """Values, states and gradients far from one: the scales are powers of two and leave no trace."""
    x, offs = inputs([130], 2, 2, 64, 48, dtype, seed=31)
    x["v"] = (x["v"] * vs).to(dtype).double()
    x["state"] = (x["state"] * ss).float().double()
    c = Call(x, offs, 1, dtype)
    o, S = c.forward()
    ro, rS = scan64(*(x[n] for n in NAMES[:5]), offs, x["state"], 1)
    assert rel(o, ro) <= tol(dtype, planes=True) and rel(S, rS) <= FP32
    g = torch.Generator().manual_seed(2)
    d_o = (torch.randn(x["v"].shape, generator=g) * ds).to(dtype).double().cuda()
    d_S = (torch.randn(x["state"].shape, generator=g) * ds).float().double().cuda()
    got = c.backward(d_o, d_S)
    leaves = [x[n].clone().requires_grad_(True) for n in NAMES]
    ro, rS = scan64(*leaves[:5], offs, leaves[5], 1)
    want = dict(zip(NAMES, torch.autograd.grad((ro * d_o).sum() + (rS * d_S).sum(), leaves)))
    for n in NAMES:
        t = tol(dtype) if n in "qkv" else 4 * FP32 if n in ("log_alpha", "beta") else FP32
        assert rel(got[n], want[n]) <= t, n


def test_q_and_k_of_other_norms():
    # (without the delta rule k need not be of unit norm)
    for scale in (1e-3, 40.0):
        x, offs = inputs([100], 2, 1, 64, 32, F32, seed=33)
        x["q"], x["k"] = (x[n] * scale for n in "qk")
        x["q"], x["k"] = (x[n].float().double() for n in "qk")
        o, S = Call(x, offs, 0, F32).forward()
        ro, rS = scan64(*(x[n] for n in NAMES[:5]), offs, x["state"], 0)
        # with small k the new terms are small beside the state and v: held against those (2^-25 of v k)
        assert rel(o, ro) <= FP32 and rel(S, rS) <= FP32


def test_constant_inputs_that_all_add_up():
    # every product of the same sign: the largest sums the scales have to leave room for
    x, offs = inputs([200], 2, 2, 128, 128, F32, seed=1)
    for n in "qk":
        x[n] = torch.full_like(x[n], 1.0).div(128 ** 0.5).float().double()
    x["v"].fill_(1.0)
    x["state"].fill_(1.0)
    x["log_alpha"].zero_()
    x["beta"].fill_(1.0)
    for delta in (0, 1):
        c = Call(x, offs, delta, F32)
        o, S = c.forward()
        ro, rS = scan64(*(x[n] for n in NAMES[:5]), offs, x["state"], delta)
        assert rel(o, ro) <= FP32 and rel(S, rS) <= FP32
        got = c.backward(torch.ones_like(x["v"]), torch.ones_like(x["state"]))
        leaves = [x[n].clone().requires_grad_(True) for n in NAMES]
        ro, rS = scan64(*leaves[:5], offs, leaves[5], delta)
        want = dict(zip(NAMES, torch.autograd.grad(ro.sum() + rS.sum(), leaves)))
        for n in NAMES:
            # (with the delta rule some of these gradients cancel to zero: measured against dv's size then)
            size = max(float(want[n].norm()), float(want["v"].norm()))
            if n == "log_alpha":
                # <dL/dS'_t, S'_t> of each token sums d_k d_v products of entries of size one, which here cancel
                # (k never changes, so a token replaces all that the state holds along it): it is off by FP32 of the
                # sum of their magnitudes, d_k d_v, in each of the T H entries
                size = max(size, 128 * 128 * (200 * 2) ** 0.5)
            assert float((got[n].double() - want[n]).norm()) <= 4 * FP32 * size, (delta, n)


def test_non_finite_values_stay_in_their_sequence_and_row():
    x, offs = inputs([100, 100, 100], 2, 2, 32, 32, F32, seed=41)
    ro, rS = scan64(*(x[n] for n in NAMES[:5]), offs, x["state"], 1)
    x["v"][130, 1, 5] = float("nan")
    x["v"][20, 0, 3] = float("inf")
    c = Call(x, offs, 1, F32)
    o, S = c.forward()
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[100:200, 1, 5] = False
    keep[0:100, 0, 3] = False
    # 16 value rows share a scale: an infinity takes the rows of its block with it
    keep[100:200, 1, :16] = False
    keep[0:100, 0, :16] = False
    assert torch.isfinite(o[keep]).all()
    assert rel(o[keep], ro[keep]) <= FP32
    assert not torch.isfinite(o[130:200, 1, 5]).any() and not torch.isfinite(o[20:100, 0, 3]).any()
    assert rel(S[2], rS[2]) <= FP32


def test_bad_offsets_are_empty_and_reported():
    x, offs = inputs([80, 90, 70], 2, 2, 32, 16, F32, seed=51)
    for bad, wrong in (([0, 80, 75, 240], [1]), ([0, 80, 170, 999], [2]), ([-5, 80, 170, 240], [0]),
                       ([0, 80, 2**31 - 1, 240], [1, 2])):
        c = Call(x, offs, 1, F32, device_offsets=bad)
        o, S = c.forward()
        assert c.check() == c.L.LORES_ERR_INVALID_ARG
        for i in range(3):
            if i in wrong:
                assert torch.equal(S[i], c.state[i])
        good = [i for i in range(3) if i not in wrong and bad[i] == offs[i] and bad[i + 1] == offs[i + 1]]
        for i in good:
            y = {n: (v[offs[i]:offs[i + 1]] if n != "state" else v[i:i + 1]) for n, v in x.items()}
            ro, rS = scan64(*(y[n] for n in NAMES[:5]), [0, offs[i + 1] - offs[i]], y["state"], 1)
            assert rel(S[i:i + 1], rS) <= FP32
        c.backward(torch.ones_like(x["v"]), torch.ones_like(x["state"]))
        assert c.check() == c.L.LORES_ERR_INVALID_ARG
    # longer than max_len
    c = Call(x, offs, 1, F32, max_len=85)
    o, S = c.forward()
    assert c.check() == c.L.LORES_ERR_INVALID_ARG
    assert torch.equal(S[1], c.state[1]) and not torch.equal(S[0], c.state[0])
    c = Call(x, offs, 1, F32, max_len=10)
    o, S = c.forward()
    assert c.check() == c.L.LORES_ERR_INVALID_ARG and torch.equal(S, c.state)


def test_without_offsets_and_without_tokens():
    x, offs = inputs([50, 50, 50], 2, 1, 64, 32, BF16, seed=61)
    a = Call(x, offs, 1, BF16)
    b = Call(x, offs, 1, BF16, with_offsets=False)
    for p, q in zip(a.forward(), b.forward()):
        assert torch.equal(p, q)
    # no tokens at all: states are copied, gradients of states pass through
    L = lib()
    S = torch.randn(2, 2, 16, 32, device="cuda")
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    out, din = torch.empty_like(S), torch.empty_like(S)
    for max_len in (0, 8):
        cfg = L.make_scan_config(2, 0, 2, 32, 16, max_len=max_len)
        work = torch.empty(L.lores_scan_workspace(cfg, True), dtype=torch.uint8, device="cuda")
        out.zero_()
        L.lores_scan_forward(cfg, None, None, None, None, None, offsets, S, None, out, work)
        assert torch.equal(out, S)
        L.lores_scan_backward(cfg, None, None, None, None, None, offsets, S, None, S, None, None, None, None,
                              None, din, work)
        assert torch.equal(din, S)


def test_states_in_place():
    x, offs = inputs([100, 30], 2, 2, 64, 32, BF16, seed=71)
    for max_len, lens in ((0, None), (16, [16, 3])):
        if lens:
            x, offs = inputs(lens, 2, 2, 64, 32, BF16, seed=72)
        a, b = (Call(x, offs, 1, BF16, max_len=max_len) for _ in range(2))
        a.forward()
        b.state_out = b.state
        b.forward()
        assert torch.equal(a.o, b.o) and torch.equal(a.state_out, b.state)
    x, offs = inputs([100, 30], 2, 2, 64, 32, BF16, seed=71)
    d_o, d_S = x["v"].clone(), x["state"].clone()
    c = Call(x, offs, 1, BF16)
    want = {n: t.clone() for n, t in c.backward(d_o, d_S).items()}
    buf = c.d_state_out
    c.L.lores_scan_backward(c.cfg, c.q, c.k, c.v, c.la, c.be, c.offsets, c.state, c.d_o, buf, c.dq, c.dk_, c.dv_,
                            c.dla, c.dbe, buf, c.work)
    assert torch.equal(buf, want["state"]) and torch.equal(c.rows(c.dq, 2, 64), want["q"])


def test_equal_calls_give_equal_bits():
    x, offs = inputs([300, 77], 4, 2, 128, 64, BF16, seed=81)
    c = Call(x, offs, 1, BF16)
    o, S = (t.clone() for t in c.forward())
    g = {n: t.clone() for n, t in c.backward(x["v"], x["state"]).items()}
    for _ in range(3):
        c.work.fill_(0xFF)
        o2, S2 = c.forward()
        assert torch.equal(o, o2) and torch.equal(S, S2)
        for n, t in c.backward(x["v"], x["state"]).items():
            assert torch.equal(g[n], t), n


@pytest.mark.parametrize("lens,max_len", [([200, 70], 0), ([7, 3], 8)])
def test_graph_capture_and_other_streams(lens, max_len):
    x, offs = inputs(lens, 2, 2, 64, 32, BF16, seed=91)
    y, _ = inputs(lens, 2, 2, 64, 32, BF16, seed=92)
    want_x, want_y = (Call(z, offs, 1, BF16, max_len=max_len) for z in (x, y))
    for w in (want_x, want_y):
        w.forward()
    # on a side stream, two calls at once with a workspace each
    s = [torch.cuda.Stream(), torch.cuda.Stream()]
    cs = [Call(z, offs, 1, BF16, max_len=max_len) for z in (x, y)]
    for c in cs:
        c.workspace(False)
    torch.cuda.synchronize()
    for _ in range(3):
        for c, st in zip(cs, s):
            c.forward(stream=st)
    torch.cuda.synchronize()
    assert torch.equal(cs[0].o, want_x.o) and torch.equal(cs[1].o, want_y.o)
    # captured once, replayed on other inputs
    c = Call(x, offs, 1, BF16, max_len=max_len)
    d_o, d_S = x["v"], x["state"]
    c.forward()
    c.backward(d_o, d_S)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    st = torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=st):
        c.L.lores_scan_forward(c.cfg, c.q, c.k, c.v, c.la, c.be, c.offsets, c.state, c.o, c.state_out, c.work)
        c.L.lores_scan_backward(c.cfg, c.q, c.k, c.v, c.la, c.be, c.offsets, c.state, c.d_o, c.d_state_out, c.dq,
                                c.dk_, c.dv_, c.dla, c.dbe, c.ds, c.work)
    for n, buf in (("q", c.q), ("k", c.k), ("v", c.v)):
        buf.copy_({"q": want_y.q, "k": want_y.k, "v": want_y.v}[n])
    c.la.copy_(want_y.la)
    c.be.copy_(want_y.be)
    c.state.copy_(want_y.state)
    c.o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    T, w = c.T, c.H * c.dv
    assert torch.equal(c.o[:, :w], want_y.o[:, :w]) and torch.equal(c.state_out, want_y.state_out)
    want = Call(y, offs, 1, BF16, max_len=max_len)
    want.workspace(True)
    g = want.backward(d_o, d_S)
    assert torch.equal(c.rows(c.dq, c.Hq, c.dk), g["q"]) and torch.equal(c.dla, g["log_alpha"])


def test_many_short_and_one_long_sequence():
    lens = [1, 2, 3, 0, 64, 1, 500, 5, 0, 0, 17] * 3
    x, offs = inputs(lens, 2, 1, 32, 8, F32, seed=101)
    c = Call(x, offs, 1, F32)
    o, S = c.forward()
    ro, rS = scan64(*(x[n] for n in NAMES[:5]), offs, x["state"], 1)
    assert rel(o, ro) <= FP32 and rel(S, rS) <= FP32


def test_a_long_sequence_with_a_state_that_does_not_decay():
    # 4096 tokens without decay: rounding must not pile up in the state
    x, offs = inputs([4096], 1, 1, 16, 4, F32, seed=111)
    x["log_alpha"].zero_()
    o, S = Call(x, offs, 0, F32).forward()
    w = x["beta"][:, 0, None] * x["v"][:, 0]
    rS = x["state"][0, 0] + w.T @ x["k"][:, 0]
    assert rel(S[0, 0], rS) <= FP32


@pytest.mark.parametrize("delta", [0, 1])
@pytest.mark.parametrize("longest", [24, 25, 32, 33])
def test_lengths_around_the_change_of_kernels(longest, delta):
    lens = [longest, 3, 0, longest - 1]
    x, offs = inputs(lens, 2, 1, 64, 36, BF16, seed=120 + longest)
    c = Call(x, offs, delta, BF16, max_len=longest)
    o, S = c.forward()
    ro, rS = scan64(*(x[n] for n in NAMES[:5]), offs, x["state"], delta)
    assert rel(o, ro) <= tol(BF16, planes=True) and rel(S, rS) <= FP32
    assert c.check() == c.L.LORES_OK


@pytest.mark.parametrize("dv,dtype", [(64, BF16), (80, F16), (64, F32)])
def test_enough_heads_for_several_rounds(dv, dtype):
    """Enough heads that CTAs take four blocks of value rows (the last CTA of a walk not all of them) and the
    preparation two heads."""
    x, offs = inputs([300, 33, 1, 130], 128, 2, 16, dv, dtype, seed=dv)
    names = [x[n].requires_grad_() for n in NAMES]
    ro, rS = scan64(*names[:5], offs, names[5], 0)
    g = torch.Generator().manual_seed(3)
    d_o = torch.randn(ro.shape, generator=g).to(dtype).double().cuda()
    d_S = torch.randn(rS.shape, generator=g).double().cuda()
    want = torch.autograd.grad([ro, rS], names, [d_o, d_S])
    x = {n: t.detach() for n, t in x.items()}
    c = Call(x, offs, 0, dtype, pad=8)
    o, S = c.forward()
    assert rel(o, ro.detach()) <= tol(dtype, planes=True) and rel(S, rS.detach()) <= FP32
    got = c.backward(d_o, d_S)
    for n, w in zip(NAMES, want):
        t = tol(dtype) if n in "qkv" else 4 * FP32 if n in ("log_alpha", "beta") else FP32
        assert rel(got[n], w) <= t, n
    assert c.check() == c.L.LORES_OK


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_the_widest_values(dtype):
    x, offs = inputs([70, 5], 1, 1, 64, 4096, dtype, seed=131)
    names = [x[n].requires_grad_() for n in NAMES]
    ro, rS = scan64(*names[:5], offs, names[5], 1)
    d_o = torch.randn(ro.shape, generator=torch.Generator().manual_seed(4)).to(dtype).double().cuda()
    want = torch.autograd.grad([ro], names, [d_o])
    x = {n: t.detach() for n, t in x.items()}
    c = Call(x, offs, 1, dtype)
    o, S = c.forward()
    assert rel(o, ro.detach()) <= tol(dtype, planes=True) and rel(S, rS.detach()) <= FP32
    got = c.backward(d_o, None)
    for n, w in zip(NAMES, want):
        t = tol(dtype) if n in "qkv" else 4 * FP32 if n in ("log_alpha", "beta") else FP32
        assert rel(got[n], w) <= t, n


@pytest.mark.parametrize("max_len", [0, 8])
def test_rows_beyond_32_bits(max_len):
    """Token rows so far apart that the last ones lie past 2^31 elements: same bits as back to back."""
    L = lib()
    T, n_seq, stride = 144, (18 if max_len else 2), 16_000_000
    x, offs = inputs([T // n_seq] * n_seq, 2, 2, 64, 64, BF16, seed=141)
    near = Call(x, offs, 1, BF16, max_len=max_len)
    o, S = (t.clone() for t in near.forward())
    g = {n: t.clone() for n, t in near.backward(x["v"], x["state"]).items()}
    ins, outs = (torch.zeros(T * stride, dtype=BF16, device="cuda") for _ in range(2))
    assert (T - 1) * stride > 2 ** 31

    def rows(buf, i):                                    # the i-th tensor: 128 columns from 128 i on
        return torch.as_strided(buf, (T, 128), (stride, 1), 128 * i)

    for i, n in enumerate("qkv"):
        rows(ins, i).copy_(getattr(near, n))
    rows(ins, 3).copy_(near.d_o)
    cfg = L.make_scan_config(n_seq, T, 2, 64, 64, dtype=BF16, max_len=max_len, q_stride=stride, k_stride=stride,
                             v_stride=stride, o_stride=stride)
    q, k, v, d_o = (rows(ins, i) for i in range(4))
    far_S = torch.empty_like(S)
    L.lores_scan_forward(cfg, q, k, v, near.la, near.be, near.offsets, near.state, rows(outs, 0), far_S, near.work)
    assert torch.equal(rows(outs, 0), o.reshape(T, 128)) and torch.equal(far_S, S)
    dla, dbe, ds = (torch.empty_like(t) for t in (near.dla, near.dbe, near.ds))
    L.lores_scan_backward(cfg, q, k, v, near.la, near.be, near.offsets, near.state, d_o, near.d_state_out,
                          rows(outs, 1), rows(outs, 2), rows(outs, 3), dla, dbe, ds, near.work)
    for i, n in enumerate("qkv"):
        assert torch.equal(rows(outs, 1 + i), g[n].reshape(T, 128)), n
    assert torch.equal(dla, g["log_alpha"]) and torch.equal(dbe, g["beta"]) and torch.equal(ds, g["state"])
    assert int(torch.count_nonzero(outs.view(T, stride)[:, 512:1024])) == 0


@pytest.mark.parametrize("dk,dv,lens,delta", [(128, 128, [300, 77], 1), (64, 100, [300], 1), (128, 64, [150, 77], 0),
                                              (16, 16, [300], 1), (32, 4, [9, 30], 1)])
def test_fp16_outputs_are_off_by_their_rounding(dk, dv, lens, delta):
    """With y the fp32 result, |o - exact| <= |round(y) - y| + |y - exact|; y is so near the exact value that it
    rounds another way for less than 1 entry in 100 (FP32 against the 2^-11 between roundings)."""
    x, offs = inputs(lens, 4, 2, dk, dv, F16, seed=150 + dk)
    o, _ = Call(x, offs, delta, F16).forward()
    ro, _ = scan64(*(x[n] for n in NAMES[:5]), offs, x["state"], delta)
    assert rel(o, ro) <= 1.01 * rel(ro.half(), ro) + FP32


@pytest.mark.parametrize("lens,H", [([300, 77], 4), ([40], 2), ([1000, 30], 64)])
def test_calls_one_behind_the_other(lens, H):
    """Kernels of a call may overlap, those of two calls may not: two problems in turn on one workspace, without waiting."""
    xs = [inputs(lens, H, H // 2, 64, 64, BF16, seed=160 + i) for i in range(2)]
    cs = [Call(x, offs, 1, BF16) for x, offs in xs]
    cs[1].work = cs[0].workspace(True)
    want = []
    for c in cs:
        o, S = (t.clone() for t in c.forward())
        g = {n: t.clone() for n, t in c.backward(c.x["v"], c.x["state"]).items()}
        torch.cuda.synchronize()
        want.append((o, S, g))
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(40):
        c, (o, S, g) = cs[i % 2], want[i % 2]
        for _ in range(2):
            c.forward()
            got = c.backward(c.x["v"], c.x["state"])
        o2, S2 = c.forward()
        bad += (o2 != o).sum() + (S2 != S).sum() + sum((got[n] != g[n]).sum() for n in NAMES)
    assert int(bad) == 0
