"""The state scan at the ends of its domain: rounding of 16-bit outputs, magnitudes far from one in a part of the
inputs, values that are not finite, offsets that do not fit.

References and tolerances as in test_gpu_scan: FP32 is what a dozen products of operands of 22 bits may be off by.
"""
import pytest
import torch

from .scan_reference import inputs, rel, scan64
from .test_gpu_scan import BF16, F16, F32, FP32, NAMES, Call, lib, tol

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def normal(like, seed, by=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(like.shape, generator=g, dtype=torch.float64) * by).to(dtype).double().cuda()


def forward64(x, offs, delta):
    return scan64(*(x[n] for n in NAMES[:5]), offs, x["state"], delta)


def backward64(x, offs, delta, d_o, d_S):
    leaves = [x[n].clone().requires_grad_(True) for n in NAMES]
    o, S = scan64(*leaves[:5], offs, leaves[5], delta)
    loss = (o * d_o).sum() if d_S is None else (o * d_o).sum() + (S * d_S).sum()
    return dict(zip(NAMES, torch.autograd.grad(loss, leaves)))


def check_gradients(got, want, dtype, times=1.0):
    # (a gate's gradient sums terms of either sign, up to four times its size: as in test_gpu_scan)
    for n in NAMES:
        t = tol(dtype) if n in "qkv" else FP32
        assert rel(got[n], want[n]) <= t * times * (4 if n in ("log_alpha", "beta") else 1), n


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("dk,dv,lens,delta", [(128, 128, [300, 77], 1), (64, 100, [300], 1), (128, 64, [150, 77], 0),
                                              (16, 16, [300], 1), (32, 4, [9, 130], 1)])
def test_16_bit_outputs_round_the_fp32_result(dk, dv, lens, delta, dtype):
    """An entry x whose fp32 result is off by e rounds to the other neighbour with probability 2 |e| / u at most, u <=
    eps |x| the distance between neighbours, and is then off by u: the squares sum to at most 2 eps sum |e| |x| <=
    2 eps FP32 |x|^2 (Cauchy), beside e itself."""
    x, offs = inputs(lens, 4, 2, dk, dv, dtype, seed=250 + dk)
    o, _ = Call(x, offs, delta, dtype).forward()
    ro, _ = forward64(x, offs, delta)
    assert rel(o, ro.to(dtype)) <= (2 * torch.finfo(dtype).eps * FP32) ** 0.5 + FP32


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("delta,heads_qk", [(1, 2), (1, 1), (0, 2), (0, 1)])
@pytest.mark.parametrize("qs,os,ss", [(4e-3, 1.0, None), (1e-3, 1.0, None), (1e-6, 1.0, None), (1e-6, 1.0, 1.0),
                                      (1e3, 1.0, None), (1e3, 1.0, 1.0), (1.0, 1e-6, 1.0), (1.0, 1.0, 1e-6)])
def test_gradients_of_outputs_and_of_states_of_different_sizes(qs, os, ss, delta, heads_qk, dtype):
    """q far from unit norm, d_o and d_state_out (None: not given) of different sizes."""
    x, offs = inputs([130, 40], 2, heads_qk, 64, 48, dtype, seed=201)
    x["q"] = (x["q"] * qs).to(dtype).double()
    d_o, d_S = normal(x["v"], 7, os, dtype), None if ss is None else normal(x["state"], 8, ss)
    got = Call(x, offs, delta, dtype).backward(d_o, d_S)
    check_gradients(got, backward64(x, offs, delta, d_o, d_S), dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ks", [300.0, 1e3, 3e3, 3e4])
def test_large_keys_inside_the_domain(ks, dtype):
    """|k|^2 beta < 1: v - S k is as large as |k| then, however small beta.  (What carries beta k, of size 1 / (18 |k|),
    is held to an absolute 2^-25 at worst; a dozen such: FP32 |k|.)"""
    x, offs = inputs([150], 2, 1, 64, 48, dtype, seed=211)
    x["k"] = (x["k"] * ks).to(dtype).double()
    x["beta"] = (x["beta"] * 0.9 / ks ** 2).float().double()
    c = Call(x, offs, 1, dtype)
    o, S = c.forward()
    ro, rS = forward64(x, offs, 1)
    assert rel(o, ro) <= tol(dtype) + FP32 * ks and rel(S, rS) <= FP32 * ks
    d_o, d_S = normal(x["v"], 7, 1.0, dtype), normal(x["state"], 8)
    got, want = c.backward(d_o, d_S), backward64(x, offs, 1, d_o, d_S)
    for n in NAMES:
        assert rel(got[n], want[n]) <= tol(dtype) + 4 * FP32 * ks, n


@pytest.mark.parametrize("delta,b", [(1, 1e-2), (1, 1e-4), (1, 1e-6), (1, 1e-12), (0, 1e-2), (0, 1e-6), (0, 1e-12),
                                     (0, 100.0), (0, 1e6)])
@pytest.mark.parametrize("heads_qk", [1, 2])
def test_beta_far_from_one(delta, b, heads_qk):
    """Zero first states, so that every result but dv's part through d_state_out and d_state_in is of beta's size."""
    x, offs = inputs([130, 30], 2, heads_qk, 64, 48, F32, seed=221)
    x["beta"] = (x["beta"] * b).float().double()
    x["state"].zero_()
    c = Call(x, offs, delta, F32)
    o, S = c.forward()
    ro, rS = forward64(x, offs, delta)
    assert rel(o, ro) <= FP32 and rel(S, rS) <= FP32
    d_o, d_S = normal(x["v"], 7), normal(x["state"], 8)
    check_gradients(c.backward(d_o, d_S), backward64(x, offs, delta, d_o, d_S), F32)


@pytest.mark.parametrize("delta", [0, 1])
@pytest.mark.parametrize("ks", [1e-3, 1e-6, 1e-10])
def test_small_keys(ks, delta):
    x, offs = inputs([130], 2, 1, 64, 48, F32, seed=222)
    x["k"] = (x["k"] * ks).float().double()
    x["state"].zero_()
    c = Call(x, offs, delta, F32)
    o, S = c.forward()
    ro, rS = forward64(x, offs, delta)
    assert rel(o, ro) <= FP32 and rel(S, rS) <= FP32
    d_o, d_S = normal(x["v"], 7), normal(x["state"], 8)
    check_gradients(c.backward(d_o, d_S), backward64(x, offs, delta, d_o, d_S), F32)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("ks", [100.0, 1e3, 1e-2])
def test_keys_of_other_norms_inside_the_domain(ks, dtype):
    """|k|^2 beta < 1 is what the delta rule asks for, whatever |k| is."""
    x, offs = inputs([150], 2, 1, 64, 48, dtype, seed=211)
    x["k"] = (x["k"] * ks).to(dtype).double()
    x["beta"] = (x["beta"] * 0.9 / ks ** 2).float().double()
    c = Call(x, offs, 1, dtype)
    o, S = c.forward()
    ro, rS = forward64(x, offs, 1)
    # v - S k and its products carry up to |S k| / |v| times the terms
    assert rel(o, ro) <= tol(dtype) + 3 * FP32 and rel(S, rS) <= 4 * FP32
    d_o, d_S = normal(x["v"], 7, 1.0, dtype), normal(x["state"], 8)
    check_gradients(c.backward(d_o, d_S), backward64(x, offs, 1, d_o, d_S), dtype, 4)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("delta", [0, 1])
def test_equal_queries_and_gradients_that_add_up(delta, dtype):
    """Every q and k alike, d_o all ones, q of norm 50: dv sums as much as it can."""
    x, offs = inputs([200], 2, 2, 128, 32, dtype, seed=212)
    x["k"].fill_(128 ** -0.5)
    x["k"] = x["k"].to(dtype).double()
    x["q"].fill_(50 * 128 ** -0.5)
    x["q"] = x["q"].to(dtype).double()
    x["log_alpha"].zero_()
    x["beta"].fill_(1.0 / 64)
    d_o = torch.ones_like(x["v"])
    got = Call(x, offs, delta, dtype).backward(d_o, None)
    want = backward64(x, offs, delta, d_o, None)
    for n in ("q", "k", "v", "state"):
        assert rel(got[n], want[n]) <= (tol(dtype) if n in "qkv" else FP32) * 4, n
    for n in ("log_alpha", "beta"):
        assert torch.isfinite(got[n]).all(), n


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("delta", [0, 1])
@pytest.mark.parametrize("la", [-20.0, -60.0])
def test_the_first_states_gradient_behind_a_strong_decay(la, delta, dtype):
    """The first token of a chunk fades the state to 1e-9 or 1e-26: so is the gradient, with all its digits."""
    x, offs = inputs([100, 64, 65], 2, 2, 64, 48, dtype, seed=231)
    for t in offs[:3]:
        x["log_alpha"][t] = la
    d_o = normal(x["v"], 7, 1.0, dtype)
    got = Call(x, offs, delta, dtype).backward(d_o, None)
    check_gradients(got, backward64(x, offs, delta, d_o, None), dtype)


@pytest.mark.parametrize("delta,dtype", [(1, F32), (0, F32), (0, BF16)])
@pytest.mark.parametrize("rows", [16, 32])
def test_zero_value_rows_beside_small_ones(rows, delta, dtype):
    """A block of value rows that holds zeros everywhere says nothing about the others' size."""
    x, offs = inputs([130], 2, 1, 64, 64, dtype, seed=235)
    d_o, d_S = normal(x["v"], 7), normal(x["state"], 8, 1e-9)
    for t, by in ((x["v"], 1e-8), (d_o, 1e-9), (x["state"].transpose(2, 3), 1e-8), (d_S.transpose(2, 3), 1.0)):
        t *= by
        t[..., :rows] = 0.0
    x["v"], d_o = x["v"].to(dtype).double(), d_o.to(dtype).double()
    x["state"], d_S = x["state"].float().double(), d_S.float().double()
    got = Call(x, offs, delta, dtype).backward(d_o, d_S)
    check_gradients(got, backward64(x, offs, delta, d_o, d_S), dtype)


@pytest.mark.parametrize("vs,ss,ks,b,delta", [(1e-20, 1e20, 1.0, 1.0, 0), (1e18, 1e-18, 1.0, 1.0, 0),
                                              (1.0, 1.0, 1.0, 1e-25, 1), (1.0, 1.0, 1e-25, 1.0, 1),
                                              (1.0, 1.0, 1e-17, 1e-17, 0)])
def test_gradients_of_parts_of_extreme_sizes(vs, ss, ks, b, delta):
    x, offs = inputs([130], 2, 2, 64, 48, F32, seed=236)
    for n, by in (("v", vs), ("state", ss), ("k", ks), ("beta", b)):
        x[n] = (x[n] * by).float().double()
    c = Call(x, offs, delta, F32)
    o, S = c.forward()
    ro, rS = forward64(x, offs, delta)
    assert rel(o, ro) <= FP32 and rel(S, rS) <= FP32
    d_o, d_S = normal(x["v"], 7), normal(x["state"], 8)
    check_gradients(c.backward(d_o, d_S), backward64(x, offs, delta, d_o, d_S), F32)


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("delta", [0, 1])
def test_queries_of_very_different_sizes(delta, dtype):
    """o_t is linear in q_t: each token's output keeps its digits beside tokens with queries 1e6 times as large."""
    x, offs = inputs([150], 2, 1, 64, 48, dtype, seed=241)
    by = 2.0 ** -(torch.arange(150, device="cuda") * 7 % 21).double()[:, None, None]
    if dtype == F16:
        by = by.clamp(min=2.0 ** -6)                     # (fp16's own range)
    x["q"] = (x["q"] * by).to(dtype).double()
    o, _ = Call(x, offs, delta, dtype).forward()
    ro, _ = forward64(x, offs, delta)
    if dtype == F16:                                     # (outputs below fp16's normal range have its absolute step)
        assert float(((o.double() - ro).abs() - ro.abs() * (2.0 ** -11 + 4 * FP32)).max()) <= 2.0 ** -25 + 8e-6
        return
    for t in range(150):
        for h in range(2):
            assert rel(o[t, h], ro[t, h]) <= tol(dtype), (t, h)


@pytest.mark.parametrize("delta", [0, 1])
def test_small_values_behind_a_dropped_state(delta):
    """v (and d_o) of 1e-5 and 1e-6 of what stands before it in the chunk, and the state dropped between."""
    for by in (1e-5, 1e-6):
        x, offs = inputs([64], 2, 1, 64, 48, F32, seed=242)
        x["v"][32:] *= by
        x["v"] = x["v"].float().double()
        x["log_alpha"][32] = -float("inf")
        o, S = Call(x, offs, delta, F32).forward()
        ro, rS = forward64(x, offs, delta)
        assert rel(o[:32], ro[:32]) <= FP32 and rel(o[32:], ro[32:]) <= FP32 and rel(S, rS) <= FP32


def test_16_bit_inputs_are_exact_far_below_the_chunks_largest():
    """One large entry in each of q, k and v; the others, 2^-20 of it, still count with all their bits."""
    x, offs = inputs([64], 1, 1, 64, 16, BF16, seed=243)
    x["state"].zero_()
    x["beta"].fill_(0.5)
    x["log_alpha"].zero_()
    for n in "qv":
        x[n] = (x[n] * 2.0 ** -20).to(BF16).double()
        x[n][0, 0, 0] = 1.0
    o, _ = Call(x, offs, 0, BF16).forward()
    ro, _ = forward64(x, offs, 0)
    # token 1 on: columns other than the large one's
    assert rel(o[1:, :, 1:], ro[1:, :, 1:]) <= tol(BF16)


def right_or_not_finite(got, want, t):
    """Nothing is a finite number where the recurrence's result is not finite, or another than it."""
    fine = torch.isfinite(want)
    assert not torch.isfinite(got[~fine]).any()
    both = fine & torch.isfinite(got)
    if both.any():
        assert rel(got[both], want[both]) <= t


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("delta", [0, 1])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "beta", "log_alpha", "state", "d_o", "d_state"])
def test_a_value_that_is_not_finite(name, value, delta, dtype):
    x, offs = inputs([150, 70], 4, 2, 64, 36, dtype, seed=251)
    d_o, d_S = normal(x["v"], 7, 1.0, dtype), normal(x["state"], 8)
    clean, clean_S = forward64(x, offs, delta)
    if name == "log_alpha":
        value = float("nan")                                 # (infinities: -inf drops the state, +inf is outside the domain)
    if name == "d_o":
        d_o[90, 1, 5] = value
    elif name == "d_state":
        d_S[0, 1, 5, 7] = value
    elif name == "state":
        x["state"][0, 1, 5, 7] = value
    else:
        x[name][(90, 1) if name in ("beta", "log_alpha") else (90, 0 if name in "qk" else 1, 5)] = value
    c = Call(x, offs, delta, dtype)
    o, S = c.forward()
    ro, rS = forward64(x, offs, delta)
    right_or_not_finite(o, ro, tol(dtype, True))
    right_or_not_finite(S, rS, FP32)
    # chunks before it, other sequences and heads that do not read it are as they were; and so are the tokens of its
    # chunk that it does not reach, where it is q
    heads = [2, 3] if name in "qk" else [0, 2, 3]
    assert rel(o[:, heads], clean[:, heads]) <= tol(dtype, True) and rel(S[:, heads], clean_S[:, heads]) <= FP32
    assert rel(o[150:], clean[150:]) <= tol(dtype, True) and rel(S[1], clean_S[1]) <= FP32
    if name != "state":
        assert rel(o[:64], clean[:64]) <= tol(dtype, True)
    if name in ("q", "d_o", "d_state"):
        others = [t for t in range(220) if t != 90 or name != "q"]
        assert rel(o[others], clean[others]) <= tol(dtype, True) and rel(S, clean_S) <= FP32
    if name in ("v", "state"):
        rows = [r for r in range(36) if r != 5]
        assert rel(o[:, :, rows], clean[:, :, rows]) <= tol(dtype, True)
    got, want = c.backward(d_o, d_S), backward64(x, offs, delta, d_o, d_S)
    for n in NAMES:
        t = tol(dtype) if n in "qkv" else 4 * FP32 if n in ("log_alpha", "beta") else FP32
        right_or_not_finite(got[n], want[n], t)
        last = got[n][1:] if n == "state" else got[n][150:]
        assert torch.isfinite(last).all() and rel(last, want[n][1:] if n == "state" else want[n][150:]) <= t, n
    assert c.check() == c.L.LORES_OK


def one_by_one(x, ranges, delta, d_o, d_S, dtype):
    """Forward and backward of each sequence (begin, end; None: empty) by itself."""
    out = []
    for i, r in enumerate(ranges):
        if r is None:
            out.append(None)
            continue
        y = {n: (v[r[0]:r[1]] if n != "state" else v[i:i + 1]) for n, v in x.items()}
        offs = [0, r[1] - r[0]]
        c = Call(y, offs, delta, dtype)
        o, S = (t.clone() for t in c.forward())
        out.append((o, S, {n: t.clone() for n, t in c.backward(d_o[r[0]:r[1]], d_S[i:i + 1]).items()}))
    return out


SPIKES = [([0, 999, 170, 240], [None, None, (170, 240)]),
          ([0, 80, 10 ** 6, 170, 240], [(0, 80), None, None, (170, 240)]),
          ([0, -7, 100, 240], [None, None, (100, 240)]),
          ([64, 10, 10, 200, 2 ** 31 - 1], [None, (10, 10), (10, 200), None]),
          # sequences that start before the end of one that fits are taken as empty too
          ([100, 240, 0, 100], [(100, 240), None, None]),
          ([0, 80, 75, 240], [(0, 80), None, None])]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("delta,heads_qk", [(1, 1), (0, 2)])
@pytest.mark.parametrize("bad,ranges", SPIKES, ids=[str(s[0]) for s in SPIKES])
def test_sequences_beside_offsets_that_do_not_fit(bad, ranges, delta, heads_qk, dtype):
    """Each sequence that fits comes out as if alone, and the others' rows and states stay."""
    N = len(ranges)
    x, _ = inputs([240 // N] * N, 2, heads_qk, 32, 16, dtype, seed=261, trail=240 - 240 // N * N)
    d_o, d_S = normal(x["v"], 7, 1.0, dtype), normal(x["state"], 8)
    c = Call(x, None, delta, dtype, device_offsets=bad)
    c.offs = bad
    o, S = c.forward()
    assert c.check() == c.L.LORES_ERR_INVALID_ARG
    got = c.backward(d_o, d_S)
    assert c.check() == c.L.LORES_ERR_INVALID_ARG
    used = torch.zeros(240, dtype=torch.bool)
    for i, (r, want) in enumerate(zip(ranges, one_by_one(x, ranges, delta, d_o, d_S, dtype))):
        if r is None:
            assert torch.equal(S[i], c.state[i]) and torch.equal(got["state"][i], d_S[i].float())
            continue
        used[r[0]:r[1]] = True
        assert torch.equal(o[r[0]:r[1]], want[0]) and torch.equal(S[i], want[1][0])
        for n in NAMES:
            mine = got[n][i:i + 1] if n == "state" else got[n][r[0]:r[1]]
            assert torch.equal(mine, want[2][n]), n
    free = (~used).cuda()
    assert (o[free] == 777).all()
    for n in NAMES[:5]:
        assert (got[n][free] == 777).all(), n


def test_many_sequences_and_one_bad_offset():
    N, each = 700, 3
    x, offs = inputs([each] * N, 1, 1, 16, 4, F32, seed=262)
    whole = Call(x, offs, 1, F32)                            # (max_len 0: the chunk kernels)
    o, S = (t.clone() for t in whole.forward())
    bad = list(offs)
    bad[300] = 10 ** 9
    c = Call(x, offs, 1, F32, device_offsets=bad)
    c.work = whole.work
    o2, S2 = c.forward()
    assert c.check() == c.L.LORES_ERR_INVALID_ARG
    keep = [i for i in range(N) if i not in (299, 300)]
    assert torch.equal(S2[keep], S[keep]) and torch.equal(S2[299:301], c.state[299:301])
    rows = [t for i in keep for t in range(offs[i], offs[i + 1])]
    assert torch.equal(o2[rows], o[rows]) and (o2[offs[299]:offs[301]] == 777).all()


@pytest.mark.parametrize("N", [200, 700, 1500])
def test_many_sequences_out_of_order(N):
    """One offset that skips ahead to token 2 N (and so makes a long sequence), the next one back in line: what starts
    before that long sequence's end is taken as empty, what starts behind it is right."""
    each, at = 3, N // 3
    x, offs = inputs([each] * N, 1, 1, 16, 4, F32, seed=263)
    d_o, d_S = normal(x["v"], 7), normal(x["state"], 8)
    whole = Call(x, offs, 1, F32)
    o, S = (t.clone() for t in whole.forward())
    g = {n: t.clone() for n, t in whole.backward(d_o, d_S).items()}
    wrong = list(offs)
    wrong[at] = 2 * N
    c = Call(x, offs, 1, F32, device_offsets=wrong)
    c.work = whole.work
    o2, S2 = c.forward()
    assert c.check() == c.L.LORES_ERR_INVALID_ARG
    g2 = c.backward(d_o, d_S)
    good = [i for i in range(N) if i < at - 1 or (i > at and offs[i] >= 2 * N)]
    empty = [i for i in range(N) if i == at or (i > at and offs[i] < 2 * N)]
    assert torch.equal(S2[good], S[good]) and torch.equal(S2[empty], c.state[empty])
    assert torch.equal(g2["state"][good], g["state"][good]) and torch.equal(g2["state"][empty], d_S[empty].float())
    rows = [t for i in good for t in range(offs[i], offs[i + 1])]
    assert torch.equal(o2[rows], o[rows])
    for n in NAMES[:5]:
        assert torch.equal(g2[n][rows], g[n][rows]), n
    y = {n: (v[offs[at - 1]:2 * N] if n != "state" else v[at - 1:at]) for n, v in x.items()}
    long = Call(y, [0, 2 * N - offs[at - 1]], 1, F32)
    lo, lS = long.forward()
    assert torch.equal(o2[offs[at - 1]:2 * N], lo) and torch.equal(S2[at - 1:at], lS)


def test_several_heads_of_a_group_in_one_block_with_the_delta_rule():
    """Enough chunks that the preparation takes two heads (and more) that share q and k."""
    for H, Hq in ((32, 16), (32, 4)):
        x, offs = inputs([1300, 33, 1290], H, Hq, 16, 4, BF16, seed=271)
        c = Call(x, offs, 1, BF16)
        o, S = c.forward()
        ro, rS = forward64(x, offs, 1)
        assert rel(o, ro) <= tol(BF16) and rel(S, rS) <= FP32


def test_gradients_of_several_heads_of_a_group_with_the_delta_rule():
    x, offs = inputs([330, 1, 300], 128, 2, 16, 4, F32, seed=272)
    d_o, d_S = normal(x["v"], 7), normal(x["state"], 8)
    got = Call(x, offs, 1, F32).backward(d_o, d_S)
    check_gradients(got, backward64(x, offs, 1, d_o, d_S), F32)


GUARD = 4096                                                 # bytes before and behind each buffer


class Guarded(Call):
    """A call whose buffers lie between guard bands, the workspace of the exact size among them."""

    def __init__(self, *a, **kw):
        super().__init__(*a, **kw)
        self.bands = []
        for n in ("q", "k", "v", "la", "be", "state", "o", "state_out"):
            setattr(self, n, self.guard(getattr(self, n)))

    def guard(self, t):
        size = t.numel() * t.element_size()
        buf = torch.full((GUARD + (size + 15) // 16 * 16 + GUARD,), 0xA5, dtype=torch.uint8, device="cuda")
        inner = buf[GUARD:GUARD + size].view(t.dtype).view(t.shape)
        inner.copy_(t)
        self.bands.append((buf, size))
        return inner

    def workspace(self, backward):
        n = self.L.lores_scan_workspace(self.cfg, backward)
        self.work = self.guard(torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda"))
        return self.work

    def run_backward(self, d_o, d_S):
        self.backward(d_o, d_S)                              # (makes the gradients' buffers)
        names = ("d_o", "d_state_out", "dq", "dk_", "dv_", "dla", "dbe", "ds")
        a = [self.guard(getattr(self, n)) for n in names]
        self.L.lores_scan_backward(self.cfg, self.q, self.k, self.v, self.la, self.be, self.offsets, self.state,
                                   *a, self.workspace(True))

    def untouched(self):
        for buf, size in self.bands:
            assert (buf[:GUARD] == 0xA5).all() and (buf[GUARD + size:] == 0xA5).all()


@pytest.mark.parametrize("lens,H,Hq,dk,dv,delta,dtype,pad,max_len", [
    ([1], 1, 1, 16, 4, 1, F32, 0, 0), ([63, 1, 64, 0, 130], 3, 3, 64, 20, 1, F32, 0, 0),
    ([17, 200, 5], 4, 2, 128, 100, 1, BF16, 0, 0), ([33, 128, 129], 4, 1, 32, 36, 1, F16, 8, 0),
    ([70, 257], 4, 4, 128, 64, 0, BF16, 0, 0), ([320], 2, 2, 32, 260, 0, BF16, 8, 0),
    ([100, 31], 8, 1, 128, 12, 0, F32, 4, 0), ([5, 0, 9], 4, 2, 128, 36, 1, BF16, 4, 9), ([40], 2, 1, 256, 20, 1, F32, 0, 0)])
def test_nothing_is_written_outside_the_buffers(lens, H, Hq, dk, dv, delta, dtype, pad, max_len):
    x, offs = inputs(lens, H, Hq, dk, dv, dtype, seed=281)
    c = Guarded(x, offs, delta, dtype, pad, max_len=max_len)
    c.forward()
    if dk < 256:
        c.run_backward(normal(x["v"], 7, 1.0, dtype), normal(x["state"], 8))
    c.untouched()


def test_many_sequences_of_one_length_and_a_captured_call():
    x, offs = inputs([3] * 300, 2, 1, 32, 8, BF16, seed=291)
    a, b = Call(x, offs, 1, BF16), Call(x, offs, 1, BF16, with_offsets=False)
    d_o, d_S = normal(x["v"], 7, 1.0, BF16), normal(x["state"], 8)
    for p, q in zip(a.forward(), b.forward()):
        assert torch.equal(p, q)
    g, h = a.backward(d_o, d_S), b.backward(d_o, d_S)
    for n in NAMES:
        assert torch.equal(g[n], h[n]), n
    want = {n: t.clone() for n, t in g.items()}
    o, S = a.o.clone(), a.state_out.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        a.L.lores_scan_forward(a.cfg, a.q, a.k, a.v, a.la, a.be, a.offsets, a.state, a.o, a.state_out, a.work)
        a.L.lores_scan_backward(a.cfg, a.q, a.k, a.v, a.la, a.be, a.offsets, a.state, a.d_o, a.d_state_out, a.dq,
                                a.dk_, a.dv_, a.dla, a.dbe, a.ds, a.work)
    for t in (a.o, a.state_out, a.dq, a.dk_, a.dv_, a.dla, a.dbe, a.ds, a.work):
        t.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a.o, o) and torch.equal(a.state_out, S)
    for n in NAMES:
        assert torch.equal(g[n], want[n]), n
    assert a.check() == a.L.LORES_OK


@pytest.mark.parametrize("dtype,delta", [(F32, 0), (F32, 1), (BF16, 0), (BF16, 1)])
def test_decay_gradients_that_are_small_beside_their_terms(dtype, delta):
    """From zero states log_alpha of a sequence's first token has no gradient at all, and behind strong decays the others'
    are far smaller than d_beta and than <d_state_out, state_out>, whose terms they are differences of."""
    x, offs = inputs([1, 5, 40, 66], 4, 2, 64, 48, dtype, seed=301, decay=10.0)
    x["state"].zero_()
    d_o, d_S = normal(x["v"], 7, 1.0, dtype), normal(x["state"], 8, 1e3)
    got = Call(x, offs, delta, dtype).backward(d_o, d_S)["log_alpha"]
    want = backward64(x, offs, delta, d_o, d_S)["log_alpha"]
    for a, b in zip(offs, offs[1:]):
        # 64-bit sums of the terms of the state; what is left of d_o's is held to FP32 of d_o's terms
        size = float(want[a:b].norm()) + float(x["beta"][a:b].norm())
        assert float((got[a:b].double() - want[a:b]).norm()) <= 4 * FP32 * size, (a, b)
    assert float(got[0].abs().max()) <= 1e-9


@pytest.mark.parametrize("delta", [0, 1])
def test_decay_gradient_of_one_token_is_the_first_states(delta):
    """One token of a sequence: d_log_alpha is a_t <dL/dS', S_0>, however large v, k and d_state_out are beside S_0."""
    x, offs = inputs([1, 1], 2, 1, 64, 40, F32, seed=302)
    x["v"] = (x["v"] * 1e6).float().double()
    if not delta:
        x["k"] = (x["k"] * 1e6).float().double()
    x["state"] = (x["state"] * 1e-5).float().double()
    d_o, d_S = normal(x["v"], 7), normal(x["state"], 8, 1e3)
    got = Call(x, offs, delta, F32).backward(d_o, d_S)["log_alpha"]
    want = backward64(x, offs, delta, d_o, d_S)["log_alpha"]
    # (sums of d_v d_k products of either sign: FP32 of a_t |dL/dS'| |S_0|)
    size = (x["log_alpha"].exp() * (d_S.norm(dim=(2, 3)) + d_o.norm(dim=2) * x["q"].norm(dim=2))
            * x["state"].norm(dim=(2, 3)))
    assert ((got.double() - want).abs() <= 4 * FP32 * size).all()


@pytest.mark.parametrize("lens,H,Hq,dk,dv,delta", [([300, 77], 4, 2, 128, 128, 1), ([300, 77], 4, 2, 128, 64, 0),
                                                   ([130, 64], 2, 2, 64, 100, 1), ([200], 2, 1, 16, 36, 0)])
def test_fp32_results_keep_their_bits(lens, H, Hq, dk, dv, delta):
    """FP32 lets every rounding go the same way.  They go either way: an operand of 22 bits is off by 2^-23 / sqrt(3) (root
    mean square), a product's two and the term it drops (2^-22 / 3) by less than 1.4 * 2^-23 together, a dozen one
    behind the other by sqrt(12) times that, 5.8e-7; sums that the tensor cores cut off add at most 2^-23 for each of
    some four in a row.  Twice all that."""
    t = 2 * (12 ** 0.5 * 1.4 + 4) * 2.0 ** -23
    x, offs = inputs(lens, H, Hq, dk, dv, F32, seed=311)
    c = Call(x, offs, delta, F32)
    o, S = c.forward()
    ro, rS = forward64(x, offs, delta)
    assert rel(o, ro) <= t and rel(S, rS) <= t
    d_o, d_S = normal(x["v"], 7), normal(x["state"], 8)
    got, want = c.backward(d_o, d_S), backward64(x, offs, delta, d_o, d_S)
    for n in NAMES:
        assert rel(got[n], want[n]) <= t * (4 if n in ("log_alpha", "beta") else 1), n
