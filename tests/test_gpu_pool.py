"""Writing and reading chosen slots of a handle's state pool, and a prompt's way through it: read slots ->
scan -> write slots -> decode steps."""
import numpy as np
import pytest
import torch

from bit_recurrent_state_lores_b200 import synth

from .harness import GpuRun
from .scan_reference import inputs, rel, scan64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def lib():
    from bit_recurrent_state_lores_b200 import lores
    return lores


def states(n, H, dv, dk, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return r(n, H, dv, dk) * torch.exp(r(n, H, dv, 1))


def slots_of(*s):
    return torch.tensor(s, dtype=torch.int32, device="cuda")


FORMATS = [
    ("int8", 128, 128, 128, [8, 8], {}),
    ("mixed", 128, 20, 32, [8, 4, 32, 6], {}),
    ("narrow", 16, 12, 16, [4, 8], {}),
    ("rtn", 32, 36, 16, [8, 5], {"stochastic": 0}),
    ("wide", 256, 64, 256, [4, 8], {}),
    ("dense", 64, 24, 32, [5, 6, 7], {"dense": 1}),
    ("channels", 64, 24, 16, [8, 8], {"group_bits": [[8, 4, 5, 6], [4, 4, 8, 7]]}),
]


@pytest.mark.parametrize("name,dk,dv,G,bits,kw", FORMATS, ids=[f[0] for f in FORMATS])
def test_slots_equal_the_whole_state_calls(name, dk, dv, G, bits, kw):
    L = lib()
    B, H = 5, len(bits)
    wl = synth.Workload(name, B=B, H=H, d_k=dk, d_v=dv, steps=1, group=G)
    S = states(B, H, dv, dk)
    a, b = GpuRun(wl, bits, seed=9, **kw), GpuRun(wl, bits, seed=9, **kw)
    try:
        L.lores_load_state(a.h, S, 17)
        # all slots at once, in another order
        order = slots_of(3, 0, 4, 1, 2)
        L.lores_write_states(b.h, B, order, S[order.long()].contiguous(), 17)
        for x, y in zip(a.export(), b.export()):
            assert np.array_equal(x, y)
        # one slot replaced: the others stay
        new = states(1, H, dv, dk, seed=3)
        S2 = S.clone()
        S2[2] = new[0]
        L.lores_load_state(a.h, S2, 23)
        full = a.dequant()
        L.lores_write_states(b.h, 1, slots_of(2), new, 23)
        out = b.dequant()
        assert torch.equal(out[2], full[2])
        L.lores_load_state(a.h, S, 17)
        old = a.dequant()
        for i in (0, 1, 3, 4):
            assert torch.equal(out[i], old[i])
        # read back some, in any type; NULL slots are 0 ..
        pick = slots_of(4, 2)
        for dt in (torch.float32, torch.bfloat16, torch.float16):
            got = torch.full((2, H, dv, dk), 7.0, device="cuda", dtype=dt)
            L.lores_read_states(b.h, 2, pick, got)
            assert torch.equal(got, out[[4, 2]].to(dt))
            got = torch.full((3, H, dv, dk), 7.0, device="cuda", dtype=dt)
            L.lores_read_states(b.h, 3, None, got)
            assert torch.equal(got, out[:3].to(dt))
        assert b.check() == L.LORES_OK
    finally:
        a.close()
        b.close()


def test_skipped_repeated_and_no_entries():
    L = lib()
    wl = synth.Workload("p", B=4, H=2, d_k=64, d_v=40, steps=1)
    g = GpuRun(wl, [8, 4], seed=1)
    try:
        S = states(4, 2, 40, 64)
        L.lores_load_state(g.h, S, 1)
        old = g.dequant()
        new = states(4, 2, 40, 64, seed=2)
        # -1, 4 and a large slot are skipped; slot 3 comes twice and its later entry counts
        L.lores_write_states(g.h, 4, slots_of(3, -1, 2**31 - 1, 3), new, 5)
        out = g.dequant()
        ref = GpuRun(wl, [8, 4], seed=1)
        L.lores_write_states(ref.h, 1, slots_of(3), new[3:].contiguous(), 5)
        assert torch.equal(out[3], ref.dequant()[3]) and torch.equal(out[:3], old[:3])
        ref.close()
        got = torch.full((4, 2, 40, 64), 7.0, device="cuda")
        L.lores_read_states(g.h, 4, slots_of(4, 0, -1, 0), got)
        assert (got[0] == 7).all() and (got[2] == 7).all()
        assert torch.equal(got[1], out[0]) and torch.equal(got[3], out[0])
        L.lores_write_states(g.h, 0, None, None, 0, dtype=L.LORES_F32)
        L.lores_read_states(g.h, 0, None, None, dtype=L.LORES_F32)
        assert torch.equal(g.dequant(), out)
        # 16-byte but not 32-byte aligned buffers
        buf = torch.zeros(4 + 4 * 2 * 40 * 64, device="cuda")
        view = buf[4:].view(4, 2, 40, 64)
        view.copy_(new)
        L.lores_write_states(g.h, 4, None, view, 5)
        a = g.dequant()
        L.lores_write_states(g.h, 4, None, new, 5)
        assert torch.equal(a, g.dequant())
        L.lores_read_states(g.h, 4, None, view)
        assert torch.equal(view, a) and (buf[:4] == 0).all()
        # 16-bit states quantize like their fp32 values
        L.lores_write_states(g.h, 4, None, new.bfloat16(), 5)
        a = g.dequant()
        L.lores_write_states(g.h, 4, None, new.bfloat16().float(), 5)
        assert torch.equal(a, g.dequant())
        assert g.check() == L.LORES_OK
        # a row that is not finite is stored as zero and reported
        new[1, 1, 7, 3] = float("nan")
        L.lores_write_states(g.h, 4, None, new, 5)
        a = g.dequant()
        assert (a[1, 1, 7] == 0).all() and torch.isfinite(a).all() and (a[1, 1, 6] != 0).any()
        assert g.check() == L.LORES_ERR_NONFINITE and g.check() == L.LORES_OK
    finally:
        g.close()


def test_refusals():
    L = lib()
    raw = L.raw_library()
    wl = synth.Workload("p", B=2, H=2, d_k=32, d_v=24, steps=1)
    g, key = GpuRun(wl, [8, 8], seed=1), GpuRun(wl, [8, 8], seed=1, axis=1)
    S = states(2, 2, 24, 32)
    p = S.data_ptr()
    bad = L.LORES_ERR_INVALID_ARG
    try:
        for n, slots, buf, dt in ((-1, None, p, 0), (3, None, p, 0), (1, None, None, 0), (1, None, p + 8, 0),
                                  (1, p + 2, p, 0), (1, None, p, 3), (1, None, p, -1)):
            assert raw.lores_write_states(g.h, n, slots, buf, dt, 0, None) == bad
            assert raw.lores_read_states(g.h, n, slots, buf, dt, None) == bad
        # a column's scale belongs to the whole tile: slots of a key-axis handle are read only
        assert raw.lores_write_states(key.h, 1, None, p, 0, 0, None) == L.LORES_ERR_UNSUPPORTED
        L.lores_load_state(key.h, S, 3)
        out = torch.empty_like(S[:1])
        L.lores_read_states(key.h, 1, slots_of(1), out)
        assert torch.equal(out[0], key.dequant()[1])
    finally:
        g.close()
        key.close()


def test_prompt_through_the_pool():
    """Two of five slots take a prompt: their states are read, carried over it and written back, then all slots
    decode.  The written codes are those of the recurrence's last states (a state off by 1e-5 of an entry moves
    a code, 1/40 of an entry, with probability 4e-4)."""
    L = lib()
    B, H, dk, dv = 5, 4, 128, 64
    bits = [8, 4, 8, 8]
    wl = synth.Workload("prompt", B=B, H=H, d_k=dk, d_v=dv, steps=4, decay="tau", seed=3)
    hp = synth.head_params(wl)
    a, b = GpuRun(wl, bits, seed=5), GpuRun(wl, bits, seed=5)
    try:
        S0 = states(B, H, dv, dk, seed=7)
        for g in (a, b):
            L.lores_load_state(g.h, S0, 1)
        pick = slots_of(3, 1)
        x, offs = inputs([150, 90], H, H, dk, dv, torch.bfloat16, seed=8)
        S = torch.empty(2, H, dv, dk, device="cuda")
        L.lores_read_states(a.h, 2, pick, S)
        x["state"] = S.double()
        cfg = L.make_scan_config(2, 240, H, dk, dv, dtype=torch.bfloat16, max_len=150)
        work = torch.empty(L.lores_scan_workspace(cfg), dtype=torch.uint8, device="cuda")
        o = torch.empty(240, H, dv, device="cuda", dtype=torch.bfloat16)
        bf = lambda n: x[n].bfloat16().contiguous()  # noqa: E731
        L.lores_scan_forward(cfg, bf("q"), bf("k"), bf("v"), x["log_alpha"].float(), x["beta"].float(),
                             torch.tensor(offs, dtype=torch.int32, device="cuda"), S, o, S, work)
        L.lores_write_states(a.h, 2, pick, S, 2)
        ro, rS = scan64(*(x[n] for n in ("q", "k", "v", "log_alpha", "beta")), offs, x["state"], 1)
        assert rel(o, ro) <= 2.0 ** -8 + 2 * 2.0 ** -11
        L.lores_write_states(b.h, 2, pick, rS.float(), 2)
        ca, cb = a.export(), b.export()
        diff = np.abs(ca[0].astype(np.int16) - cb[0].astype(np.int16)) != 0
        assert diff.mean() <= 4e-4 and np.allclose(ca[1], cb[1], rtol=1e-4, atol=0)
        da, db = a.dequant(), b.dequant()
        for i in (0, 2, 4):
            assert torch.equal(da[i], db[i])
        for t in range(3, 6):
            inp = synth.step_inputs(wl, t, hp, device="cuda")
            oa, ob = a.step(inp, t).clone(), b.step(inp, t)
            for i in (0, 2, 4):
                assert torch.equal(oa[i], ob[i])
            # slots 1 and 3 start from states that differ in few codes, by one step of 1/7 or 1/127 of the row's
            # largest entry: sqrt(4e-4) * (1/7) * 2 (largest over rms) of the state
            assert rel(oa[[1, 3]], ob[[1, 3]]) <= 6e-3
        assert a.check() == L.LORES_OK and b.check() == L.LORES_OK
    finally:
        a.close()
        b.close()


def test_slots_beyond_32_bits():
    """A pool of more than 4 GB: the last slot's state goes in and out, the others stay zero."""
    L = lib()
    B, H, d = 2100, 32, 128
    h = L.lores_create(B, H, d, d, head_bits=[32] * H)
    try:
        S = states(2, H, d, d, seed=7)
        L.lores_write_states(h, 2, slots_of(B - 1, 1040), S, 0)
        back = torch.full((3, H, d, d), 777.0, device="cuda")
        L.lores_read_states(h, 3, slots_of(1040, 0, B - 1), back)
        assert torch.equal(back[0], S[1]) and torch.equal(back[2], S[0])
        assert (back[1] == 0).all()
        assert L.lores_check_errors(h) == L.LORES_OK
    finally:
        L.lores_destroy(h)


def test_fp32_heads_report_what_is_not_finite_alone():
    """An fp32 head copies a row whatever its size; only infinities and NaN are reported."""
    L = lib()
    wl = synth.Workload("p", B=2, H=2, d_k=32, d_v=24, steps=1)
    g = GpuRun(wl, [32, 8], seed=1)
    try:
        S = states(2, 2, 24, 32)
        S[1, 0, 3, 5] = 2.0 ** 110
        L.lores_write_states(g.h, 2, None, S, 5)
        assert torch.equal(g.dequant()[:, 0], S[:, 0]) and g.check() == L.LORES_OK
        S[1, 0, 3, 5] = float("inf")
        L.lores_write_states(g.h, 2, None, S, 5)
        assert torch.equal(g.dequant()[:, 0], S[:, 0]) and g.check() == L.LORES_ERR_NONFINITE
        S[1, 0, 3, 5] = 1.0
        S[0, 1, 2, 2] = 2.0 ** 110                          # a quantized head stores such a row as zero
        L.lores_write_states(g.h, 2, None, S, 5)
        assert (g.dequant()[0, 1, 2] == 0).all() and g.check() == L.LORES_ERR_NONFINITE
    finally:
        g.close()
