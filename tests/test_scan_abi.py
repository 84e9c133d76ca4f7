"""Refusals and sizes of the state scan and of the pool's write and read, on the CPU: every check
returns before a pointer is used or CUDA is touched, so plain aligned addresses do."""
import ctypes as C

import pytest

A = 0x10000                                        # an aligned address


def lib():
    from bit_recurrent_state_lores_b200 import lores as L
    return L


def config(**kw):
    args = dict(n_seq=2, total=128, heads=4, d_k=64, d_v=32)
    args.update(kw)
    return lib().make_scan_config(**args)


BAD = [dict(n_seq=0), dict(total=-1), dict(total=2**31), dict(max_len=-1), dict(heads=0),
       dict(heads=65536), dict(heads_qk=3), dict(heads_qk=-1), dict(heads_qk=8), dict(d_k=48),
       dict(d_k=0), dict(d_k=512), dict(d_v=0), dict(d_v=6), dict(d_v=4100), dict(delta=2),
       dict(delta=-1), dict(dtype=3), dict(dtype=-1), dict(device=-1), dict(q_stride=128),
       dict(k_stride=258), dict(v_stride=-4), dict(o_stride=130), dict(n_seq=2**20, heads=4096)]


@pytest.mark.parametrize("kw", BAD, ids=[str(b) for b in BAD])
def test_bad_configurations_are_refused(kw):
    L = lib()
    cfg = config(**kw)
    n = C.c_uint64(7)
    raw = L.raw_library()
    assert raw.lores_scan_workspace(C.byref(cfg), 0, C.byref(n)) == L.LORES_ERR_INVALID_ARG
    assert n.value == 7
    assert raw.lores_scan_forward(C.byref(cfg), A, A, A, A, A, A, A, A, A, A, 1 << 40,
                                  None) == L.LORES_ERR_INVALID_ARG
    assert raw.lores_scan_backward(C.byref(cfg), A, A, A, A, A, A, A, A, A, A, A, A, A, A, A, A,
                                   1 << 40, None) == L.LORES_ERR_INVALID_ARG


def test_workspace_sizes():
    L = lib()
    cfg = config()
    fwd, bwd = L.lores_scan_workspace(cfg), L.lores_scan_workspace(cfg, backward=True)
    assert 256 <= fwd < bwd
    # short sequences need no per-chunk matrices
    assert L.lores_scan_workspace(config(max_len=16)) == 256
    assert L.lores_scan_workspace(config(d_k=256)) == 256
    assert L.lores_scan_workspace(config(max_len=32)) == 256
    assert L.lores_scan_workspace(config(max_len=33)) == fwd
    assert L.lores_scan_workspace(config(max_len=24, delta=0)) == 256
    assert L.lores_scan_workspace(config(max_len=25, delta=0)) > 256
    # no tokens: still a workspace (the error word)
    assert L.lores_scan_workspace(config(total=0)) >= 256
    # shared q and k take less of it, sums over heads that share them more of the backward pass's
    assert L.lores_scan_workspace(config(heads_qk=1)) < fwd
    assert L.lores_scan_workspace(config(delta=0)) < fwd
    raw = L.raw_library()
    n = C.c_uint64()
    assert raw.lores_scan_workspace(None, 0, C.byref(n)) == L.LORES_ERR_INVALID_ARG
    assert raw.lores_scan_workspace(C.byref(cfg), 2, C.byref(n)) == L.LORES_ERR_INVALID_ARG
    assert raw.lores_scan_workspace(C.byref(cfg), 0, None) == L.LORES_ERR_INVALID_ARG


def test_backward_refuses_the_widest_keys():
    L = lib()
    with pytest.raises(L.LoresError) as e:
        L.lores_scan_workspace(config(d_k=256), backward=True)
    assert e.value.status == L.LORES_ERR_UNSUPPORTED


# argument positions of the pointers that must be given
FORWARD = ["q", "k", "v", "log_alpha", "beta", "offsets", "state_in", "o", "state_out", "workspace"]
BACKWARD = ["q", "k", "v", "log_alpha", "beta", "offsets", "state_in", "d_o", "d_state_out", "dq",
            "dk", "dv", "dlog_alpha", "dbeta", "d_state_in", "workspace"]
OPTIONAL = {"offsets", "state_in", "state_out", "d_state_out", "d_state_in"}
FOUR = {"log_alpha", "beta", "offsets", "dlog_alpha", "dbeta"}          # 4-byte alignment


def call(name, names, cfg, nbytes=1 << 40, **over):
    args = [over.get(n, A) for n in names]
    return getattr(lib().raw_library(), name)(C.byref(cfg), *args, nbytes, None)


@pytest.mark.parametrize("name,names", [("lores_scan_forward", FORWARD),
                                        ("lores_scan_backward", BACKWARD)])
def test_pointers_are_checked(name, names):
    L = lib()
    cfg = config()
    for n in names:
        if n not in OPTIONAL:
            assert call(name, names, cfg, **{n: None}) == L.LORES_ERR_INVALID_ARG, n
        wrong = A + 2 if n in FOUR else A + 8
        assert call(name, names, cfg, **{n: wrong}) == L.LORES_ERR_INVALID_ARG, n
    need = L.lores_scan_workspace(cfg, backward="backward" in name)
    assert call(name, names, cfg, nbytes=need - 1) == L.LORES_ERR_INVALID_ARG
    # without offsets the sequences have one length
    assert call(name, names, config(n_seq=3), offsets=None) == L.LORES_ERR_INVALID_ARG
    raw = lib().raw_library()
    assert getattr(raw, name)(None, *[A] * len(names), 1 << 40, None) == L.LORES_ERR_INVALID_ARG


def test_check_errors_arguments():
    L = lib()
    raw = L.raw_library()
    cfg = config()
    assert raw.lores_scan_check_errors(None, A, None) == L.LORES_ERR_INVALID_ARG
    assert raw.lores_scan_check_errors(C.byref(cfg), None, None) == L.LORES_ERR_INVALID_ARG


def test_pool_calls_refuse_a_null_handle():
    L = lib()
    raw = L.raw_library()
    assert raw.lores_write_states(None, 1, A, A, 0, 0, None) == L.LORES_ERR_INVALID_ARG
    assert raw.lores_read_states(None, 1, A, A, 0, None) == L.LORES_ERR_INVALID_ARG


def test_dtype_names():
    import torch
    L = lib()
    assert config(dtype=torch.bfloat16).dtype == L.LORES_BF16
    assert config(dtype=torch.float16).dtype == L.LORES_F16
    assert config(dtype=torch.float32).dtype == L.LORES_F32
    with pytest.raises(TypeError):
        config(dtype=torch.float64)
