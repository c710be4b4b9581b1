"""The cache operators without a GPU: refusals come before any CUDA call, the workspace is a host
function, and the 64-bit definitions that the GPU tests compare with hold themselves."""

import ctypes

import numpy as np
import pytest
import torch

import kv_util as ku

F32, F16, BF16 = 0, 1, 2
OK, INVALID, UNSUPPORTED = 0, 1, 2
A = ctypes.c_void_p(0x10000)      # never dereferenced
ODD = ctypes.c_void_p(0x10001)


def _append(so, **kw):
    a = dict(dtype=F16, B=2, S=3, Nq=8, Nkv=2, H=64, q=A, k=None, v=None, qw=None, kw=None, eps=1e-6, cos=A, sin=A,
             rows=32, pos=None, past=A, inter=0, rd=0, qo=ctypes.c_void_p(0x90000), kc=A, vc=A, ks=A, vs=A, L=32,
             st=None, stream=None)
    a.update(kw)
    return so.rope_apply_qkv_fp8(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), UNSUPPORTED), (dict(Nq=0), INVALID), (dict(Nkv=3), INVALID), (dict(Nkv=0), INVALID),
    (dict(H=63), INVALID), (dict(H=0), INVALID), (dict(B=-1), INVALID), (dict(S=-1), INVALID), (dict(inter=2), INVALID),
    (dict(rd=63), INVALID), (dict(rd=66), INVALID), (dict(rd=-2), INVALID), (dict(rows=-1), INVALID),
    (dict(L=0), INVALID), (dict(L=2 ** 31), UNSUPPORTED), (dict(q=None), INVALID), (dict(q=ODD), INVALID),
    (dict(qo=None), INVALID), (dict(qo=A), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID),
    (dict(ks=None), INVALID), (dict(vs=ODD), INVALID), (dict(past=None), INVALID), (dict(cos=None), INVALID),
    (dict(k=A), INVALID), (dict(v=A), INVALID), (dict(k=A, v=ODD), INVALID), (dict(pos=ODD), INVALID),
    (dict(qw=A), INVALID), (dict(kw=A), INVALID), (dict(qw=A, kw=A, eps=-1.0), INVALID),
    (dict(qw=A, kw=A, eps=float("nan")), INVALID), (dict(qw=A, kw=A, H=66), UNSUPPORTED), (dict(st=ODD), INVALID),
    (dict(B=2 ** 40, S=2 ** 30), INVALID),
])
def test_append_refuses_before_launch(lib, kw, status):
    so = lib.load_library()
    assert _append(so, **kw) == status
    assert so.rope_last_error()


def _attend(so, fp8=False, **kw):
    a = dict(dtype=F16, B=2, S=3, Nq=8, Nkv=2, H=64, q=A, kc=A, vc=A, ks=A, vs=A, L=32, past=A, scale=0.1, cap=0.0,
             slopes=None, docs=None, prefix=None, out=A, st=None, ws=None, wsb=0, stream=None)
    a.update(kw)
    if not fp8:
        del a["ks"], a["vs"]
    return (so.kv_attention_fp8 if fp8 else so.kv_attention)(*a.values())


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=7), UNSUPPORTED), (dict(Nq=0), INVALID), (dict(Nkv=3), INVALID), (dict(H=0), INVALID),
    (dict(H=257), UNSUPPORTED), (dict(B=-1), INVALID), (dict(S=-2), INVALID), (dict(L=0), INVALID),
    (dict(L=2 ** 31), UNSUPPORTED), (dict(S=2 ** 31), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(cap=-1.0), INVALID), (dict(cap=float("inf")), INVALID),
    (dict(cap=float("nan")), INVALID), (dict(q=None), INVALID), (dict(q=ODD), INVALID), (dict(kc=None), INVALID),
    (dict(vc=None), INVALID), (dict(past=None), INVALID), (dict(past=ODD), INVALID), (dict(out=None), INVALID),
    (dict(slopes=ODD), INVALID), (dict(docs=ODD), INVALID), (dict(prefix=ODD), INVALID), (dict(st=ODD), INVALID),
    (dict(ws=ODD, wsb=64), INVALID), (dict(wsb=-1), INVALID), (dict(B=2 ** 30, S=2 ** 30, Nq=2 ** 20), INVALID),
])
def test_attention_refuses_before_launch(lib, fp8, kw, status):
    so = lib.load_library()
    assert _attend(so, fp8, **kw) == status
    assert so.rope_last_error()


def test_scales_are_checked(lib):
    so = lib.load_library()
    assert _attend(so, True, ks=None) == INVALID
    assert _attend(so, True, vs=ODD) == INVALID


@pytest.mark.parametrize("fp8", [False, True])
def test_out_is_no_input(lib, fp8):
    so = lib.load_library()
    for name in ("q", "kc", "vc"):
        at = {n: ctypes.c_void_p(0x20000 + 0x10000 * i) for i, n in enumerate(("q", "kc", "vc"))}
        at.update({name: A, "out": A})
        assert _attend(so, fp8, **at) == INVALID
        assert b"alias" in so.rope_last_error()


def test_empty_calls_launch_nothing(lib):
    so = lib.load_library()
    for kw in (dict(B=0), dict(S=0)):
        assert _append(so, **kw, q=None, qo=None) == OK
        assert _attend(so, **kw, q=None, out=None) == OK
        assert _attend(so, True, **kw, q=None, out=None) == OK


def test_workspace_is_a_host_function(lib):
    assert lib.kv_attention_workspace(0, 1, 8, 2, 64, 128) == 0
    few = lib.kv_attention_workspace(1, 1, 8, 2, 64, 65536)
    assert few > 0
    with pytest.raises(lib.RopeError):
        lib.kv_attention_workspace(1, 1, 8, 3, 64, 128)
    with pytest.raises(lib.RopeError):
        lib.kv_attention_workspace(1, 1, 8, 2, 257, 128)


def test_binding_refuses_cpu_tensors(lib):
    q = torch.zeros((1, 1, 64), dtype=torch.float16)
    c = torch.zeros((1, 1, 4, 64), dtype=torch.float16)
    with pytest.raises(ValueError):
        lib.kv_attention(q, c, c, torch.zeros(1, dtype=torch.int32), num_heads=1)
    with pytest.raises(ValueError):
        lib.rope_apply_qkv_fp8(torch.zeros((1, 1, 3 * 64), dtype=torch.float16), c[0, 0, :, :32], c[0, 0, :, :32],
                               num_heads=1, kv_num_heads=1, k_cache=c, v_cache=c, k_scale=c, v_scale=c,
                               past_seq_lens=c)


# --------------------------------------------------------------------------
# the definitions
# --------------------------------------------------------------------------

def test_e4m3_against_torch():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(20000) * 10.0 ** rng.uniform(-3, 2.2, 20000), np.linspace(-448, 448, 7169),
                        [0.0, -0.0]]).astype(np.float32)
    x = x[np.abs(x) <= 448]
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ku.e4m3(x), want)
    assert np.array_equal(ku._VALUES[:127], torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy())
    assert ku.e4m3(np.array([np.inf, -np.inf, 1e9, np.nan])).tolist() == [126, 254, 126, 127]


def test_scale_is_the_smallest_power_of_two():
    for a in (448.0, 448.0001, 447.9, 1.75, 1.7500001, 1e-30, 3.4e38, 0.0, 2.0 ** -140):
        s = ku.scale_of(a)
        assert a <= 448 * s and np.log2(s) == int(np.log2(s))
        assert s == 2.0 ** -120 or 448 * s / 2 < a


def test_attention_definition_by_hand():
    """Two keys with scores 0 and ln 3: weights 1/4 and 3/4."""
    q = torch.tensor([[[1.0]]], dtype=torch.float64)
    k = torch.tensor([[[[0.0], [np.log(3.0)], [9.0]]]], dtype=torch.float64)
    v = torch.tensor([[[[4.0], [8.0], [100.0]]]], dtype=torch.float64)
    out, _ = ku.attention(q, k, v, [1], 1, 1.0)
    assert abs(float(out) - 7.0) < 1e-12
    # a bias of ln 3 by distance evens them out; another document leaves the second alone
    out, _ = ku.attention(q, k, v, [1], 1, 1.0, slopes=torch.tensor([-np.log(3.0)]))
    assert abs(float(out) - 6.0) < 1e-12
    out, _ = ku.attention(q, k, v, [1], 1, 1.0, docs=np.array([[5, 6, 6]]))
    assert float(out) == 8.0
    out, _ = ku.attention(q, k, v, [0], 1, 1.0, prefix=[3])
    assert float(out) == 4.0  # the prefix ends with the rows that exist


def test_append_keeps_older_rows():
    """One row at a time: the older codes follow a growing scale. A value is off by half a code's step, 2^-4
    of it, once, and by half a subnormal step, 2^-10 of the scale, at each growth: 2 * 2^-10 of the last
    scale in all, since the scales at least double; twice that where both fall together."""
    rng = np.random.default_rng(1)
    codes, scale = np.zeros((1, 1, 40, 8), np.uint8), np.ones((1, 1, 3), np.float32)
    rows = rng.standard_normal((40, 8)) * 2.0 ** np.arange(40)[:, None] / 2.0 ** 20
    for t in range(40):
        ku.append(codes, scale, rows[None, t:t + 1, None], [t])
    got = ku.values(codes, scale)[0, 0]
    s = np.repeat(scale[0, 0], 16)[:40, None]
    assert (np.abs(got - rows) <= 2.0 ** -4 * np.abs(rows) + 2 * 2.0 ** -10 * s * 2).all()
