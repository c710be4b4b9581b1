"""The paged-cache operators without a GPU: refusals come before any CUDA call, the workspace is a host function,
and the 64-bit definitions that the GPU tests compare with hold themselves."""

import ctypes

import numpy as np
import pytest
import torch

import kv_util as ku
import paged_util as pu

F32, F16, BF16 = 0, 1, 2
OK, INVALID, UNSUPPORTED = 0, 1, 2
A = ctypes.c_void_p(0x10000)      # never dereferenced
B = ctypes.c_void_p(0x90000)
C = ctypes.c_void_p(0xd0000)
ODD = ctypes.c_void_p(0x10001)


def _append(so, **kw):
    a = dict(dtype=F16, B=2, tokens=6, Nq=8, Nkv=2, H=64, q=A, k=None, v=None, qw=None, kw=None, eps=1e-6, cos=A, sin=A,
             rows=32, pos=None, past=A, starts=None, table=A, width=4, inter=0, rd=0, qo=B, kp=A, vp=C, pages=9, ps=16,
             stride=2 * 16 * 64, st=None, stream=None)
    a.update(kw)
    return so.rope_apply_qkv_paged(*a.values())


def _attend(so, **kw):
    a = dict(dtype=F16, B=2, tokens=6, most=3, Nq=8, Nkv=2, H=64, q=A, kp=A, vp=A, pages=9, ps=16, stride=2 * 16 * 64,
             table=A, width=4, past=A, starts=None, scale=0.1, cap=0.0, window=0, slopes=None, masks=None, out=B, st=None,
             ws=None, wsb=0, stream=None)
    a.update(kw)
    return so.kv_attention_paged(*a.values())


def _keep(so, **kw):
    a = dict(dtype=F16, B=2, Nkv=2, H=64, kp=A, vp=C, pages=9, ps=16, stride=2 * 16 * 64, table=A, width=4, past=A, kept=A,
             most=5, lens=A, st=None, stream=None)
    a.update(kw)
    return so.kv_keep_paged(*a.values())


COMMON = [
    (dict(dtype=7), UNSUPPORTED), (dict(Nkv=0), INVALID), (dict(H=0), INVALID), (dict(B=-1), INVALID),
    (dict(B=2 ** 31), UNSUPPORTED), (dict(ps=0), INVALID), (dict(width=0), INVALID), (dict(ps=2 ** 31), UNSUPPORTED),
    (dict(width=2 ** 27, stride=2 ** 40), UNSUPPORTED), (dict(width=2 ** 40), UNSUPPORTED), (dict(pages=0), INVALID),
    (dict(pages=2 ** 31), UNSUPPORTED), (dict(stride=2 * 16 * 64 - 1), INVALID), (dict(stride=-1), INVALID),
    (dict(pages=2 ** 30, stride=2 ** 40), INVALID), (dict(kp=None), INVALID), (dict(vp=None), INVALID), (dict(kp=ODD), INVALID),
    (dict(table=None), INVALID), (dict(table=ODD), INVALID), (dict(past=None), INVALID), (dict(past=ODD), INVALID),
    (dict(st=ODD), INVALID),
]


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(Nq=0), INVALID), (dict(Nkv=3, stride=2 ** 20), INVALID), (dict(H=63), INVALID), (dict(tokens=-1), INVALID),
    (dict(tokens=2 ** 31), UNSUPPORTED), (dict(tokens=7), INVALID), (dict(inter=2), INVALID), (dict(rd=63), INVALID),
    (dict(rd=66), INVALID), (dict(rd=-2), INVALID), (dict(rows=-1), INVALID), (dict(q=None), INVALID), (dict(q=ODD), INVALID),
    (dict(qo=None), INVALID), (dict(qo=A), INVALID), (dict(starts=ODD), INVALID), (dict(cos=None), INVALID), (dict(k=A), INVALID),
    (dict(v=A), INVALID), (dict(k=A, v=ODD), INVALID), (dict(pos=ODD), INVALID), (dict(qw=A), INVALID), (dict(kw=A), INVALID),
    (dict(qw=A, kw=A, eps=-1.0), INVALID), (dict(qw=A, kw=A, eps=float("nan")), INVALID), (dict(qw=A, kw=ODD), INVALID),
])
def test_append_refuses_before_launch(lib, kw, status):
    so = lib.load_library()
    assert _append(so, **kw) == status
    assert so.rope_last_error()


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(Nq=0), INVALID), (dict(Nkv=3, stride=2 ** 20), INVALID), (dict(H=257, stride=2 ** 20), UNSUPPORTED),
    (dict(tokens=-1), INVALID), (dict(tokens=2 ** 31), UNSUPPORTED), (dict(tokens=7), INVALID), (dict(most=0), INVALID),
    (dict(most=-1), INVALID), (dict(most=7), INVALID), (dict(most=2), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(scale=2.0 ** 101), INVALID), (dict(cap=-1.0), INVALID),
    (dict(cap=float("inf")), INVALID), (dict(window=-1), INVALID), (dict(masks=A, window=3), INVALID),
    (dict(masks=A, slopes=A), INVALID), (dict(masks=A, tokens=130, most=65), INVALID), (dict(masks=ODD), INVALID),
    (dict(slopes=ODD), INVALID), (dict(starts=ODD), INVALID), (dict(q=None), INVALID), (dict(q=ODD), INVALID),
    (dict(out=None), INVALID), (dict(ws=ODD, wsb=64), INVALID), (dict(wsb=-1), INVALID),
    (dict(tokens=2 ** 30, B=2 ** 20, most=2 ** 10, Nq=2 ** 30), INVALID),
])
def test_attention_refuses_before_launch(lib, kw, status):
    so = lib.load_library()
    assert _attend(so, **kw) == status
    assert so.rope_last_error()


@pytest.mark.parametrize("kw,status", COMMON + [
    (dict(most=-1), INVALID), (dict(most=2 ** 21), UNSUPPORTED), (dict(kept=None), INVALID), (dict(kept=ODD), INVALID),
    (dict(lens=None), INVALID), (dict(lens=ODD), INVALID),
])
def test_keep_refuses_before_launch(lib, kw, status):
    so = lib.load_library()
    assert _keep(so, **kw) == status
    assert so.rope_last_error()


def test_out_is_no_input(lib):
    so = lib.load_library()
    for name in ("q", "kp", "vp"):
        at = {n: ctypes.c_void_p(0x20000 + 0x10000 * i) for i, n in enumerate(("q", "kp", "vp"))}
        at.update({name: B, "out": B})
        assert _attend(so, **at) == INVALID
        assert b"alias" in so.rope_last_error()


def test_pages_that_are_written_are_two(lib):
    so = lib.load_library()
    for call, kw in ((_append, dict(vp=A)), (_append, dict(qo=C)), (_append, dict(kp=B)), (_keep, dict(vp=A))):
        assert call(so, **kw) == INVALID


def test_empty_calls_launch_nothing(lib):
    so = lib.load_library()
    assert _append(so, tokens=0, q=None, qo=None) == OK
    assert _append(so, B=0, tokens=5, q=None) == OK
    assert _attend(so, tokens=0, most=0, q=None, out=None) == OK
    assert _attend(so, B=0, tokens=0, most=0, q=None) == OK
    assert _keep(so, B=0, kept=None) == OK
    assert _keep(so, most=0, kept=None) == OK


def test_workspace_is_a_host_function(lib):
    for t in (torch.float32, torch.float16, torch.bfloat16):
        assert lib.kv_attention_paged_workspace(t, 0, 0, 0, 8, 2, 64, 16, 8) == 0
        assert lib.kv_attention_paged_workspace(t, 1, 1, 1, 8, 2, 64, 16, 4096) > 0
        for bad in ((1, 1, 1, 8, 3, 64, 16, 8), (1, 1, 1, 8, 2, 257, 16, 8), (1, 1, 2, 8, 2, 64, 16, 8),
                    (1, 1, 1, 8, 2, 64, 0, 8)):
            with pytest.raises(lib.RopeError):
                lib.kv_attention_paged_workspace(t, *bad)
    with pytest.raises(lib.RopeError):
        lib.kv_attention_paged_workspace(torch.float64, 1, 1, 1, 8, 2, 64, 16, 8)


def test_binding_refuses(lib):
    q = torch.zeros((3, 64), dtype=torch.float16)
    k = torch.zeros((4, 1, 16, 64), dtype=torch.float16)
    i = torch.zeros((3, 1), dtype=torch.int32)
    with pytest.raises(ValueError):
        lib.kv_attention_paged(q, k, k, i, i[:, 0], num_heads=1, query_starts=i[:, 0])
    with pytest.raises(ValueError):
        lib.kv_keep_paged(k, k, i, i[:, 0], i, i[:, 0])
    with pytest.raises(ValueError):
        lib.rope_apply_qkv_paged(torch.zeros((3, 192), dtype=torch.float16), q, q, num_heads=1, kv_num_heads=1, k_pages=k,
                                 v_pages=k, page_table=i, past_seq_lens=i[:, 0], query_starts=i[:, 0])


def test_short_way_leaves_the_rest_to_the_binding(lib):
    """The compiled short way declines what is not all as it should be, without an error of its own."""
    short = lib._short_way()
    if not short:
        pytest.skip("binding.cpp is not compiled here")
    q = torch.zeros((3, 64), dtype=torch.float16)
    k = torch.zeros((4, 1, 16, 64), dtype=torch.float16)
    i = torch.zeros((3, 1), dtype=torch.int32)
    p, s = i[:, 0].contiguous(), torch.zeros(4, dtype=torch.int32)
    for fn, args in ((short.attention, (0, 0, q, k, k, i, p, 1, s, 1, None, 0.0, 0, None, None, None, None, None)),
                     (short.keep, (0, 0, k, k, i, p, i, p, None)),
                     (short.append, (0, 0, q, q, q, None, 1, 1, k, k, i, p, s, q, q, 0, 0, None, None, None, None, 1e-6))):
        assert fn(*args) is None                    # CPU tensors
        for n in range(len(args)):
            for bad in ("x", None, 1.5, 2 ** 70):
                assert fn(*args[:n], bad, *args[n + 1:]) is None
        assert fn(*args[:-1]) is None and fn() is None


# --------------------------------------------------------------------------
# the definitions
# --------------------------------------------------------------------------

def test_visible_by_hand():
    assert pu.visible(3, 2, 5, 0).tolist() == [True] * 4 + [False]
    assert pu.visible(3, 2, 5, 1, window=2).tolist() == [False] * 3 + [True] * 2
    assert pu.visible(-2, 3, 1, 0).tolist() == [False]
    assert pu.visible(2, 3, 5, 0, word=0b101).tolist() == [True, True, True, False, True]
    assert pu.visible(1, 70, 71, 0, word=-1).tolist() == [True] * 65 + [False] * 6


def test_trees_are_closed_under_ancestors():
    masks, depths = pu.random_trees([64, 1, 20], np.random.default_rng(0))
    for lo, n in ((0, 64), (64, 1), (65, 20)):
        for i in range(n):
            w = masks[lo + i] & (2 ** 64 - 1)
            assert w >> i & 1 and w < 2 ** (i + 1) and bin(w).count("1") == depths[lo + i] + 1
            for t in range(i):
                if w >> t & 1:
                    assert masks[lo + t] & (2 ** 64 - 1) & ~w == 0


def test_definition_is_the_contiguous_one():
    """Pages dealt out in disorder against kv_util.attention over the rows that they hold."""
    rng = np.random.default_rng(2)
    past, new, ps, N, G, H = [9, 0, 30], [3, 20, 1], 8, 2, 3, 16
    table, pages = pu.table_for(rng, [p + n for p, n in zip(past, new)], ps)
    k, v = (torch.from_numpy(rng.standard_normal((pages, N, ps, H))) for _ in range(2))
    starts = [0, 3, 23, 24]
    q = torch.from_numpy(rng.standard_normal((26, G * N * H)))
    out, bound, owned = pu.attention(q, k, v, table, past, starts, G * N, 0.3, cap=4.0, weight_eps=2.0 ** -11)
    assert owned.tolist() == [True] * 24 + [False] * 2
    for b in range(3):
        total = past[b] + new[b]
        kk, vv = (pu.rows_of(x, table[b], total)[None] for x in (k, v))
        want, limit = ku.attention(q[None, starts[b]:starts[b + 1]], kk, vv, [past[b]], G * N, 0.3, 4.0, weight_eps=2.0 ** -11)
        assert torch.allclose(out[starts[b]:starts[b + 1]], want[0], rtol=1e-12, atol=1e-12)
        # the same count of roundings; the largest value is of those that some token of the sequence sees
        assert (bound[starts[b]:starts[b + 1]] >= limit[0] * (1 - 1e-9)).all()


def test_bad_pages_hold_zeros_by_definition():
    k = torch.ones((2, 1, 4, 3))
    rows = pu.rows_of(k, [1, -1, 2, 0, 99], 15)
    assert rows[0, :, 0].tolist() == [1.0] * 4 + [0.0] * 8 + [1.0] * 3
