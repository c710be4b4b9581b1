"""Attention over the caches on the GPU where numbers are far apart: value scales of blocks that a row does not
see, caps of every size, infinite keys under a cap, small queries over large keys."""

import numpy as np
import pytest
import torch

import kv_util as ku
from test_gpu_kv import _call, _make, _want

pytestmark = pytest.mark.gpu

# scales that no append writes: far too large, far too small, between powers of two, negative, not finite
WILD = [2.0 ** 30, 1e30, 3.7e20, 2.0 ** 126, 3.4e38, 1e-40, 0.0, -1.0, -2.5e33, 1234.5, float("nan"), float("inf"),
        float("-inf")]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S, G", [(1, 4), (5, 4), (5, 2), (100, 4), (300, 1)])
@pytest.mark.parametrize("H", [64, 128, 256])
@pytest.mark.parametrize("cap", [0.0, 6.0])
def test_scales_that_no_row_sees(lib, cuda, dtype, S, G, H, cap):
    """A padded front and a hole between documents, whose blocks' scales hold anything."""
    B, N, L = 2, 2, 700
    past = [L - S - 40, 333]
    a = _make(51, dtype, B, S, G * N, N, H, L, past, True, cap=cap)
    ids = torch.zeros((B, L), dtype=torch.int32)
    ids[:, :48], ids[:, 160:208], ids[0, 272:288] = 7, 8, 9
    a["docs"] = ids
    want, bound = _want(a, cuda)
    ku.close(_call(lib, a, cuda), want, bound)
    hidden = [n for n in range(-(-L // 16)) if bool((ids[0, 16 * n:16 * n + 16] != 0).all())]
    for turn in range(5):
        for name in ("ks", "vs"):
            for n, blk in enumerate(hidden):
                a[name][0, :, blk] = WILD[(n + 3 * turn) % len(WILD)]
                if blk != 17:  # the second sequence has no third hole
                    a[name][1, :, blk] = WILD[(n + 3 * turn + 5) % len(WILD)]
        ku.close(_call(lib, a, cuda), want, bound, f"turn {turn}")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S, G", [(5, 4), (5, 1), (40, 2), (150, 4), (300, 1)])
@pytest.mark.parametrize("up", [20, 30, 60])
def test_value_scales_ahead_of_a_query(lib, cuda, dtype, S, G, up):
    """Blocks of later tokens, of another document and behind a prefix have scales 2^up larger: rows that do not
    see them keep their accuracy."""
    B, N, H, L = 2, 2, 64, 500
    past = [L - S - 3, 100 - S % 16 + 14]  # drafts that begin in one block and end in the next
    for extra in ({}, dict(alibi=True), dict(prefix=30), dict(docs=3)):
        a = _make(52, dtype, B, S, G * N, N, H, L, past, True, **extra)
        if extra.get("docs"):
            ids = torch.zeros((B, L), dtype=torch.int32)
            ids[:, 64:128] = 3
            for b in range(B):
                ids[b, past[b] + S // 2:] = 4  # half of the rows see only each other
            a["docs"] = ids
            a["vs"][:, :, 4:8] *= 2.0 ** up
            a["vs"][:, 0] = torch.where(torch.arange(a["vs"].shape[2]) < 4, 1.0, 2.0 ** -40) * a["vs"][:, 0]
        for b in range(B):
            last = (past[b] + S - 1) // 16
            first = max(past[b] // 16 + 1, last - 3)
            a["vs"][b, :, first:last + 1] *= 2.0 ** up
        want, bound = _want(a, cuda)
        keep = want.abs() + bound < (3e4 if dtype == "f16" else 1e38)  # what the output's type holds
        ku.close(_call(lib, a, cuda)[keep], want[keep], bound[keep], str(extra))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S, G", [(2, 4), (4, 4), (3, 4), (100, 1)])
@pytest.mark.parametrize("up", [20, 30, 60])
def test_value_scales_of_another_rows_document(lib, cuda, dtype, S, G, up):
    """Two documents in turns along the cache, the second one's value scales 2^up larger; tokens of either."""
    N, H, L = 2, 64, 8200
    past = L - S - 60
    a = _make(57, dtype, 1, S, G * N, N, H, L, [past], True)
    ids = (torch.arange(L) // 64 % 4 == 1).int() * 4
    ids[past:] = torch.arange(L - past) % 2 * 4
    a["docs"] = ids[None].int()
    second = (ids[::16] == 4) & (torch.arange(0, L, 16) + 16 <= past)
    a["vs"] = torch.where(second, 2.0 ** up, 1.0) * a["vs"]
    want, bound = _want(a, cuda)
    keep = want.abs() + bound < (3e4 if dtype == "f16" else 1e38)
    for room in (None, 0):
        ws = None if room is None else torch.empty(room, dtype=torch.uint8, device=cuda)
        ku.close(_call(lib, a, cuda, workspace=ws)[keep], want[keep], bound[keep], str(room))


def _tight(a, dev, scale):
    """kv_util.attention's result with a bound whose share for the cap goes with the capped score, not with the
    cap: tanh(y) for |y| <= 0.4 by a polynomial to 1.2e-7 of it, above as 1 - 2 / (1 + e^(2y)) by an exponential
    to 2^-22 and a reciprocal to 2^-23, which is off by 2 / (1 + e) (e / (1 + e) 2^-22 + 3 * 2^-24) + 2^-25, at
    most 4 * 2^-22 of tanh(y) (at y = -0.4); two more roundings for scaling. 10 * 2^-23 in all. A negative
    exponential's result below 2^-126 counts as 0, which is 1e-38 of the cap's largest value, 1."""
    out, old = _want(a, dev, scale)
    cap = a["softcap"]
    if "ks" in a:
        k, v = (torch.from_numpy(ku.values(a[n].numpy(), a[n + "s"].numpy())).to(dev) for n in ("k", "v"))
    else:
        k, v = a["k"].double().to(dev), a["v"].double().to(dev)
    q = a["q"].double().to(dev)
    B, S, _ = q.shape
    N, H, Nq = k.shape[1], k.shape[3], a["num_heads"]
    G = Nq // N
    t = a["q"].dtype
    weight_eps = 2.0 ** -24 if t == torch.float32 else 2.0 ** -11 if "ks" in a else ku.EPS[t]
    bound = torch.zeros((B, S, Nq, H), dtype=torch.float64, device=dev)
    qh = q.view(B, S, Nq, H)
    for b in range(B):
        for s in range(S):
            past = int(a["past"][b])
            n = past + s + 1
            for h in range(N):
                kk, vv, rows = k[b, h, :n], v[b, h, :n], qh[b, s, h * G:(h + 1) * G]
                d = (H + 8) * 2.0 ** -23 * (rows.abs() @ kk.abs().T) * abs(scale)
                y = cap * torch.tanh(rows @ kk.T * scale / cap)
                d = d + 10 * 2.0 ** -23 * y.abs()
                if a["slopes"] is not None:
                    bias = a["slopes"][h * G:(h + 1) * G, None].double().to(dev) * (past + s - torch.arange(n, device=dev))
                    y, d = y - bias, d + 4 * 2.0 ** -23 * bias
                d = d + 4 * 2.0 ** -23 * y.abs()
                p = torch.softmax(y, -1)
                off = p * torch.expm1(2 * d.clamp(max=50.0))
                mean = p @ vv.abs()
                total = (2 * weight_eps + (n + 16) * 2.0 ** -23) * mean + off @ vv.abs() + off.sum(-1, keepdim=True) * mean
                if weight_eps > 2.0 ** -20:
                    total = total + n * 2.0 ** -25 * vv.abs().amax()
                bound[b, s, h * G:(h + 1) * G] = total
    return out, bound.view(B, S, -1)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S, G", [(1, 4), (6, 4), (70, 4)])
@pytest.mark.parametrize("cap", [0.05, 1.0, 50.0, 1e4, 1e5, 1e6, 1e9, 1e20, 3e38])
def test_caps_of_every_size(lib, cuda, dtype, fp8, S, G, cap):
    """Scores of a few units under caps from far below them to far above, next to keys whose scores are about
    -cap / 2 where the storage type holds such: a large cap tends to none."""
    N, H, L = 2, 64, 400
    for alibi in (False, True):
        a = _make(53, dtype, 1, S, G * N, N, H, L, [L - S - 30], fp8, cap=cap, alibi=alibi, qscale=0.3)
        a["q"] = a["q"].view(1, S, G * N, H).clone()
        a["q"][..., 0] = 1.0
        a["q"] = a["q"].view(1, S, -1)
        low = -min(cap / 2, 2.0 ** 15)  # of the first dimension, in a few keys
        if fp8:
            a["ks"][:] = 2.0 ** -6  # as _make's scale of the middle
            a["k"][..., 0] = 0
            e = max(-100.0, np.floor(np.log2(-low / 256)))
            for blk in (3, 9, 20):  # whole blocks
                a["ks"][:, :, blk] = 2.0 ** e
                a["k"][:, :, 16 * blk:16 * blk + 16] = 0
                a["k"][:, :, 16 * blk:16 * blk + 16, 0] = int(ku.e4m3(np.array(low / 2.0 ** e)))
        else:
            a["k"][..., 0] = 0
            for j in (3, 50, 51, 200, 333):
                a["k"][:, :, j, 1:] = 0
                a["k"][:, :, j, 0] = low
        want, bound = _tight(a, cuda, 1.0)
        ku.close(_call(lib, a, cuda, scale=1.0), want, bound, str(alibi))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S", [1, 6, 70])
@pytest.mark.parametrize("cap, scale", [(1e-38, 1.0), (1e-44, 1.0), (1e-30, 1e20), (2.0, 1.2e30), (2.0, -1.2e30), (0.0, 1e-45),
                                        (3e38, 1e-45)])
def test_caps_and_scales_at_the_ends_of_their_type(lib, cuda, dtype, fp8, S, cap, scale):
    """Queries of zeros among others, whose score is 0 whatever the scale, and of 1e-3: a vanishing cap or scale
    weighs all keys alike; with a vast scale a score is at either end of the cap."""
    a = _make(54, dtype, 1, S, 8, 2, 64, 300, [300 - S - 9], fp8, cap=cap)
    a["q"] = a["q"].view(1, S, 8, 64).clone()
    a["q"][:, :, ::3] = 0
    a["q"] = a["q"].view(1, S, -1)
    got = _call(lib, a, cuda, scale=scale)
    if abs(scale) < 2:  # all scores are within 1e-30 of 0
        b = dict(a, q=torch.zeros_like(a["q"]), softcap=0.0)
        want, bound = _want(b, cuda, 1.0)
        ku.close(got, want, bound)
        return
    k = torch.from_numpy(ku.values(a["k"].numpy(), a["ks"].numpy())) if fp8 else a["k"].double()
    v = torch.from_numpy(ku.values(a["v"].numpy(), a["vs"].numpy())) if fp8 else a["v"].double()
    for s in range(S):
        n = 300 - S - 9 + s + 1
        for h in range(8):
            y = k[0, h // 4, :n] @ a["q"][0, s, 64 * h:64 * h + 64].double()
            assert not a["q"][0, s, 64 * h:64 * h + 64].any() or float(y.abs().min()) > 0
            p = torch.softmax(cap * torch.sign(y) * (1.0 if scale > 0 else -1.0), -1)
            want = p @ v[0, h // 4, :n]
            limit = (2.0 ** -9 if dtype != "bf16" else 2.0 ** -6) * (p @ v[0, h // 4, :n].abs()) + n * 2.0 ** -24
            assert ((got[0, s, 64 * h:64 * h + 64].double().cpu() - want).abs() <= limit).all(), (s, h)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S", [1, 6, 40, 130])
@pytest.mark.parametrize("alibi", [False, True])
def test_infinite_keys_under_a_cap(lib, cuda, dtype, S, alibi):
    """A visible key whose product with the query is -inf scores -softcap wherever it lies: in a key tile that
    is partly hidden, in a whole tile, in a tile of nothing else; hidden ones stay hidden."""
    L = 420
    for bad in ([3], [3, 60, 130, 131, 390], list(range(128)), list(range(100, 280)), list(range(L))):
        a = _make(55, dtype, 1, S, 2, 1, 64, L, [L - S - 5], False, cap=2.0, alibi=alibi)
        a["q"] = a["q"].abs() + 0.1
        b = dict(a, k=a["k"].clone())
        b["k"][0, 0, bad] = -64.0  # a product far below -softcap
        want, bound = _want(b, cuda)
        a["k"][0, 0, bad] = float("-inf")
        ku.close(_call(lib, a, cuda), want, bound, f"{len(bad)} keys")
        docs = torch.zeros((1, L), dtype=torch.int32)
        docs[0, bad[:len(bad) // 2]] = 1
        docs[0, L - S - 5:] = 0
        for x in (a, b):
            x["docs"] = docs
        want, bound = _want(b, cuda)
        ku.close(_call(lib, a, cuda), want, bound, f"{len(bad)} keys, documents")


@pytest.mark.parametrize("S", [1, 6, 70])
@pytest.mark.parametrize("cap", [0.0, 3.0])
@pytest.mark.parametrize("down", [60, 100, 118])
def test_small_queries_over_large_keys(lib, cuda, S, cap, down):
    """bfloat16 queries near 2^-down over 8-bit keys near 2^down: the scores are a few units. And the other way."""
    for sign in (-1, 1):
        e = down if sign < 0 else min(down, 110)  # scales are 2^-120 at least
        a = _make(56, "bf16", 1, S, 8, 2, 64, 300, [300 - S], True, cap=cap)
        a["q"] = (a["q"].float() * 2.0 ** (sign * e)).to(torch.bfloat16)
        a["ks"] = a["ks"] * 2.0 ** (-sign * e)
        want, bound = _want(a, cuda, 0.3)
        ku.close(_call(lib, a, cuda, scale=0.3), want, bound, str(sign))
