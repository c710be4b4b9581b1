"""The paged-cache operators on the GPU against their 64-bit definitions (paged_util), against the contiguous
operators' bits, and runs of them together."""

import numpy as np
import pytest
import torch

import kv_util as ku
import paged_util as pu

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _make(seed, dtype, Nq, Nkv, H, ps, past, new, lead=0, behind=0, cap=0.0, window=0, alibi=False, tree=False,
          qscale=1.0):
    """Host tensors of a call: `lead` tokens before the first sequence, `behind` after the last."""
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    t = T[dtype]
    table, pages = pu.table_for(rng, [p + n for p, n in zip(past, new)], ps)
    starts = [lead]
    for n in new:
        starts.append(starts[-1] + n)
    tokens = starts[-1] + behind
    a = dict(Nq=Nq, past=past, starts=starts, table=table, cap=cap, window=window, most=max(new + [1]))
    a["q"] = (torch.randn((tokens, Nq * H), generator=g) * qscale).to(t)
    a["k"], a["v"] = (torch.randn((pages, Nkv, ps, H), generator=g).to(t) for _ in range(2))
    a["slopes"] = torch.exp2(-8.0 * (torch.arange(Nq) + 1.0) / Nq) if alibi else None
    a["masks"] = None
    if tree:
        a["masks"] = [0x5555] * lead + pu.random_trees(new, rng)[0] + [-1] * behind
    return a


def _i32(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


def _call(lib, a, dev, **kw):
    masks = None if a["masks"] is None else torch.tensor(a["masks"], dtype=torch.int64, device=dev)
    kw.setdefault("max_query_len", a["most"])
    return lib.kv_attention_paged(a["q"].to(dev), a["k"].to(dev), a["v"].to(dev), _i32(a["table"], dev),
                                  _i32(a["past"], dev), num_heads=a["Nq"], query_starts=_i32(a["starts"], dev),
                                  softcap=a["cap"], window=a["window"],
                                  alibi_slopes=None if a["slopes"] is None else a["slopes"].to(dev), tree_masks=masks, **kw)


def _want(a, dev, scale=None, most=None):
    H = a["k"].shape[3]
    t = a["q"].dtype
    return pu.attention(a["q"].to(dev), a["k"].to(dev), a["v"].to(dev), a["table"], a["past"], a["starts"], a["Nq"],
                        H ** -0.5 if scale is None else scale, a["cap"], a["window"],
                        None if a["slopes"] is None else a["slopes"].to(dev), a["masks"], weight_eps=ku.EPS[t], most=most)


def _check(lib, a, dev, what="", **kw):
    """The call's rows against the definition; rows that are nobody's stay as they were."""
    out = torch.full_like(a["q"], 7.0).to(dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    got = _call(lib, a, dev, out=out, status=status, **kw)
    want, bound, owned = _want(a, dev, kw.get("scale"))
    assert torch.equal(got[~owned], torch.full_like(got[~owned], 7.0)), what
    pu.close(got[owned], want[owned], bound[owned], what)
    assert int(status) == 0, what
    return got


# (Nq, Nkv, H, page size, past, new): single tokens, drafts, prompts, both; pages that end inside a tile and pages
# as long as a cache; lengths of zero and one; sequences without tokens
SHAPES = {
    "one": (4, 1, 64, 16, [0], [1]),
    "token": (8, 2, 128, 16, [0, 17, 299], [1, 1, 1]),
    "token_odd": (7, 1, 96, 8, [0, 15, 16, 127, 130], [1] * 5),
    "token_long": (8, 2, 128, 64, [4999, 2049], [1, 1]),
    "token_mha": (3, 3, 32, 32, [63, 64], [1, 1]),
    "token_wide": (16, 8, 256, 16, [199, 31], [1, 1]),
    "token_group": (40, 2, 64, 24, [149, 90], [1, 1]),
    "token_page": (8, 2, 128, 1024, [700, 1023], [1, 1]),
    "few": (8, 2, 128, 16, [0, 395, 64], [4, 2, 3]),
    "few_group": (21, 3, 64, 128, [128, 257], [2, 1]),
    "holes": (8, 2, 64, 16, [5, 0, 40, 33], [0, 1, 0, 2]),
    "chunk": (8, 2, 128, 16, [0, 263], [70, 61]),
    "chunk_mha": (2, 2, 64, 64, [0], [150]),
    "chunk_odd": (6, 2, 80, 40, [7, 369], [131, 99]),
    "chunk_wide": (4, 2, 256, 16, [100], [67]),
    "chunk_group": (28, 4, 128, 256, [250], [40]),
    "prompt": (4, 1, 128, 32, [0], [300]),
    "mixed": (8, 2, 128, 16, [100, 0, 77, 511, 3], [1, 260, 1, 2, 75]),
    "mixed_small": (12, 2, 64, 8, [300, 20, 0], [1, 33, 130]),
    "mixed_many": (8, 2, 128, 16, [7 * i % 400 for i in range(100)], [1] * 40 + [150] + [2] * 58 + [33]),
    "mixed_wide": (4, 4, 256, 32, [11 * i % 300 for i in range(60)], [90] + [2] * 59),
    "mixed_narrow": (6, 6, 64, 8, [5 * i % 200 for i in range(50)], [3] * 20 + [300, 40] + [1] * 28),
    "scalar": (4, 2, 19, 16, [3, 51], [9, 1]),
    "tiny_head": (4, 4, 2, 16, [3, 33], [33, 2]),
    "tiny_page": (8, 2, 64, 1, [30, 0], [3, 50]),
    "odd_page": (8, 2, 128, 20, [30, 77], [3, 70]),
}
MASKS = {
    "plain": {}, "cap": dict(cap=5.0, qscale=3.0), "alibi": dict(alibi=True), "window": dict(window=37),
    "window_one": dict(window=1), "all": dict(cap=20.0, alibi=True, window=100),
}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("masks", ["plain", "all"])
def test_attention(lib, cuda, dtype, shape, masks):
    _check(lib, _make(1, dtype, *SHAPES[shape], **MASKS[masks]), cuda)


@pytest.mark.parametrize("shape", ["token", "token_long", "few", "chunk", "chunk_odd", "mixed", "mixed_small", "chunk_wide"])
@pytest.mark.parametrize("masks", ["cap", "alibi", "window", "window_one"])
def test_each_mask(lib, cuda, shape, masks):
    for dtype in ("f16", "bf16", "f32"):
        _check(lib, _make(2, dtype, *SHAPES[shape], **MASKS[masks]), cuda, dtype)


TREES = {
    "one": (8, 2, 128, 16, [500], [60]),
    "root": (8, 2, 128, 16, [0, 40], [1, 1]),
    "empty_past": (4, 4, 64, 32, [0, 1], [64, 33]),
    "batch": (32, 8, 128, 16, [0, 15, 300, 1000], [26, 64, 1, 40]),
    "few": (8, 8, 64, 8, [100, 7], [3, 16]),
    "wide": (4, 2, 256, 64, [77, 130], [20, 9]),
    "pad": (10, 5, 96, 24, [50, 3], [31, 5]),
    "scalar": (4, 2, 19, 16, [30], [20]),
}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", TREES)
@pytest.mark.parametrize("cap", [0.0, 8.0])
def test_trees(lib, cuda, dtype, shape, cap):
    _check(lib, _make(3, dtype, *TREES[shape], tree=True, cap=cap, lead=2, behind=3), cuda)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_masks_are_any_words(lib, cuda, dtype):
    """Bits ahead of a token, bits of tokens that do not exist, words without a bit; with nothing behind, such a
    token sees no key and gives 0."""
    rng = np.random.default_rng(5)
    a = _make(4, dtype, 8, 2, 128, 16, [0, 21, 0], [30, 17, 2], tree=True)
    a["masks"] = [int(x) for x in rng.integers(-2 ** 63, 2 ** 63 - 1, 49)]
    a["masks"][3] = a["masks"][47] = 0
    a["masks"][48] = -4  # only tokens that do not exist
    got = _check(lib, a, cuda)
    assert not got[3].any() and not got[47].any() and not got[48].any()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("kind", ["token", "chunk", "mixed"])
def test_tokens_of_nobody(lib, cuda, dtype, kind):
    """Rows before the first sequence and behind the last one are left as they were."""
    _check(lib, _make(6, dtype, *SHAPES[kind], lead=3, behind=41), cuda)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_random_shapes(lib, cuda, dtype):
    rng = np.random.default_rng(12)
    for n in range(24):
        Nkv, G = int(rng.integers(1, 4)), int(rng.integers(1, 9))
        H = int(rng.choice([8, 16, 24, 48, 64, 72, 96, 112, 128, 160, 256]))
        B = int(rng.integers(1, 6))
        new = rng.choice([0, 1, 1, 2, 4, 16, 17, 50, 129], B).tolist()
        past = rng.integers(0, 500, B).tolist()
        a = _make(100 + n, dtype, G * Nkv, Nkv, H, int(rng.choice([8, 16, 32, 48, 64, 128, 7])), past, new,
                  lead=int(rng.integers(0, 3)), behind=int(rng.integers(0, 3)) + (sum(new) == 0),
                  cap=float(rng.choice([0, 10.0])), alibi=bool(rng.integers(2)), window=int(rng.choice([0, 0, 1, 33, 200])))
        _check(lib, a, cuda, str((new, past, G, Nkv, H)))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", ["token", "token_odd", "few", "chunk", "prompt", "chunk_wide", "mixed"])
@pytest.mark.parametrize("window", [0, 30])
def test_nothing_hidden_is_used(lib, cuda, dtype, shape, window):
    """NaN and infinities behind the last row, in front of the window and ahead of a token change nothing."""
    a = _make(7, dtype, *SHAPES[shape], window=window)
    want, bound, owned = _want(a, cuda)
    keep = owned.clone()
    ps = a["k"].shape[2]
    for b, (p, lo, hi) in enumerate(zip(a["past"], a["starts"], a["starts"][1:])):
        n = hi - lo
        last = (p + n - 1) // ps
        for name, bad in (("k", float("nan")), ("v", float("inf"))):
            x = a[name]
            x[a["table"][b][last], :, (p + n - 1) % ps + 1:] = bad
            if window:
                for j in range(max(0, p - window + 1)):
                    x[a["table"][b][j // ps], :, j % ps] = bad
            if n > 1:
                x[a["table"][b][last], :, (p + n - 1) % ps] = bad  # the last token's row, seen by it alone
        if n > 1:
            keep[hi - 1] = False
    used = {x for row, p, lo, hi in zip(a["table"], a["past"], a["starts"], a["starts"][1:]) for x in row[:-(-(p + hi - lo) // ps)]}
    for x in range(a["k"].shape[0]):
        if x not in used:
            a["k"][x], a["v"][x] = float("inf"), float("nan")
    got = _call(lib, a, cuda)
    pu.close(got[keep], want[keep], bound[keep])
    assert not torch.isfinite(got[owned & ~keep]).any()  # and what is seen is not hidden


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("shape", ["token", "chunk", "mixed"])
def test_bad_pages_hold_zeros(lib, cuda, dtype, shape):
    a = _make(8, dtype, *SHAPES[shape])
    ps = a["k"].shape[2]
    for b, bad in zip(range(len(a["past"])), (-1, 2 ** 31 - 1, a["k"].shape[0], -2 ** 31, 10 ** 6)):
        a["table"][b][(a["past"][b] + a["starts"][b + 1] - a["starts"][b] - 1) // ps // 2] = bad
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    got = _call(lib, a, cuda, status=status)
    want, bound, owned = _want(a, cuda)
    pu.close(got[owned], want[owned], bound[owned])
    assert int(status) == 4


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_rows_outside_the_table(lib, cuda, dtype):
    """Lengths below zero and beyond the table: what the formula says, and status bit 2."""
    for past in ([-3, 10], [300, 10], [-2 ** 31, 10], [2 ** 31 - 1, 10]):
        for new in ([1, 1], [5, 2], [70, 1]):
            a = _make(9, dtype, 8, 2, 64, 16, [60, 10], new)
            a["past"] = past
            a["table"][0] = [int(x) for x in np.random.default_rng(0).permutation(a["k"].shape[0])[:len(a["table"][0])]]
            status = torch.zeros(1, dtype=torch.int32, device=cuda)
            got = _call(lib, a, cuda, status=status)
            want, bound, owned = _want(a, cuda)
            pu.close(got[owned], want[owned], bound[owned], str((past, new)))
            assert int(status) == 4


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_longer_sequences_are_left_out(lib, cuda, dtype):
    a = _make(10, dtype, 8, 2, 64, 16, [60, 10, 5], [1, 40, 3])
    for most in (1, 2, 39):
        out = torch.full_like(a["q"], 7.0).to(cuda)
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        _call(lib, a, cuda, max_query_len=most, out=out, status=status)
        want, bound, owned = _want(a, cuda, most=most)
        assert torch.equal(out[~owned], torch.full_like(out[~owned], 7.0))
        pu.close(out[owned], want[owned], bound[owned], str(most))
        assert int(status) == 4


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("scale,cap", [(-0.3, 0.0), (0.0, 0.0), (4.0, 0.0), (-0.5, 3.0), (1.0, 1e30)])
def test_scales(lib, cuda, dtype, scale, cap):
    for shape in ("token", "chunk", "mixed"):
        _check(lib, _make(11, dtype, *SHAPES[shape], cap=cap), cuda, shape, scale=scale)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_without_starts(lib, cuda, dtype):
    """(B, S, hidden) is what query_starts of equal lengths say."""
    for B, S in ((3, 1), (2, 4), (2, 70)):
        a = _make(12, dtype, 8, 2, 128, 16, list(range(20, 20 + 60 * B, 60)), [S] * B)
        want = _call(lib, a, cuda)
        got = lib.kv_attention_paged(a["q"].to(cuda).view(B, S, -1), a["k"].to(cuda), a["v"].to(cuda), _i32(a["table"], cuda),
                                     _i32(a["past"], cuda), num_heads=8)
        assert torch.equal(got.view(B * S, -1), want)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_pages_of_one_tensor(lib, cuda, dtype):
    """K and V side by side in each page: a stride between pages that is not theirs."""
    for shape in ("token", "chunk", "mixed", "odd_page"):
        a = _make(13, dtype, *SHAPES[shape])
        both = torch.stack([a["k"], a["v"]], 1).to(cuda)
        b = dict(a, k=both[:, 0], v=both[:, 1])
        assert torch.equal(_call(lib, a, cuda), _call(lib, b, cuda))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_contiguous_cache_is_pages(lib, cuda, dtype):
    """A contiguous cache is a pool of B pages: kv_attention's definition."""
    g = torch.Generator().manual_seed(3)
    B, Nq, Nkv, H, L = 3, 8, 2, 128, 203
    for S in (1, 3, 90):
        q = torch.randn((B, S, Nq * H), generator=g).to(T[dtype]).to(cuda)
        k, v = (torch.randn((B, Nkv, L, H), generator=g).to(T[dtype]).to(cuda) for _ in range(2))
        past = _i32([0, 57, L - S], cuda)
        got = lib.kv_attention_paged(q, k, v, torch.arange(B, dtype=torch.int32, device=cuda)[:, None].contiguous(), past,
                                     num_heads=Nq)
        want, bound = ku.attention(q.double(), k.double(), v.double(), past.tolist(), Nq, H ** -0.5, weight_eps=ku.EPS[T[dtype]])
        pu.close(got, want, bound)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("room", [None, 0, 4096, 200_000])
def test_workspaces(lib, cuda, dtype, room):
    """Less workspace than planned splits less; its contents do not matter."""
    for shape in ("token_long", "mixed", "one", "mixed_many", "prompt"):
        a = _make(14, dtype, *SHAPES[shape])
        ws = None if room is None else torch.full((room,), 255, dtype=torch.uint8, device=cuda)
        _check(lib, a, cuda, shape, workspace=ws)


# --------------------------------------------------------------------------
# append
# --------------------------------------------------------------------------

def _append_case(seed, dtype, Nq, Nkv, H, ps, past, new, norm=False, inter=0, rd=0, separate=False, lead=0, behind=0,
                 positions=False):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    t = T[dtype]
    table, pages = pu.table_for(rng, [p + n for p, n in zip(past, new)], ps)
    starts = [lead]
    for n in new:
        starts.append(starts[-1] + n)
    tokens, rows = starts[-1] + behind, 700
    a = dict(Nq=Nq, Nkv=Nkv, H=H, past=past, starts=starts, table=table, inter=inter, rd=rd)
    a["q"] = torch.randn((tokens, (Nq if separate else Nq + 2 * Nkv) * H), generator=g).to(t)
    a["key"], a["value"] = ((torch.randn((tokens, Nkv * H), generator=g).to(t) for _ in range(2)) if separate else (None, None))
    a["cos"], a["sin"] = (torch.randn((rows, (rd or H) // 2), generator=g).to(t) for _ in range(2))
    a["k"], a["v"] = (torch.randn((pages, Nkv, ps, H), generator=g).to(t) for _ in range(2))
    a["qw"], a["kw"] = ((torch.rand(H, generator=g) + 0.5).to(t) for _ in range(2)) if norm else (None, None)
    a["pos"] = torch.from_numpy(rng.integers(0, rows, tokens)) if positions else None
    return a


def _append(lib, a, dev, k, v, **kw):
    on = {n: None if a[n] is None else a[n].to(dev) for n in ("q", "key", "value", "cos", "sin", "qw", "kw", "pos")}
    return lib.rope_apply_qkv_paged(on["q"], on["cos"], on["sin"], on["pos"], num_heads=a["Nq"], kv_num_heads=a["Nkv"],
                                    k_pages=k, v_pages=v, page_table=_i32(a["table"], dev),
                                    past_seq_lens=_i32(a["past"], dev), query_starts=_i32(a["starts"], dev), key=on["key"],
                                    value=on["value"], interleaved=a["inter"], rotary_embedding_dim=a["rd"],
                                    q_norm_weight=on["qw"], k_norm_weight=on["kw"], **kw)


def _check_append(lib, a, dev, what=""):
    """Against the bits of the Q/K operators, one sequence at a time, and every other row as it was."""
    k, v = a["k"].to(dev), a["v"].to(dev)
    q_out = torch.full((a["q"].shape[0], a["Nq"] * a["H"]), 7.0, dtype=a["q"].dtype, device=dev)
    status = torch.zeros(1, dtype=torch.int32, device=dev)
    _append(lib, a, dev, k, v, q_out=q_out, status=status)
    want_q, want_k, want_v = torch.full_like(q_out, 7.0), a["k"].to(dev), a["v"].to(dev)
    ps = want_k.shape[2]
    for b, (p, lo, hi) in enumerate(zip(a["past"], a["starts"], a["starts"][1:])):
        if lo == hi:
            continue
        part = {n: None if a[n] is None else a[n][None, lo:hi].to(dev) for n in ("q", "key", "value", "pos")}
        rest = {n: None if a[n] is None else a[n].to(dev) for n in ("cos", "sin", "qw", "kw")}
        kc, vc = (torch.zeros((1, a["Nkv"], p + hi - lo, a["H"]), dtype=q_out.dtype, device=dev) for _ in range(2))
        q, _ = lib.rope_apply_qkv(part["q"], rest["cos"], rest["sin"], part["pos"], num_heads=a["Nq"], kv_num_heads=a["Nkv"],
                                  key=part["key"], value=part["value"], interleaved=a["inter"], rotary_embedding_dim=a["rd"],
                                  k_cache=kc, v_cache=vc, past_seq_lens=_i32([p], dev), q_norm_weight=rest["qw"],
                                  k_norm_weight=rest["kw"])
        want_q[lo:hi] = q[0]
        for j in range(p, p + hi - lo):
            want_k[a["table"][b][j // ps], :, j % ps] = kc[0, :, j]
            want_v[a["table"][b][j // ps], :, j % ps] = vc[0, :, j]
    for name, got, want in (("q", q_out, want_q), ("k", k, want_k), ("v", v, want_v)):
        assert torch.equal(got, want), f"{what} {name}"
    assert int(status) == 0, what


APPENDS = {
    "decode": (32, 8, 128, 16, [0, 15, 16, 300], [1] * 4),
    "one_head": (1, 1, 64, 8, [3], [2]),
    "odd_heads": (7, 1, 96, 24, [0, 77], [5, 3]),
    "prompt": (28, 4, 128, 64, [10, 0], [200, 131]),
    "holes": (8, 2, 64, 16, [5, 0, 40, 33], [0, 1, 0, 2]),
    "tiny_page": (6, 3, 32, 1, [4, 9], [7, 1]),
    "odd_page": (6, 3, 40, 20, [4, 90], [70, 1]),
    "wide": (4, 2, 256, 16, [9], [33]),
    "scalar": (4, 2, 6, 16, [9, 0], [33, 1]),
    "many": (8, 8, 64, 16, list(range(200)), [1] * 200),
}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", APPENDS)
def test_append(lib, cuda, dtype, shape):
    H = APPENDS[shape][2]
    for n, kw in enumerate((dict(), dict(inter=1, rd=H // 2 if H % 4 == 0 else 0), dict(separate=True, positions=True),
                            dict(lead=2, behind=5, positions=True, rd=2))):
        _check_append(lib, _append_case(20 + n, dtype, *APPENDS[shape], **kw), cuda, str(kw))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", APPENDS)
def test_append_norm(lib, cuda, dtype, shape):
    H = APPENDS[shape][2]
    if dtype == "f32" and H > 128:
        pytest.skip("the contiguous operator refuses such heads")
    for n, kw in enumerate((dict(), dict(inter=1, rd=H // 2 if H % 4 == 0 else 0, separate=True), dict(lead=1, behind=2, positions=True))):
        if (H // 2) % 8 and H > 32:
            kw = dict(kw, rd=16)
        a = _append_case(30 + n, dtype, *APPENDS[shape], norm=True, **kw)
        try:
            _check_append(lib, a, cuda, str(kw))
        except lib.RopeError as e:
            assert "units" in str(e)  # the contiguous operator's limit


def test_append_outside(lib, cuda):
    """Rows outside the table and pages outside the pool take nothing; positions outside the tables are copied."""
    a = _append_case(40, "f16", 4, 2, 64, 16, [10, 40], [3, 4])
    for past, bad, flags in (([-2, 40], None, 5), ([46, 40], None, 4), ([10, 40], -1, 4), ([10, 40], 10 ** 6, 4)):
        c = dict(a, past=past, table=[list(r) for r in a["table"]])
        c["table"][0] = c["table"][0][:1] + [x % a["k"].shape[0] for x in c["table"][0][1:]]
        if bad is not None:
            c["table"][1][40 // 16] = bad
        k, v = c["k"].to(cuda), c["v"].to(cuda)
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        before_k, before_v = k.clone(), v.clone()
        q = _append(lib, c, cuda, k, v, status=status)
        assert int(status) == flags
        full = _append(lib, a, cuda, k.clone(), v.clone())
        if bad is not None:
            assert torch.equal(q, full)
            changed = (k != before_k).flatten(1).any(1).nonzero().flatten().tolist()
            assert set(changed) <= {c["table"][0][0]}
        else:
            assert torch.equal(q[3:], full[3:])
            assert (v != before_v).flatten(1).any(1).sum() <= 2


def test_append_in_place(lib, cuda):
    a = _append_case(41, "bf16", 8, 2, 128, 16, [10, 40], [30, 4], separate=True, norm=True)
    k, v = a["k"].to(cuda), a["v"].to(cuda)
    want = _append(lib, a, cuda, k.clone(), v.clone())
    q = a["q"].to(cuda)
    got = _append(lib, dict(a, q=q), cuda, k, v, q_out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


# --------------------------------------------------------------------------
# keep
# --------------------------------------------------------------------------

def _keep(lib, dev, k, v, table, past, paths, width=None, **kw):
    width = max([len(p) for p in paths] + [1]) if width is None else width
    kept = _i32([p + [-5] * (width - len(p)) for p in paths], dev).view(len(paths), width)
    lib.kv_keep_paged(k, v, _i32(table, dev), _i32(past, dev), kept, _i32([len(p) for p in paths], dev), **kw)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("Nkv,H,ps", [(8, 128, 16), (1, 64, 64), (3, 19, 7), (2, 256, 1), (5, 96, 24)])
def test_keep(lib, cuda, dtype, Nkv, H, ps):
    rng = np.random.default_rng(50)
    past = [0, 5, 100, 63, 33]
    new = [64, 20, 60, 1, 30]
    table, pages = pu.table_for(rng, [p + n for p, n in zip(past, new)], ps)
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((pages, Nkv, ps, H), generator=g).to(T[dtype]).to(cuda) for _ in range(2))
    paths = [sorted(rng.choice(n, min(n, m), replace=False).tolist()) for n, m in zip(new, (40, 1, 9, 1, 0))]
    paths[1] = [19]
    want = {}
    for name, x in (("k", k), ("v", v)):
        y = x.clone()
        for b, path in enumerate(paths):
            for i, r in enumerate(path):
                y[table[b][(past[b] + i) // ps], :, (past[b] + i) % ps] = x[table[b][(past[b] + r) // ps], :, (past[b] + r) % ps]
        want[name] = y
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    _keep(lib, cuda, k, v, table, past, paths, status=status)
    assert torch.equal(k, want["k"]) and torch.equal(v, want["v"]) and int(status) == 0


def test_keep_refuses_sequences(lib, cuda):
    """Indices that do not ascend, twice the same, below zero, outside the table, in bad pages; counts below zero
    and above the width: that sequence stays as it is, the others' rows move."""
    rng = np.random.default_rng(51)
    ps, past = 16, [20, 30]
    good = [1, 3, 8]
    for paths, lens, spoil in (([good, [3, 1]], None, None), ([good, [2, 2]], None, None), ([good, [-1, 2]], None, None),
                               ([good, [1, 500]], None, None), ([good, [2 ** 31 - 1]], None, None), ([good, [0, 5]], [3, -1], None),
                               ([good, [0, 5]], [3, 4], None), ([good, [0, 17]], None, -1), ([good, [0, 17]], None, 10 ** 7)):
        table, pages = pu.table_for(rng, [90, 90], ps)
        if spoil is not None:
            table[1][(30 + 17) // ps] = spoil
        k, v = (torch.randn((pages, 2, ps, 64), device=cuda, dtype=torch.float16) for _ in range(2))
        want = [x.clone() for x in (k, v)]
        for x, y in zip((k, v), want):
            for i, r in enumerate(good):
                y[table[0][(20 + i) // ps], :, (20 + i) % ps] = x[table[0][(20 + r) // ps], :, (20 + r) % ps]
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        kept = _i32([p + [0] * (3 - len(p)) for p in paths], cuda)
        lib.kv_keep_paged(k, v, _i32(table, cuda), _i32(past, cuda), kept, _i32(lens or [len(p) for p in paths], cuda),
                          status=status)
        assert int(status) == 4, paths
        assert torch.equal(k, want[0]) and torch.equal(v, want[1]), paths


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("captured", [False, True])
def test_speculative_steps(lib, cuda, dtype, captured):
    """Prompts, then rounds of draft trees: append by depth, attend with masks, keep a path; the cache that
    results is that of the accepted tokens appended one behind the other, and each tree token's attention is
    that of its path. The rounds' calls run eagerly or from one graph that is replayed with new inputs."""
    t = T[dtype]
    B, Nq, Nkv, H, ps, n = 3, 8, 2, 64, 16, 12
    rng = np.random.default_rng(60)
    g = torch.Generator().manual_seed(60)
    lens = [17, 1, 40]
    width = 8
    table = _i32(rng.permutation(B * width).reshape(B, width).tolist(), cuda)
    k, v = lib.kv_cache_paged(B * width, Nkv, ps, H, t, cuda)
    angle = torch.arange(width * ps, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, H, 2).double() / H)
    cos, sin = angle.cos().to(t).to(cuda), angle.sin().to(t).to(cuda)
    starts = [0]
    for x in lens:
        starts.append(starts[-1] + x)
    heads = dict(num_heads=Nq, kv_num_heads=Nkv)
    prompt = torch.randn((starts[-1], (Nq + 2 * Nkv) * H), generator=g).to(t).to(cuda)
    past = torch.zeros(B, dtype=torch.int32, device=cuda)
    lib.rope_apply_qkv_paged(prompt, cos, sin, **heads, k_pages=k, v_pages=v, page_table=table, past_seq_lens=past,
                             query_starts=_i32(starts, cuda))
    # the accepted tokens so far, in a contiguous cache by the contiguous operator
    kc, vc = (torch.zeros((B, Nkv, width * ps, H), dtype=t, device=cuda) for _ in range(2))
    for b in range(B):
        lib.rope_apply_qkv(prompt[None, starts[b]:starts[b + 1]], cos, sin, **heads, k_cache=kc[b:b + 1], v_cache=vc[b:b + 1],
                           past_seq_lens=past[:1])
    past = _i32(lens, cuda)
    tree_starts = _i32([b * n for b in range(B + 1)], cuda)
    qkv = torch.zeros((B * n, (Nq + 2 * Nkv) * H), dtype=t, device=cuda)
    positions = torch.zeros(B * n, dtype=torch.int64, device=cuda)
    masks = torch.zeros(B * n, dtype=torch.int64, device=cuda)
    kept, kept_lens = torch.zeros((B, 4), dtype=torch.int32, device=cuda), torch.zeros(B, dtype=torch.int32, device=cuda)

    def attend():
        q = lib.rope_apply_qkv_paged(qkv, cos, sin, positions, **heads, k_pages=k, v_pages=v, page_table=table,
                                     past_seq_lens=past, query_starts=tree_starts)
        return lib.kv_attention_paged(q, k, v, table, past, num_heads=Nq, query_starts=tree_starts, max_query_len=n,
                                      tree_masks=masks)

    def keep():
        lib.kv_keep_paged(k, v, table, past, kept, kept_lens)
        past.add_(kept_lens)

    graphs = []
    for step in range(4):
        words, depths = pu.random_trees([n] * B, rng)
        new = torch.randn((B * n, (Nq + 2 * Nkv) * H), generator=g).to(t).to(cuda)
        qkv.copy_(new)
        masks.copy_(torch.tensor(words, device=cuda))
        base = past.tolist()
        positions.copy_(torch.tensor([base[b] + depths[b * n + i] for b in range(B) for i in range(n)], device=cuda))
        paths = []
        for b in range(B):
            leaf = int(rng.integers(0, n))
            path = [i for i in range(n) if words[b * n + leaf] >> i & 1][:4]
            paths.append(path)
        kept.copy_(torch.tensor([p + [0] * (4 - len(p)) for p in paths], device=cuda))
        kept_lens.copy_(torch.tensor([len(p) for p in paths], device=cuda))
        if captured and not graphs:
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                attend()  # warms up; repeating it changes nothing
            torch.cuda.current_stream().wait_stream(side)
            for fn in (attend, keep):
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    result = fn()
                graphs.append((graph, result))
        if captured:
            graphs[0][0].replay()
            out = graphs[0][1]
        else:
            out = attend()
        # each token of the accepted path: the contiguous operators over its path
        for b in range(B):
            for i, r in enumerate(paths[b]):
                q, _ = lib.rope_apply_qkv(new[None, b * n + r:b * n + r + 1], cos, sin, **heads, k_cache=kc[b:b + 1],
                                          v_cache=vc[b:b + 1], past_seq_lens=_i32([base[b] + i], cuda))
                want, bound = ku.attention(q.double(), kc[b:b + 1].double(), vc[b:b + 1].double(), [base[b] + i], Nq,
                                           H ** -0.5, weight_eps=ku.EPS[t])
                pu.close(out[b * n + r], want.view(-1), bound.view(-1), f"step {step}")
        if captured:
            graphs[1][0].replay()
        else:
            keep()
    for b in range(B):
        total = int(past[b])
        for pages, cache in ((k, kc), (v, vc)):
            got = pu.rows_of(pages, table[b].tolist(), total)
            assert torch.equal(got, cache[b, :, :total].double())


def test_streams_and_devices(lib, cuda):
    a = _make(61, "f16", *SHAPES["mixed"])
    want = _call(lib, a, cuda)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _call(lib, a, cuda, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)


def test_two_graphs_share_a_workspace(lib, cuda):
    """Two captured calls with one workspace, replayed in turn, keep nothing of each other in it."""
    calls = []
    need = 0
    for seed, shape in ((62, "token_long"), (63, "mixed")):
        a = _make(seed, "bf16", *SHAPES[shape])
        args = dict(q=a["q"].to(cuda), k=a["k"].to(cuda), v=a["v"].to(cuda), t=_i32(a["table"], cuda), p=_i32(a["past"], cuda),
                    s=_i32(a["starts"], cuda))
        tokens, (_, N, ps, H) = args["q"].shape[0], a["k"].shape
        need = max(need, lib.kv_attention_paged_workspace(args["q"].dtype, len(a["past"]), tokens, a["most"], a["Nq"], N, H, ps,
                                                          args["t"].shape[1]))
        calls.append((a, args))
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device=cuda)
    graphs = []
    for a, x in calls:
        def run(a=a, x=x):
            return lib.kv_attention_paged(x["q"], x["k"], x["v"], x["t"], x["p"], num_heads=a["Nq"], query_starts=x["s"],
                                          max_query_len=a["most"], workspace=ws)
        want = run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = run()
        graphs.append((graph, got, want))
    for _ in range(3):
        for graph, got, want in graphs:
            got.zero_()
            graph.replay()
            assert torch.equal(got, want)


@pytest.mark.parametrize("shape,kernel", [
    ("one", "token"), ("few", "token"), ("chunk", "tile"), ("mixed", "tile"), ("mixed_many", "token"), ("odd_page", "simple"),
    ("token_page", "token")])
def test_kernels_are_the_ones_meant(lib, cuda, shape, kernel):
    for dtype in ("f16", "bf16"):
        _call(lib, _make(65, dtype, *SHAPES[shape]), cuda)
        assert lib.last_kernel() == f"paged_{kernel}_kernel"


def test_same_call_same_bits(lib, cuda):
    for shape in ("token_long", "mixed", "chunk", "mixed_many"):
        a = _make(64, "bf16", *SHAPES[shape])
        want = _call(lib, a, cuda)
        for _ in range(5):
            assert torch.equal(_call(lib, a, cuda), want)


def test_short_way_and_ctypes_agree(lib, cuda, monkeypatch):
    """Calls through csrc/binding.cpp and through ctypes: the same results, refusals and streams."""
    assert lib._short_way()
    a = _make(70, "bf16", *SHAPES["mixed"], lead=1, behind=2)
    b = _append_case(71, "f16", *APPENDS["odd_heads"], norm=True, positions=True)
    for name in ("attention", "append", "keep"):
        results = []
        for short in (lib._short_way(), False):
            monkeypatch.setattr(lib, "_short", short)
            if not short:
                monkeypatch.setattr(lib, "_short_way", lambda: False)
            if name == "attention":
                out = torch.zeros_like(a["q"]).to(cuda)
                assert _call(lib, a, cuda, out=out) is out
                results.append([out])
                with pytest.raises(lib.RopeError):
                    _call(lib, dict(a, window=-1), cuda)
                with pytest.raises(ValueError):
                    _call(lib, a, cuda, workspace=torch.zeros(64, device=cuda))
                with pytest.raises(ValueError):
                    _call(lib, dict(a, q=a["q"].t()), cuda)
            elif name == "append":
                k, v = b["k"].to(cuda), b["v"].to(cuda)
                results.append([_append(lib, b, cuda, k, v), k, v])
                with pytest.raises(lib.RopeError):
                    _append(lib, dict(b, inter=3), cuda, k, v)
                with pytest.raises(ValueError):
                    _append(lib, b, cuda, k.float(), v)
            else:
                g = torch.Generator().manual_seed(2)
                k, v = (torch.randn((6, 2, 16, 64), generator=g).half().to(cuda) for _ in range(2))
                _keep(lib, cuda, k, v, [[0, 3], [5, 1]], [4, 10], [[1, 5], [0, 2, 9]])
                results.append([k, v])
                with pytest.raises(ValueError):
                    _keep(lib, cuda, k, v.float(), [[0, 3], [5, 1]], [4, 10], [[1, 5], [0, 2, 9]])
            monkeypatch.undo()
        for x, y in zip(*results):
            assert torch.equal(x, y)
