"""The cache operators on the GPU against their 64-bit definitions (kv_util): attention over caches in
the storage type and in 8 bits, the 8-bit append, and runs of them together."""

import numpy as np
import pytest
import torch

import kv_util as ku

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def _make(seed, dtype, B, S, Nq, Nkv, H, L, past, fp8, cap=0.0, alibi=False, docs=0, prefix=0, qscale=1.0):
    g = torch.Generator().manual_seed(seed)
    t = T[dtype]
    a = {"q": (torch.randn((B, S, Nq * H), generator=g) * qscale).to(t), "past": torch.tensor(past, dtype=torch.int32),
         "num_heads": Nq, "softcap": cap}
    k, v = torch.randn((B, Nkv, L, H), generator=g), torch.randn((B, Nkv, L, H), generator=g)
    if fp8:
        for name, x in (("k", k), ("v", v)):
            # codes of every size, blocks whose scales lie far apart, and values of another magnitude than keys
            a[name] = torch.from_numpy(ku.e4m3((x * 60).numpy()))
            e = torch.randint(-3, 4, (B, Nkv, -(-L // 16)), generator=g).float()
            a[name + "s"] = torch.exp2(e - (6 if name == "k" else 13))
    else:
        a["k"], a["v"] = k.to(t), v.to(t)
    a["slopes"] = torch.exp2(-8.0 * (torch.arange(Nq) + 1.0) / Nq) if alibi else None
    a["docs"] = torch.sort(torch.randint(0, docs, (B, L), generator=g), dim=1).values.to(torch.int32) if docs else None
    a["prefix"] = torch.randint(0, prefix + 1, (B,), generator=g).to(torch.int32) if prefix else None
    return a


def _call(lib, a, dev, **kw):
    c = {n: (x.to(dev) if isinstance(x, torch.Tensor) else x) for n, x in a.items()}
    more = dict(num_heads=c["num_heads"], softcap=c["softcap"], alibi_slopes=c["slopes"], document_ids=c["docs"],
                prefix_lens=c["prefix"], **kw)
    if "ks" in c:
        return lib.kv_attention_fp8(c["q"], c["k"], c["v"], c["ks"], c["vs"], c["past"], **more)
    return lib.kv_attention(c["q"], c["k"], c["v"], c["past"], **more)


def _want(a, dev, scale=None):
    if "ks" in a:
        k = torch.from_numpy(ku.values(a["k"].cpu().numpy(), a["ks"].cpu().numpy()))
        v = torch.from_numpy(ku.values(a["v"].cpu().numpy(), a["vs"].cpu().numpy()))
    else:
        k, v = a["k"].double(), a["v"].double()
    t = a["q"].dtype
    # the weights are held in float32 for float32, else in T, in float16 over 8-bit caches
    eps = 2.0 ** -24 if t == torch.float32 else 2.0 ** -11 if "ks" in a else ku.EPS[t]
    H = k.shape[3]
    return ku.attention(a["q"].double().to(dev), k.to(dev), v.to(dev), a["past"], a["num_heads"],
                        H ** -0.5 if scale is None else scale, a["softcap"],
                        None if a["slopes"] is None else a["slopes"].to(dev),
                        None if a["docs"] is None else a["docs"].cpu().numpy(), a["prefix"], weight_eps=eps)


def _check(lib, a, dev, what="", **kw):
    got = _call(lib, a, dev, **kw)
    want, bound = _want(a, dev, kw.get("scale"))
    ku.close(got, want, bound, what)
    return got


# (B, S, Nq, Nkv, H, L, past): one token to chunks, odd sizes, lengths that end inside a tile, of one, of the whole cache
SHAPES = {
    "one": (1, 1, 4, 1, 64, 1, [0]),
    "token": (3, 1, 8, 2, 128, 300, [0, 17, 299]),
    "token_odd": (5, 1, 7, 1, 96, 131, [0, 15, 16, 127, 130]),
    "token_long": (2, 1, 8, 2, 128, 5000, [4999, 2049]),
    "token_mha": (2, 1, 3, 3, 32, 100, [63, 64]),
    "token_wide": (2, 1, 16, 8, 256, 200, [199, 31]),
    "token_group": (2, 1, 40, 2, 64, 150, [149, 90]),
    "few": (2, 5, 8, 2, 128, 400, [0, 395]),
    "few_group": (2, 3, 21, 3, 64, 260, [128, 257]),
    "chunk": (2, 70, 8, 2, 128, 333, [0, 263]),
    "chunk_mha": (1, 150, 2, 2, 64, 150, [0]),
    "chunk_odd": (2, 131, 6, 2, 80, 500, [7, 369]),
    "chunk_wide": (1, 67, 4, 2, 256, 190, [100]),
    "chunk_group": (1, 40, 28, 4, 128, 290, [250]),
    "prompt": (1, 300, 4, 1, 128, 300, [0]),
    "scalar": (2, 9, 4, 2, 19, 60, [3, 51]),
    "tiny_head": (2, 33, 4, 4, 2, 66, [3, 33]),
}
MASKS = {
    "plain": {}, "cap": dict(cap=5.0, qscale=3.0), "alibi": dict(alibi=True), "docs": dict(docs=4), "prefix": dict(prefix=120),
    "all": dict(cap=20.0, alibi=True, docs=2, prefix=300),
}


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("masks", ["plain", "all"])
def test_attention(lib, cuda, dtype, shape, masks):
    B, S, Nq, Nkv, H, L, past = SHAPES[shape]
    _check(lib, _make(1, dtype, B, S, Nq, Nkv, H, L, past, False, **MASKS[masks]), cuda)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("masks", ["plain", "all"])
def test_attention_fp8(lib, cuda, dtype, shape, masks):
    B, S, Nq, Nkv, H, L, past = SHAPES[shape]
    _check(lib, _make(2, dtype, B, S, Nq, Nkv, H, L, past, True, **MASKS[masks]), cuda)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", ["token", "few", "chunk", "chunk_odd", "chunk_group"])
@pytest.mark.parametrize("masks", ["cap", "alibi", "docs", "prefix"])
def test_each_mask(lib, cuda, fp8, shape, masks):
    B, S, Nq, Nkv, H, L, past = SHAPES[shape]
    for dtype in ("f16", "bf16"):
        _check(lib, _make(3, dtype, B, S, Nq, Nkv, H, L, past, fp8, **MASKS[masks]), cuda, dtype)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_random_shapes(lib, cuda, fp8, dtype):
    rng = np.random.default_rng(11 + fp8)
    for n in range(16):
        Nkv = int(rng.integers(1, 4))
        G = int(rng.integers(1, 9))
        H = int(rng.choice([8, 16, 24, 48, 64, 72, 96, 112, 128, 160, 256]))
        B, S = int(rng.integers(1, 4)), int(rng.choice([1, 2, 4, 16, 17, 50, 129]))
        L = int(rng.integers(S, 700))
        past = rng.integers(0, L - S + 1, B).tolist()
        a = _make(100 + n, dtype, B, S, G * Nkv, Nkv, H, L, past, fp8, cap=float(rng.choice([0, 10.0])),
                  alibi=bool(rng.integers(2)), docs=int(rng.choice([0, 3])), prefix=int(rng.choice([0, 200])))
        _check(lib, a, cuda, str((B, S, G, Nkv, H, L, past)))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", ["token", "token_odd", "few", "chunk", "prompt", "chunk_wide"])
def test_nothing_hidden_is_used(lib, cuda, dtype, fp8, shape):
    """NaN and infinities behind the last row, in other documents and ahead of a query change nothing."""
    B, S, Nq, Nkv, H, L, past = SHAPES[shape]
    L += 40
    a = _make(4, dtype, B, S, Nq, Nkv, H, L, past, fp8)
    a["docs"] = torch.zeros((B, L), dtype=torch.int32)
    for b in range(B):
        a["docs"][b, 1:past[b] // 2] = 9  # holes: rows of another document between and before
        a["docs"][b, past[b] + S - 1:] = 5  # the last token starts a document of its own
    want, bound = _want(a, cuda)
    ku.close(_call(lib, a, cuda), want, bound)
    for b in range(B):
        for name in ("k", "v"):
            x = a[name]
            rows = (a["docs"][b] == 9).nonzero().flatten()
            if fp8:
                bad = torch.tensor([127, 255], dtype=torch.uint8)
            else:
                bad = torch.tensor([float("nan"), float("inf")], dtype=x.dtype)
            x[b, :, past[b] + S:] = bad[0]
            x[b, :, rows[::2]] = bad[0]
            x[b, :, rows[1::2]] = bad[1]
            if S > 1:
                x[b, :, past[b] + S - 1] = bad[int(name == "v")]  # seen by the last token alone
        if fp8:
            a["ks"][b, :, (past[b] + S + 15) // 16:] = float("nan")
            a["vs"][b, :, (past[b] + S + 15) // 16:] = float("inf")
    got = _call(lib, a, cuda)
    keep = S - 1 if S > 1 else 1
    ku.close(got[:, :keep], want[:, :keep], bound[:, :keep])
    if S > 1:
        assert not torch.isfinite(got[:, -1]).any()  # and what is seen is not hidden


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S", [1, 4, 100])
def test_rows_that_see_nothing(lib, cuda, dtype, fp8, S):
    """Negative and too large past lengths: such rows see what the formula says, or give 0; status bit 2."""
    past = [-3, -200, 150, 260, 400]
    for extra in ({}, dict(docs=3), dict(prefix=40)):
        a = _make(5, dtype, 5, S, 8, 2, 64, 256, past, fp8, **extra)
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        got = _check(lib, a, cuda, str(extra), status=status)
        assert int(status) == 4
        assert not got[1].any()
        if not extra:
            assert not got[0, :3].any() and (S < 4 or bool(got[0, 3].any()))
    a = _make(5, dtype, 2, S, 8, 2, 64, 256, [0, 256 - S], fp8)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    _check(lib, a, cuda, status=status)
    assert int(status) == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("S", [1, 20])
def test_scores_far_apart(lib, cuda, dtype, fp8, S):
    """Scores of hundreds: one key outweighs all others; the running maximum moves at nearly every key."""
    a = _make(6, dtype, 2, S, 4, 2, 64, 1500, [1500 - S, 700], fp8)
    ramp = torch.linspace(0.01, 1.0, 1500)
    if fp8:
        e = torch.floor(torch.log2(torch.linspace(0.01, 0.5, a["ks"].shape[2])))
        a["ks"] = torch.exp2(e).expand_as(a["ks"]).contiguous()
    else:
        a["k"] = (a["k"] * ramp[:, None] * 30).to(T[dtype])
    _check(lib, a, cuda, scale=1.0)
    a["q"] = -a["q"]
    _check(lib, a, cuda, scale=-0.5)


@pytest.mark.parametrize("fp8", [False, True])
def test_infinite_scores(lib, cuda, fp8):
    """A NaN in a visible key makes its rows NaN; scores of -inf weigh nothing; only -inf gives 0."""
    for S in (1, 40):
        a = _make(7, "bf16", 1, S, 2, 1, 64, 100, [60 - S], fp8)
        a["q"] = a["q"].abs() + 0.1
        if fp8:
            a["k"][0, 0, 3] = 127
        else:
            a["k"][0, 0, 3] = float("nan")
        assert torch.isnan(_call(lib, a, cuda)).all()
        if not fp8:
            a["k"][0, 0, 3] = float("-inf")
            got = _call(lib, a, cuda)
            b = dict(a, k=a["k"].clone(), docs=torch.zeros((1, 100), dtype=torch.int32))
            b["k"][0, 0, 3] = 0
            b["docs"][0, 3] = 1
            want, bound = _want(b, cuda)
            ku.close(got, want, bound)
            a["k"][:] = float("-inf")
            assert not _call(lib, a, cuda).any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("S", [1, 3, 200])
def test_workspace(lib, cuda, fp8, S):
    """Any workspace gives the result up to rounding; its contents do not matter; nothing outside it is written."""
    a = _make(8, "f16", 1, S, 8, 2, 128, 9000, [9000 - S - 7], fp8)
    want, bound = _want(a, cuda)
    need = lib.kv_attention_workspace(1, S, 8, 2, 128, 9000)
    for room in (0, 100, need // 2, max(0, need - 1), need, need + 1000):
        ws = torch.full((room + 256,), 255, dtype=torch.uint8, device=cuda)
        got = _call(lib, a, cuda, workspace=ws[:room])
        ku.close(got, want, bound, str(room))
        assert (ws[room:] == 255).all()
    first = _call(lib, a, cuda)
    for _ in range(3):
        assert torch.equal(_call(lib, a, cuda), first)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_unaligned(lib, cuda, dtype, fp8):
    """Tensors that start one element into their storage."""
    for S in (1, 40):
        a = _make(9, dtype, 2, S, 4, 2, 64, 100, [0, 60 - S // 2], fp8)
        want, bound = _want(a, cuda)
        c = {}
        for n in ("q", "k", "v"):
            flat = torch.empty(a[n].numel() + 1, dtype=a[n].dtype, device=cuda)
            c[n] = flat[1:].view(a[n].shape)
            c[n].copy_(a[n])
        out = torch.empty(a["q"].numel() + 3, dtype=a["q"].dtype, device=cuda).fill_(7.0)
        got = out[1:-2].view(a["q"].shape)
        _call(lib, dict(a, **c), cuda, out=got)
        ku.close(got, want, bound)
        assert float(out[0]) == 7.0 and (out[-2:] == 7.0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_streams_and_graphs(lib, cuda, fp8):
    """A call on another stream, two at once, and two captured graphs that replay at the same time."""
    cases = [_make(20 + n, "f16", 1, S, 8, 2, 128, 4000, [4000 - S], fp8) for n, S in enumerate((1, 64))]
    cases = [{n: (x.to(cuda) if isinstance(x, torch.Tensor) else x) for n, x in a.items()} for a in cases]
    want = [_call(lib, a, cuda).clone() for a in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[_call(lib, a, cuda, stream=s) for a, s in zip(cases, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for row in got:
        for g, w in zip(row, want):
            assert torch.equal(g, w)
    graphs, outs = [], []
    for a, s in zip(cases, streams):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(_call(lib, a, cuda))
        graphs.append(g)
    for _ in range(10):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)


def test_refusals_of_the_binding(lib, cuda):
    a = _make(1, "f16", 2, 1, 4, 2, 64, 32, [0, 1], False)
    c = {n: (x.to(cuda) if isinstance(x, torch.Tensor) else x) for n, x in a.items()}

    def call(**kw):
        return lib.kv_attention(**{**dict(query=c["q"], k_cache=c["k"], v_cache=c["v"], past_seq_lens=c["past"],
                                          num_heads=4), **kw})

    call()
    for bad in (dict(query=c["q"].float()), dict(query=c["q"][:1]), dict(k_cache=c["k"][..., :32]),
                dict(v_cache=c["v"].transpose(1, 2)), dict(past_seq_lens=c["past"].long()),
                dict(past_seq_lens=c["past"][:1]), dict(num_heads=3), dict(alibi_slopes=torch.ones(3, device=cuda)),
                dict(document_ids=torch.zeros((2, 31), dtype=torch.int32, device=cuda)),
                dict(prefix_lens=torch.zeros(2, dtype=torch.int32)), dict(out=c["q"][:1]),
                dict(workspace=torch.zeros(8, device=cuda))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(lib.RopeError):
        call(softcap=-1.0)
    with pytest.raises(lib.RopeError):
        call(**{n: x.to(torch.int16) for n, x in (("query", c["q"]), ("k_cache", c["k"]), ("v_cache", c["v"]))})


# --------------------------------------------------------------------------
# the 8-bit append
# --------------------------------------------------------------------------

def _append_case(lib, dev, dtype, B, S, Nq, Nkv, H, L, past, rd=0, inter=0, norm=False, packed=True, rows=None, seed=0,
                 positions=False, size=1.0, offset=0, scales=None):
    """One append against what rope_apply_qkv stores, rounded by the definition."""
    g = torch.Generator().manual_seed(seed)
    t = T[dtype]

    def put(x):
        flat = torch.empty(x.numel() + offset, dtype=x.dtype, device=dev)
        flat[offset:].copy_(x.flatten().to(dev))
        return flat[offset:].view(x.shape)

    rows = L if rows is None else rows
    h = (rd or H) // 2
    angle = torch.rand((rows, h), generator=g) * 6.28
    x = (torch.randn((B, S, (Nq + 2 * Nkv) * H), generator=g) * size).to(t)
    cos, sin = put(angle.cos().to(t)), put(angle.sin().to(t))
    pos = torch.randint(-2, rows + 2, (B, S), generator=g).to(dev) if positions else None
    pastd = torch.tensor(past, dtype=torch.int32, device=dev)
    w = [put((torch.rand(H, generator=g) + 0.5).to(t)) for _ in range(2)] if norm else [None, None]
    kw = dict(num_heads=Nq, kv_num_heads=Nkv, past_seq_lens=pastd, interleaved=inter, rotary_embedding_dim=rd,
              q_norm_weight=w[0], k_norm_weight=w[1])
    if packed:
        q = put(x)
    else:
        q = put(x[..., :Nq * H])
        kw.update(key=put(x[..., Nq * H:(Nq + Nkv) * H]), value=put(x[..., (Nq + Nkv) * H:]))
    # the same call over a cache long enough for every row, in the storage type
    shift = max(0, -min(past))
    span = max(past) + S + shift
    kc, vc = (torch.zeros((B, Nkv, span, H), dtype=t, device=dev) for _ in range(2))
    shown = pos if pos is not None else pastd.long()[:, None] + torch.arange(S, device=dev)
    want_status, status = (torch.zeros(1, dtype=torch.int32, device=dev) for _ in range(2))
    q_want, _ = lib.rope_apply_qkv(q, cos, sin, shown.contiguous(), k_cache=kc, v_cache=vc, status=want_status,
                                   **{**kw, "past_seq_lens": pastd + shift})
    new = [torch.stack([c[b, :, past[b] + shift:past[b] + shift + S].transpose(0, 1) for b in range(B)]).double().cpu().numpy()
           for c in (kc, vc)]
    codes = [torch.randint(0, 127, (B, Nkv, L, H), generator=g, dtype=torch.uint8) for _ in range(2)]
    sc = [torch.exp2(torch.randint(-12, 0, (B, Nkv, -(-L // 16)), generator=g).float()) if scales is None else
          torch.full((B, Nkv, -(-L // 16)), scales) for _ in range(2)]
    dcodes, dsc = [c.to(dev).view(torch.float8_e4m3fn) for c in codes], [s.to(dev) for s in sc]
    got_q = lib.rope_apply_qkv_fp8(q, cos, sin, pos, k_cache=dcodes[0], v_cache=dcodes[1], k_scale=dsc[0], v_scale=dsc[1],
                                   status=status, **kw)
    as_int = torch.int32 if t == torch.float32 else torch.int16
    assert torch.equal(got_q.view(as_int), q_want.view(as_int))
    outside = any(p < 0 or p + S > L for p in past)
    assert int(status) == (int(want_status) & 1) | (4 if outside else 0)
    for i in range(2):
        c, s = codes[i].numpy().copy(), sc[i].numpy().copy()
        ku.append(c, s, new[i], past)
        assert np.array_equal(dsc[i].cpu().numpy(), s), "scales"
        assert np.array_equal(dcodes[i].view(torch.uint8).cpu().numpy(), c), "codes"


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("S", [1, 3, 16, 41])
def test_append(lib, cuda, dtype, norm, S):
    for inter, rd, packed, positions in ((0, 0, True, False), (1, 32, False, True), (0, 32, True, True), (1, 0, False, False)):
        _append_case(lib, cuda, dtype, 4, S, 6, 2, 64, 96, [0, 5, 16, 96 - S], rd=rd, inter=inter, norm=norm, packed=packed,
                     positions=positions, rows=90 if positions else None, seed=S)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [(2, 5, 4, 2, 128, 64, [3, 40]), (1, 70, 5, 5, 256, 100, [13]), (3, 2, 3, 1, 32, 33, [0, 31, 14]),
                                   (2, 19, 2, 1, 6, 50, [1, 20]), (2, 4, 2, 2, 20, 30, [7, 13]), (2, 17, 4, 4, 96, 70, [15, 16])])
def test_append_shapes(lib, cuda, dtype, shape):
    _append_case(lib, cuda, dtype, *shape, seed=3)
    _append_case(lib, cuda, dtype, *shape, seed=4, packed=False, inter=1)


@pytest.mark.parametrize("S", [1, 7, 40])
def test_append_outside(lib, cuda, S):
    """Rows before and behind the cache are not stored; a cache length that ends inside a block."""
    _append_case(lib, cuda, "f16", 5, S, 4, 2, 64, 37, [-2, -60, 36, 37, 300], seed=5, rows=400)
    _append_case(lib, cuda, "bf16", 3, S, 4, 2, 64, 37, [0, 10, 30], seed=5, rows=20, offset=1)


@pytest.mark.parametrize("scales", [2.0 ** -30, 2.0 ** 20, 2.0 ** -120])
def test_append_scales(lib, cuda, scales):
    """Older scales far below and far above what the new rows need."""
    _append_case(lib, cuda, "f16", 3, 4, 4, 2, 64, 64, [1, 15, 40], seed=6, scales=scales)
    _append_case(lib, cuda, "f32", 3, 20, 4, 2, 64, 64, [1, 15, 40], seed=7, size=1e30, scales=scales)
    _append_case(lib, cuda, "bf16", 3, 20, 4, 2, 64, 64, [1, 15, 40], seed=7, size=1e-30, scales=scales)
    _append_case(lib, cuda, "bf16", 2, 20, 4, 2, 64, 64, [0, 17], seed=7, size=0.0, scales=scales)


def test_append_special_values(lib, cuda):
    """Infinities are stored as the largest code, NaN as NaN; neither moves the scale."""
    B, S, N, H, L = 1, 5, 1, 64, 32
    x = torch.ones((B, S, 3 * H), dtype=torch.float16)
    x[0, 0, 2 * H], x[0, 1, 2 * H + 1], x[0, 2, 2 * H + 2] = float("inf"), float("-inf"), float("nan")
    kc, vc, ks, vs = lib.kv_cache_fp8(B, N, L, H, cuda)
    one = torch.ones((L, H // 2), dtype=torch.float16, device=cuda)
    lib.rope_apply_qkv_fp8(x.to(cuda), one, torch.zeros_like(one), num_heads=1, kv_num_heads=1, k_cache=kc, v_cache=vc,
                           k_scale=ks, v_scale=vs, past_seq_lens=torch.zeros(1, dtype=torch.int32, device=cuda))
    v = vc.float().cpu()[0, 0]
    assert float(vs[0, 0, 0]) == 2.0 ** -8 and float(ks[0, 0, 0]) == 2.0 ** -8
    assert v[0, 0] == 448 and v[1, 1] == -448 and torch.isnan(v[2, 2]) and v[3, 3] == 256
    assert float(vs[0, 0, 1]) == 1.0 and not vc.float()[0, 0, 5:].any()


def test_append_refusals(lib, cuda):
    a = dict(query=torch.zeros((2, 3, 8 * 64), dtype=torch.float16, device=cuda),
             cos_cache=torch.zeros((9, 32), dtype=torch.float16, device=cuda),
             sin_cache=torch.zeros((9, 32), dtype=torch.float16, device=cuda), num_heads=4, kv_num_heads=2,
             past_seq_lens=torch.zeros(2, dtype=torch.int32, device=cuda))
    kc, vc, ks, vs = lib.kv_cache_fp8(2, 2, 20, 64, cuda)
    a.update(k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs)
    lib.rope_apply_qkv_fp8(**a)
    for bad in (dict(k_cache=kc.float()), dict(v_cache=vc[:, :, :16]), dict(k_scale=ks[..., :1]), dict(v_scale=vs.double()),
                dict(cos_cache=a["cos_cache"][:, :16]), dict(sin_cache=a["sin_cache"].float()),
                dict(past_seq_lens=None), dict(value=a["query"]), dict(query=a["query"][..., :7]),
                dict(position_ids=torch.zeros((2, 3), device=cuda)), dict(kv_num_heads=1)):
        with pytest.raises((ValueError, lib.RopeError)):
            lib.rope_apply_qkv_fp8(**{**a, **bad})
    with pytest.raises(lib.RopeError):
        lib.rope_apply_qkv_fp8(**{**a, "q_norm_weight": torch.ones(64, dtype=torch.float16, device=cuda)})


def test_append_on_another_stream_and_captured(lib, cuda):
    B, S, Nq, N, H, L = 2, 1, 4, 2, 64, 64
    x = torch.randn((B, S, (Nq + 2 * N) * H), device=cuda).half()
    cs = torch.rand((L, H // 2), device=cuda).half()
    past = torch.tensor([4, 20], dtype=torch.int32, device=cuda)
    kw = dict(num_heads=Nq, kv_num_heads=N, past_seq_lens=past)
    names = ("k_cache", "v_cache", "k_scale", "v_scale")
    ref = dict(zip(names, lib.kv_cache_fp8(B, N, L, H, cuda)))
    other = dict(zip(names, lib.kv_cache_fp8(B, N, L, H, cuda)))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=torch.cuda.Stream()):
        qg = lib.rope_apply_qkv_fp8(x, cs, cs, **kw, **other)
    for step in range(30):
        past.copy_(torch.tensor([4 + step, 20 + step]))
        x.copy_(torch.randn_like(x) * (1 + step))
        q = lib.rope_apply_qkv_fp8(x, cs, cs, **kw, **ref)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(q, qg)
    for n in names:
        assert torch.equal(ref[n].view(torch.uint8), other[n].view(torch.uint8))


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_prompt_and_its_next_tokens(lib, cuda, dtype):
    """A prompt in two chunks, then token by token: append and attention over both kinds of caches. The 8-bit
    results are those of the values that the caches stand for, and the others of what rope_apply_qkv stored."""
    t = T[dtype]
    B, Nq, N, H, L = 2, 8, 2, 64, 200
    g = torch.Generator().manual_seed(1)
    angle = torch.arange(L)[:, None] * 10000.0 ** (-torch.arange(0, H, 2) / H)
    cos, sin = angle.cos().to(t).to(cuda), angle.sin().to(t).to(cuda)
    kc, vc = (torch.full((B, N, L, H), float("nan"), dtype=t, device=cuda) for _ in range(2))
    k8, v8, ks, vs = lib.kv_cache_fp8(B, N, L, H, cuda)
    k8.view(torch.uint8).fill_(127)
    past = torch.zeros(B, dtype=torch.int32, device=cuda)
    for S in [40, 77, 1, 1, 1, 6, 1, 1]:
        x = torch.randn((B, S, (Nq + 2 * N) * H), generator=g).to(t).to(cuda)
        kw = dict(num_heads=Nq, kv_num_heads=N, past_seq_lens=past)
        q, _ = lib.rope_apply_qkv(x, cos, sin, None, k_cache=kc, v_cache=vc, **kw)
        q8 = lib.rope_apply_qkv_fp8(x, cos, sin, None, k_cache=k8, v_cache=v8, k_scale=ks, v_scale=vs, **kw)
        assert torch.equal(q, q8)
        out = lib.kv_attention(q, kc, vc, past, num_heads=Nq, softcap=30.0)
        out8 = lib.kv_attention_fp8(q, k8, v8, ks, vs, past, num_heads=Nq, softcap=30.0)
        hp = past.cpu().numpy()
        n = int(hp.max()) + S
        want, bound = ku.attention(q.double(), kc[:, :, :n].double(), vc[:, :, :n].double(), hp, Nq, H ** -0.5, 30.0,
                                   weight_eps=ku.EPS[t])
        ku.close(out, want, bound)
        vals = [torch.from_numpy(ku.values(c.view(torch.uint8).cpu().numpy(), s.cpu().numpy())).to(cuda)
                for c, s in ((k8, ks), (v8, vs))]
        want, bound = ku.attention(q.double(), *vals, hp, Nq, H ** -0.5, 30.0, weight_eps=2.0 ** -11)
        ku.close(out8, want, bound)
        past += S


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(lib, cuda, fp8):
    """Caches of more than 2^31 elements: the last sequence's head lies behind them."""
    B, N, H, L, n = 2, 4, 128, 2200000, 3001
    past = torch.tensor([100, 3000], dtype=torch.int32, device=cuda)
    t = torch.bfloat16
    g = torch.Generator().manual_seed(3)
    x = torch.randn((B, 1, (8 + 2 * N) * H), generator=g).to(t).to(cuda)
    cs = [torch.ones((n, H // 2), dtype=t, device=cuda), torch.zeros((n, H // 2), dtype=t, device=cuda)]
    k, v = torch.randn((B, N, n, H), generator=g), torch.randn((B, N, n, H), generator=g)
    kw = dict(num_heads=8, kv_num_heads=N, past_seq_lens=past)
    if fp8:
        kc, vc, ks, vs = lib.kv_cache_fp8(B, N, L, H, cuda)
        kc.view(torch.uint8)[:, :, :n] = torch.from_numpy(ku.e4m3(k.numpy() * 100)).to(cuda)
        vc.view(torch.uint8)[:, :, :n] = torch.from_numpy(ku.e4m3(v.numpy() * 100)).to(cuda)
        ks.fill_(2.0 ** -7)
        vs.fill_(2.0 ** -7)
        q = lib.rope_apply_qkv_fp8(x, *cs, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, **kw)
        got = lib.kv_attention_fp8(q, kc, vc, ks, vs, past, num_heads=8)
        kd, vd = (torch.from_numpy(ku.values(c[:, :, :3008].view(torch.uint8).cpu().numpy(), s[:, :, :188].cpu().numpy())).to(cuda)
                  for c, s in ((kc, ks), (vc, vs)))
    else:
        kc, vc = torch.empty((B, N, L, H), dtype=t, device=cuda), torch.empty((B, N, L, H), dtype=t, device=cuda)
        kc[:, :, :n], vc[:, :, :n] = k.to(t).to(cuda), v.to(t).to(cuda)
        q, _ = lib.rope_apply_qkv(x, *cs, None, k_cache=kc, v_cache=vc, **kw)
        got = lib.kv_attention(q, kc, vc, past, num_heads=8)
        kd, vd = kc[:, :, :n].double(), vc[:, :, :n].double()
    want, bound = ku.attention(q.double(), kd, vd, past.cpu().numpy(), 8, H ** -0.5, weight_eps=2.0 ** -11 if fp8 else 2.0 ** -8)
    ku.close(got, want, bound)
