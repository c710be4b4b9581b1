"""The cache operators on the GPU where the choice of kernel, the dealing of work and the ends of the
value ranges matter: many sequences, ragged lengths, far documents, wide groups, extreme ids and lengths."""

import numpy as np
import pytest
import torch

import kv_util as ku
from test_gpu_kv import SHAPES, _call, _check, _make, _want

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape", ["token", "few", "chunk", "chunk_wide", "scalar"])
@pytest.mark.parametrize("scale", [0.0, -0.3, 0.02])
def test_scales_of_the_scores(lib, cuda, fp8, shape, scale):
    """No scale, a negative one (the largest product is then the smallest score) and a small one."""
    B, S, Nq, Nkv, H, L, past = SHAPES[shape]
    for extra in ({}, dict(cap=4.0), dict(alibi=True), dict(cap=4.0, alibi=True)):
        a = _make(31, "f16", B, S, Nq, Nkv, H, L, past, fp8, **extra)
        _check(lib, a, cuda, str(extra), scale=scale)


@pytest.mark.parametrize("fp8", [False, True])
def test_more_sequences_than_are_dealt(lib, cuda, fp8):
    rng = np.random.default_rng(5)
    past = rng.integers(0, 90, 1100).tolist()
    past[7], past[1099] = -1, 89
    a = _make(32, "bf16", 1100, 1, 2, 1, 32, 90, past, fp8)
    got = _check(lib, a, cuda)
    assert lib.last_kernel() == "kv_token_kernel" and not got[7].any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B, Nkv, S", [(300, 2, 1), (61, 1, 2), (5, 3, 4), (700, 3, 1)])
def test_ragged_sequences(lib, cuda, fp8, B, Nkv, S):
    """Lengths from nothing to the whole cache, dealt in units of keys that end anywhere in a sequence; the
    last size has so many sequences that each goes to a CTA of its own."""
    rng = np.random.default_rng(B)
    L = 700
    past = np.where(rng.random(B) < 0.3, rng.integers(-S, 2, B), rng.integers(0, L - S + 1, B))
    past[0], past[-1] = L - S, 0
    a = _make(33, "f16", B, S, 4 * Nkv, Nkv, 64, L, past.tolist(), fp8, cap=float(rng.choice([0.0, 9.0])))
    first = _check(lib, a, cuda)
    for _ in range(3):
        assert torch.equal(_call(lib, a, cuda), first)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("S, Nq, Nkv", [(1, 160, 1), (3, 129, 1), (2, 66, 2), (19, 13, 1)])
def test_wide_groups(lib, cuda, fp8, S, Nq, Nkv):
    """Rows of one token that span row tiles; groups that do not divide them."""
    for extra in ({}, dict(alibi=True, docs=3), dict(prefix=250, cap=7.0)):
        a = _make(34, "bf16", 2, S, Nq, Nkv, 64, 400, [0, 400 - S], fp8, **extra)
        _check(lib, a, cuda, str(extra))
        assert lib.last_kernel() == "kv_tile_kernel"


@pytest.mark.parametrize("S, L", [(5, 4200), (12, 8300)])
def test_drafts_over_many_codes(lib, cuda, S, L):
    """More than 16 rows that stay with the kernel for few: several row tiles of a head, dealt out."""
    rng = np.random.default_rng(S)
    past = rng.integers(0, L - S + 1, 8)
    past[0], past[5] = L - S, 0
    for dtype, extra in (("bf16", {}), ("f16", dict(cap=8.0, alibi=True, prefix=700))):
        a = _make(42, dtype, 8, S, 32, 8, 64, L, past.tolist(), True, **extra)
        _check(lib, a, cuda, dtype)
        assert lib.last_kernel() == "kv_token_kernel"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B, S, Nq, Nkv, H, L", [(1, 1, 8, 8, 128, 4096), (2, 9, 12, 2, 64, 1000), (3, 4, 16, 1, 96, 130),
                                                 (1, 16, 4, 2, 256, 300), (1, 1, 16, 1, 128, 65)])
def test_clusters(lib, cuda, fp8, B, S, Nq, Nkv, H, L):
    """Few problems, each split over a cluster: shares of no unit, of one, of many; rows of several tiles."""
    for past in (0, 1, 63, 64, 100, L - S):
        past = min(past, L - S)
        for extra in ({}, dict(cap=6.0, docs=3), dict(alibi=True, prefix=50)):
            a = _make(43, "bf16", B, S, Nq, Nkv, H, L, [past] * (B - 1) + [0], fp8, **extra)
            first = _check(lib, a, cuda, f"{past} {extra}")
            assert lib.last_kernel() == "kv_token_kernel"
            assert torch.equal(_call(lib, a, cuda, workspace=torch.empty(0, dtype=torch.uint8, device=cuda)), first)


@pytest.mark.parametrize("fp8, S", [(False, 24), (True, 24), (True, 72)])
def test_documents_of_a_long_row(lib, cuda, fp8, S):
    """More key tiles than a CTA lists documents of (4096 of 128 keys), with a workspace for splits and without."""
    L = 4096 * 128 + 3000
    a = _make(35, "f16", 1, S, 1, 1, 16, L, [L - S - 5], fp8)
    j = np.arange(L)
    ids = (j // 1000) % 40
    ids[-40:] = np.where(np.arange(40) % 3 == 0, 5, 17)  # rows of two documents
    a["docs"] = torch.from_numpy(ids.astype(np.int32))[None]
    want, bound = _want(a, cuda)
    for room in (None, 16):
        ws = None if room is None else torch.empty(room, dtype=torch.uint8, device=cuda)
        got = _call(lib, a, cuda, workspace=ws)
        assert lib.last_kernel() == ("kv_token_kernel" if fp8 and S == 24 else "kv_tile_kernel")
        ku.close(got, want, bound, str(room))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("S", [1, 5, 60])
def test_extreme_numbers(lib, cuda, fp8, S):
    """Document ids, prefix lengths and past lengths at the ends of their type."""
    lo, hi = -2 ** 31, 2 ** 31 - 1
    L = 140
    for dtype in ("f32", "f16"):
        a = _make(36, dtype, 4, S, 8, 2, 64, L, [L - S, 70, 70, 3], fp8, prefix=4)
        docs = np.zeros((4, L), np.int32)
        docs[0, 60:], docs[1, 72:], docs[2, ::2], docs[3] = hi, lo, hi, lo
        docs[2, 1::2] = lo
        a["docs"] = torch.from_numpy(docs)
        a["prefix"] = torch.tensor([hi, lo, 100, -1], dtype=torch.int32)
        _check(lib, a, cuda)
        b = _make(37, dtype, 4, S, 8, 2, 64, L, [lo, hi, hi - S + 1, -S], fp8)
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        got = _call(lib, b, cuda, status=status)
        assert int(status) == 4
        assert not got[0].any() and not got[3].any()  # behind the end of a past length of 2^31 - 1 lies the whole cache
        b["past"] = torch.tensor([L, L, L, L], dtype=torch.int32)  # a row that far on sees all of it too
        _check(lib, b, cuda)
        for n in (1, 2):
            far = _call(lib, dict(b, past=torch.full((4,), hi, dtype=torch.int32)), cuda)
            whole = _call(lib, b, cuda)
            assert torch.equal(far[n], whole[n])


@pytest.mark.parametrize("shape", ["token", "few", "chunk", "scalar"])
def test_codes_as_bytes_and_as_floats(lib, cuda, shape):
    B, S, Nq, Nkv, H, L, past = SHAPES[shape]
    a = _make(38, "bf16", B, S, Nq, Nkv, H, L, past, True)
    one = _call(lib, a, cuda)
    f8 = {n: a[n].view(torch.float8_e4m3fn) for n in ("k", "v")}
    assert a["k"].dtype == torch.uint8 and torch.equal(one, _call(lib, dict(a, **f8), cuda))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("shape, kernel", [("token", "kv_token_kernel"), ("few_group", "kv_token_kernel"),
                                           ("chunk_mha", "kv_tile_kernel"), ("prompt", "kv_tile_kernel"),
                                           ("scalar", "kv_simple_kernel")])
def test_kernels_and_the_simt_variant(lib, cuda, fp8, shape, kernel):
    """Which kernel a call takes, and that the plain one agrees."""
    B, S, Nq, Nkv, H, L, past = SHAPES[shape]
    a = _make(39, "f16", B, S, Nq, Nkv, H, L, past, fp8, cap=15.0, docs=2)
    _check(lib, a, cuda)
    assert lib.last_kernel() == kernel
    with lib.variant("simt"):
        _check(lib, a, cuda)
        assert lib.last_kernel() == "kv_simple_kernel"
    _check(lib, a, cuda)
    assert lib.last_kernel() == kernel


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("S", [1, 33])
def test_no_rows(lib, cuda, fp8, S):
    """No sequences or no tokens: nothing is launched, nothing is written."""
    a = _make(41, "f16", 2, S, 4, 2, 64, 50, [3, 4], fp8)
    for cut in ("batch", "tokens"):
        c = dict(a)
        if cut == "batch":
            for n in ("q", "k", "v", "past", "ks", "vs"):
                if n in c:
                    c[n] = c[n][:0]
        else:
            c["q"] = c["q"][:, :0]
        got = _call(lib, c, cuda)
        assert got.shape == c["q"].shape


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_a_captured_step_that_moves_on(lib, cuda, dtype):
    """One captured decode step (append, attention, the lengths advanced) replayed token after token, against
    the same calls made one by one."""
    t = {"f16": torch.float16, "bf16": torch.bfloat16}[dtype]
    B, Nq, N, H, L = 3, 8, 2, 128, 300
    g = torch.Generator().manual_seed(6)
    angle = torch.arange(L)[:, None] * 10000.0 ** (-torch.arange(0, H, 2) / H)
    cos, sin = angle.cos().to(t).to(cuda), angle.sin().to(t).to(cuda)
    xs = torch.randn((12, B, 1, (Nq + 2 * N) * H), generator=g).to(t).to(cuda)
    outs = []
    for captured in (False, True):
        k8, v8, ks, vs = lib.kv_cache_fp8(B, N, L, H, cuda)
        past = torch.tensor([0, 15, 250], dtype=torch.int32, device=cuda)
        x = xs[0].clone()

        def step():
            q = lib.rope_apply_qkv_fp8(x, cos, sin, num_heads=Nq, kv_num_heads=N, k_cache=k8, v_cache=v8, k_scale=ks,
                                       v_scale=vs, past_seq_lens=past)
            out = lib.kv_attention_fp8(q, k8, v8, ks, vs, past, num_heads=Nq)
            past.add_(1)
            return out

        if captured:
            step()  # loads the kernels
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = step()
            for c in (k8, v8):
                c.view(torch.uint8).zero_()
            ks.fill_(1.0)  # as kv_cache_fp8 makes them
            vs.fill_(1.0)
            past.copy_(torch.tensor([0, 15, 250]))
        rows = []
        for n in range(len(xs)):
            x.copy_(xs[n])
            if captured:
                graph.replay()
            else:
                out = step()
            rows.append(out.clone())
        outs.append((rows, k8.view(torch.uint8).clone(), v8.view(torch.uint8).clone(), ks.clone(), vs.clone()))
    for one, two in zip(outs[0][0], outs[1][0]):
        assert torch.equal(one, two)
    for one, two in zip(outs[0][1:], outs[1][1:]):
        assert torch.equal(one, two)


@pytest.mark.parametrize("fp8", [False, True])
def test_many_rows_past_32_bits(lib, cuda, fp8):
    """Prompts over caches of more than 2^31 elements, by the kernel for many rows and the plain one."""
    B, N, H, L, S, n = 2, 4, 128, 2200000, 40, 300
    g = torch.Generator().manual_seed(4)
    q = torch.randn((B, S, 8 * H), generator=g).to(torch.bfloat16).to(cuda)
    past = torch.tensor([n - S, 100], dtype=torch.int32, device=cuda)
    x = [torch.randn((B, N, n, H), generator=g) for _ in range(2)]
    if fp8:
        kc, vc, ks, vs = lib.kv_cache_fp8(B, N, L, H, cuda)
        for c, y, s in ((kc, x[0], ks), (vc, x[1], vs)):
            c.view(torch.uint8)[:, :, :n] = torch.from_numpy(ku.e4m3(y.numpy() * 100)).to(cuda)
            s.fill_(2.0 ** -7)
        call = lambda: lib.kv_attention_fp8(q, kc, vc, ks, vs, past, num_heads=8)  # noqa: E731
        kd, vd = (torch.from_numpy(ku.values(c[:, :, :304].view(torch.uint8).cpu().numpy(), s[:, :, :19].cpu().numpy())).to(cuda)
                  for c, s in ((kc, ks), (vc, vs)))
    else:
        kc, vc = (torch.empty((B, N, L, H), dtype=torch.bfloat16, device=cuda) for _ in range(2))
        for c, y in ((kc, x[0]), (vc, x[1])):
            c[:, :, :n] = y.to(torch.bfloat16).to(cuda)
        call = lambda: lib.kv_attention(q, kc, vc, past, num_heads=8)  # noqa: E731
        kd, vd = kc[:, :, :n].double(), vc[:, :, :n].double()
    want, bound = ku.attention(q.double(), kd, vd, past.cpu().numpy(), 8, H ** -0.5, weight_eps=2.0 ** -11 if fp8 else 2.0 ** -8)
    ku.close(call(), want, bound)
    assert lib.last_kernel() == "kv_tile_kernel"
    with lib.variant("simt"):
        ku.close(call(), want, bound)
        assert lib.last_kernel() == "kv_simple_kernel"
