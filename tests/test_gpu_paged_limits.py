"""The paged-cache operators where what a call allows ends: starts outside the tokens, rows below 0, bounds above the
tokens, queries of nobody, pages of one tensor, heads that no other operator takes."""

import numpy as np
import pytest
import torch

import paged_util as pu
from test_gpu_paged import MASKS, T, _append, _append_case, _call, _check, _i32, _keep, _make, _want
from test_gpu_paged_edges import _tokens, _unaligned

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# query_starts outside [0, tokens]: they count as clipped, for the append as for attention
# --------------------------------------------------------------------------

RAW, CLIPPED = [-3, 5, 5, 60], [0, 5, 5, 38]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H,norm", [(64, False), (64, True), (38, False), (38, True)])
def test_append_clips_starts(lib, cuda, dtype, H, norm):
    """Both append kernels (heads of 38 are the unaligned one's): rows, rotation and status of the clipped starts."""
    a = _append_case(80, dtype, 8, 2, H, 16, [7, 3, 20], [5, 0, 33], norm=norm)
    results = []
    for starts in (CLIPPED, RAW):
        k, v, status = a["k"].to(cuda), a["v"].to(cuda), torch.zeros(1, dtype=torch.int32, device=cuda)
        q = _append(lib, dict(a, starts=starts), cuda, k, v, status=status)
        results.append((q, k, v))
        assert int(status) == 0, starts
    for x, y in zip(*results):
        assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("new", [[5, 0, 33], [5, 0, 4], [40, 0, 50]])
def test_append_and_attention_clip_alike(lib, cuda, dtype, new):
    """What attention pairs with a token is what the append stored for it, and no sequence is flagged as too long."""
    Nq, Nkv, H, ps, past = 8, 2, 64, 16, [7, 3, 20]
    a = _append_case(81, dtype, Nq, Nkv, H, ps, past, new)
    tokens, most = sum(new), max(new)
    starts = [-3, new[0], new[0], tokens + 9]
    k, v = a["k"].to(cuda), a["v"].to(cuda)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    q = _append(lib, dict(a, starts=starts), cuda, k, v, status=status)
    b = dict(Nq=Nq, q=q, k=k, v=v, table=a["table"], past=past, starts=starts, cap=0.0, window=0, slopes=None, masks=None, most=most)
    got = _call(lib, b, cuda, status=status)
    assert int(status) == 0
    k2, v2 = a["k"].to(cuda), a["v"].to(cuda)
    q2 = _append(lib, a, cuda, k2, v2)
    want, bound, owned = _want(dict(b, q=q2, k=k2, v=v2, starts=a["starts"]), cuda)
    assert owned.all()
    pu.close(got, want, bound)


# --------------------------------------------------------------------------
# trees whose first rows lie below 0
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("new", [[1, 1], [4, 2], [16, 2], [20, 9], [64, 3]])
@pytest.mark.parametrize("below", [-1, -3, -19, -63])
def test_trees_below_row_zero(lib, cuda, dtype, new, below):
    """A draft at a row below 0 sees what its word says: key j, from 0 on, if bit j - past is set."""
    rng = np.random.default_rng(90)
    for cap in (0.0, 5.0):
        a = _make(91, dtype, 8, 2, 64, 16, [60, 10], new, tree=True, cap=cap)
        a["past"] = [below, 10]
        a["table"][0] = rng.permutation(a["k"].shape[0])[:len(a["table"][0])].tolist()
        a["masks"] = [int(x) for x in rng.integers(-2 ** 63, 2 ** 63 - 1, sum(new))]
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        got = _call(lib, a, cuda, status=status)
        want, bound, owned = _want(a, cuda)
        assert owned.all() and int(status) == 4
        pu.close(got, want, bound, str(cap))


# --------------------------------------------------------------------------
# max_query_len as a bound of its own
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("short", [True, False])
def test_a_bound_above_the_tokens(lib, cuda, dtype, short, monkeypatch):
    """A server's fixed bound, in a step with fewer tokens: the call with as many as there are."""
    if not short:
        monkeypatch.setattr(lib, "_short", False)
        monkeypatch.setattr(lib, "_short_way", lambda: False)
    for new, tree in (([60], True), ([3, 1], True), ([1, 1, 1], False), ([70, 1], False), ([0, 0], False)):
        a = _make(92, dtype, 8, 2, 64, 16, [100 + i for i in range(len(new))], new, tree=tree, behind=0)
        want = _call(lib, a, cuda, max_query_len=sum(new))
        for most in (64, 100, 8192, 2 ** 40):
            if most >= sum(new):
                status = torch.zeros(1, dtype=torch.int32, device=cuda)
                assert torch.equal(_call(lib, a, cuda, max_query_len=most, status=status), want), most
                assert int(status) == 0
        if sum(new):
            exact, bound, _ = _want(a, cuda)
            pu.close(want, exact, bound)


# --------------------------------------------------------------------------
# tokens of nobody
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("heads", [(8, 2, 128), (8, 2, 64), (4, 2, 256), (12, 2, 64)])
@pytest.mark.parametrize("masks", ["plain", "cap", "alibi", "window"])
def test_queries_of_nobody_change_no_bit(lib, cuda, dtype, heads, masks):
    """What lies in Q behind the last sequence and before the first (the padding of a captured step): zeros, large
    numbers, infinities and NaN give the sequences the same bits."""
    Nq, Nkv, H = heads
    for new in ([61, 3], [90, 33], [17, 200]):
        a = _make(93, dtype, Nq, Nkv, H, 16, [300, 777], new, lead=2, behind=70, **MASKS[masks])
        lo, hi = a["starts"][0], a["starts"][-1]
        a["q"][:lo], a["q"][hi:] = 0.0, 0.0
        want = _check(lib, a, cuda, str(new))[lo:hi]
        for bad in (60000.0, float("inf"), float("nan")):
            a["q"][:lo], a["q"][hi:] = bad, bad
            assert torch.equal(_call(lib, a, cuda)[lo:hi], want), (new, bad)
        a["q"][hi:] = (torch.randn((70, Nq * H), generator=torch.Generator().manual_seed(1)) * 300).to(a["q"].dtype)
        assert torch.equal(_call(lib, a, cuda)[lo:hi], want), new


# --------------------------------------------------------------------------
# keep
# --------------------------------------------------------------------------

@pytest.mark.parametrize("bad", [-1, 10 ** 7])
@pytest.mark.parametrize("path,spoiled", [([0, 2, 17], 0), ([0], 0), ([0, 1, 2, 3], 0), ([0, 1, 17], 1), ([1, 17], 1)])
def test_keep_looks_at_rows_that_stay(lib, cuda, path, spoiled, bad):
    """A kept row that has its place already counts like the others: its page has to be there."""
    ps, past = 16, [20, 31]
    table, pages = pu.table_for(np.random.default_rng(94), [90, 90], ps)
    table[1][(31 + path[0]) // ps if spoiled == 0 else (31 + path[-1]) // ps] = bad
    k, v = (torch.randn((pages, 2, ps, 64), device=cuda, dtype=torch.float16) for _ in range(2))
    want = [x.clone() for x in (k, v)]
    for x, y in zip((k, v), want):
        y[table[0][21 // ps], :, 21 % ps] = x[table[0][25 // ps], :, 25 % ps]
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    _keep(lib, cuda, k, v, table, past, [[0, 5], path], status=status)
    assert int(status) == 4
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


def test_keep_of_nothing_is_not_flagged(lib, cuda):
    """No row is kept of a sequence whose length is not one, and whose pages are not there: nothing to flag."""
    k, v = (torch.randn((4, 2, 16, 64), device=cuda, dtype=torch.float16) for _ in range(2))
    want = [x.clone() for x in (k, v)]
    for past in (-1, -2 ** 31, 2 ** 31 - 1, 500):
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        _keep(lib, cuda, k, v, [[-1, -1], [0, 1]], [past, 3], [[], []], width=2, status=status)
        assert int(status) == 0, past
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("H", [64, 19])
def test_keep_and_append_in_pages_of_one_tensor(lib, cuda, dtype, H):
    """K and V side by side in each page, for what writes pages as for what reads them."""
    a = _append_case(95, dtype, 8, 2, H - H % 2, 16, [7, 3, 20], [25, 1, 33])
    k, v = a["k"].to(cuda), a["v"].to(cuda)
    both = torch.stack([k, v], 1).contiguous()
    results = []
    for x, y in ((k, v), (both[:, 0], both[:, 1])):
        results.append(_append(lib, a, cuda, x, y))
        status = torch.zeros(1, dtype=torch.int32, device=cuda)
        _keep(lib, cuda, x, y, a["table"], a["past"], [[1, 4, 24], [0], [30, 32]], status=status)
        assert int(status) == 0
    assert torch.equal(*results) and torch.equal(both[:, 0], k) and torch.equal(both[:, 1], v)
    if H % 2:
        x, y = (torch.randn((5, 2, 16, H), device=cuda).to(k.dtype) for _ in range(2))
        both = torch.stack([x, y], 1).contiguous()
        for p, q in ((x, y), (both[:, 0], both[:, 1])):
            _keep(lib, cuda, p, q, [[3, 1, 4]], [13], [[2, 5, 30]])
        assert torch.equal(both[:, 0], x) and torch.equal(both[:, 1], y)


def test_keep_says_what_is_wrong(lib, cuda):
    k, v = (torch.zeros((5, 2, 16, 64), device=cuda) for _ in range(2))
    both = torch.zeros((5, 2, 2, 16, 64), device=cuda)
    for x, y, said in ((both[:, 0], v, "same stride"), (k, v.half(), "v_pages"), (k.transpose(1, 2), v.transpose(1, 2), "k_pages"),
                       (k.cpu(), v, "k_pages"), (k[0], v[0], "k_pages")):
        with pytest.raises(ValueError, match=said):
            lib.kv_keep_paged(x, y, _i32([[3, 1, 4]], cuda), _i32([13], cuda), _i32([[2, 5, 30]], cuda), _i32([3], cuda))


# --------------------------------------------------------------------------
# QK-Norm where no other operator has the bits to compare with
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,H,rd,inter,unaligned", [
    ("f32", 256, 0, 0, False), ("f32", 256, 64, 1, False), ("f32", 140, 0, 0, False), ("f32", 256, 0, 0, True), ("f16", 96, 0, 0, True),
    ("bf16", 96, 0, 1, True), ("f16", 96, 16, 0, False), ("bf16", 256, 0, 0, True), ("f16", 512, 0, 0, False), ("f16", 38, 0, 0, False)])
def test_append_norm_by_definition(lib, cuda, dtype, H, rd, inter, unaligned):
    """z = T(w T(x r)), r = 1 / sqrt(mean x^2 + eps), then the rotation, in 64 bits: heads of more than 32 units, with
    lanes that take several, and 16-bit heads in loads of one element."""
    Nq, Nkv, ps, past, new = 6, 2, 16, [7, 100], [33, 1]
    a = _append_case(96, dtype, Nq, Nkv, H, ps, past, new, norm=True, inter=inter, rd=rd)
    t = a["q"].dtype
    k, v = a["k"].to(cuda), a["v"].to(cuda)
    q = a["q"].to(cuda)
    if unaligned:
        q = _unaligned(q)
    status = torch.zeros(1, dtype=torch.int32, device=cuda)
    got = _append(lib, dict(a, q=q), cuda, k, v, status=status)
    assert int(status) == 0
    b, s = _tokens(a)
    row = torch.tensor(past)[b] + s
    x = a["q"].double().view(-1, Nq + 2 * Nkv, H)
    w = torch.cat([a["qw"].double().expand(Nq, H), a["kw"].double().expand(Nkv, H)])
    z = x[:, :Nq + Nkv] / (x[:, :Nq + Nkv].square().mean(-1, keepdim=True) + 1e-6).sqrt() * w
    half = (rd or H) // 2
    c, sn = a["cos"].double()[row][:, None], a["sin"].double()[row][:, None]
    if inter:
        one, two = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    else:
        one, two = slice(0, half), slice(half, 2 * half)
    y, size = z.clone(), z.abs()
    y[..., one] = z[..., one] * c - z[..., two] * sn
    y[..., two] = z[..., two] * c + z[..., one] * sn
    size[..., one] = (z[..., one] * c).abs() + (z[..., two] * sn).abs()
    size[..., two] = (z[..., two] * c).abs() + (z[..., one] * sn).abs()
    # Three roundings to T of half a step each (x r, w times that, the result, whose size is at most `size`); in 32 bits
    # the squares' sum of H terms (H 2^-24, half of that in r), the mean, root and quotient (4 2^-24) and the
    # rotation (3 2^-24); 2 % for their products. Below float16's normal numbers a rounding is off by 2^-25 instead, which w
    # (below 1.5) and the coefficients (below 6) carry on to less than 2^-20.
    half_step = torch.finfo(t).eps / 2
    most = 1.02 * (3 * half_step + (H / 2 + 7) * 2.0 ** -24) * size + (2.0 ** -20 if t == torch.float16 else 0.0)
    assert a["cos"].abs().max() < 6 and a["sin"].abs().max() < 6
    assert ((got.cpu().double().view(-1, Nq, H) - y[:, :Nq]).abs() <= most[:, :Nq]).all()
    page = torch.tensor([a["table"][int(i)][int(r) // ps] for i, r in zip(b, row)])
    assert ((k.cpu().double()[page, :, row % ps] - y[:, Nq:]).abs() <= most[:, Nq:]).all()
    assert torch.equal(v.cpu()[page, :, row % ps], a["q"].view(-1, Nq + 2 * Nkv, H)[:, Nq + Nkv:])


# --------------------------------------------------------------------------
# both kernels of a mixed batch at a time
# --------------------------------------------------------------------------

@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_mixed_batches_in_a_chain(lib, cuda, cap):
    """Append, attention, keep and append again with nothing between them, in batches whose attention is two kernels at a
    time, the second of which does not wait for what came before: the bits of the same calls with waits between them."""
    Nq, Nkv, H, ps, B = 8, 2, 128, 16, 130
    b = _append_case(97, "bf16", Nq, Nkv, H, ps, [11 * i % 300 for i in range(B)], [1] * (B - 2) + [200, 2])
    starts, past, table = (_i32(b[n], cuda) for n in ("starts", "past", "table"))
    q, cos, sin = (b[n].to(cuda) for n in ("q", "cos", "sin"))
    kept, lens = _i32([[0]] * (B - 2) + [[5], [1]], cuda), _i32([1] * B, cuda)
    calls = dict(num_heads=Nq, query_starts=starts, max_query_len=200, softcap=cap)

    pages = [b[n].to(cuda) for n in ("k", "v")]

    def step(wait):
        k, v = (x.clone() for x in pages)
        outs = []
        for turn in range(3):
            qo = lib.rope_apply_qkv_paged(q + turn, cos, sin, num_heads=Nq, kv_num_heads=Nkv, k_pages=k, v_pages=v, page_table=table,
                                          past_seq_lens=past, query_starts=starts)
            wait()
            outs.append(lib.kv_attention_paged(qo, k, v, table, past, **calls))
            wait()
            lib.kv_keep_paged(k, v, table, past, kept, lens)
            wait()
            outs.append(lib.kv_attention_paged(qo, k, v, table, past, **calls))
            wait()
        return [*outs, k, v]

    want = step(torch.cuda.synchronize)
    assert lib.last_kernel() == "paged_token_kernel"
    for _ in range(5):
        for x, y in zip(step(lambda: None), want):
            assert torch.equal(x, y)
    assert lib.last_kernel() == "paged_token_kernel"
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(lambda: None)
    for _ in range(3):
        for x in got[:6]:
            x.zero_()
        graph.replay()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_mixed_batches_replayed_with_other_lengths(lib, cuda, dtype):
    """One captured call for a mixed batch; the shares of both kernels follow the lengths of each replay."""
    Nq, Nkv, H, ps, B, width, most = 8, 2, 128, 16, 120, 40, 300
    tokens = 700
    steps = [([0] * B, [1] * B), ([7 * b % 300 for b in range(B)], [1] * (B - 1) + [300]), ([5 * b for b in range(B)], [2, 0] * 60),
             ([17] * B, [0] * B), ([3 * b for b in range(B)], [200, 300] + [1] * 60 + [0] * (B - 62)), ([630] + [4] * (B - 1), [5] * B)]
    q = torch.zeros((tokens, Nq * H), dtype=T[dtype], device=cuda)
    k, v = (torch.zeros((B * width, Nkv, ps, H), dtype=T[dtype], device=cuda) for _ in range(2))
    table, past, starts = torch.zeros((B, width), dtype=torch.int32, device=cuda), _i32([0] * B, cuda), _i32([0] * (B + 1), cuda)
    out = torch.zeros_like(q)

    def run():
        lib.kv_attention_paged(q, k, v, table, past, num_heads=Nq, query_starts=starts, max_query_len=most, out=out)

    run()
    assert lib.last_kernel() == "paged_token_kernel"
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i, (p, n) in enumerate(steps):
        a = _make(98 + i, dtype, Nq, Nkv, H, ps, p, n, behind=tokens - sum(n))
        pages = a["k"].shape[0]
        q.copy_(a["q"])
        k.fill_(float("nan"))[:pages] = a["k"].to(cuda)
        v.fill_(float("nan"))[:pages] = a["v"].to(cuda)
        table.copy_(_i32([row + [-7] * (width - len(row)) for row in a["table"]], cuda))
        past.copy_(_i32(p, cuda))
        starts.copy_(_i32(a["starts"], cuda))
        out.fill_(7.0)
        graph.replay()
        want, bound, owned = _want(a, cuda)
        pu.close(out[owned], want[owned], bound[owned], str(i))
        assert torch.equal(out[~owned], torch.full_like(out[~owned], 7.0)), i
