"""The paged-cache operators at their ends: many sequences, odd groups and alignments, far pages, shared pages, pages
that end anywhere in a tile, lengths that change between replays, two calls at a time."""

import numpy as np
import pytest
import torch

import paged_util as pu
from test_gpu_paged import APPENDS, SHAPES, T, _append, _append_case, _call, _check, _i32, _keep, _make, _want

pytestmark = pytest.mark.gpu


def _unaligned(x, elements=1):
    """A copy of x that begins `elements` behind a 16-byte boundary."""
    flat = torch.empty(x.numel() + 16, dtype=x.dtype, device=x.device)
    y = flat[elements:elements + x.numel()].view(x.shape)
    y.copy_(x)
    assert y.data_ptr() % 16
    return y


def _tokens(a):
    """(sequence, index in it) of each token."""
    pairs = [(b, s) for b, (x, y) in enumerate(zip(a["starts"], a["starts"][1:])) for s in range(y - x)]
    return torch.tensor([b for b, _ in pairs]), torch.tensor([s for _, s in pairs])


@pytest.mark.parametrize("ps", [8, 16, 24, 32, 40, 64, 128, 192])
@pytest.mark.parametrize("heads", [(8, 2, 64), (8, 2, 128), (4, 2, 256), (8, 2, 72)])
def test_last_key_anywhere(lib, cuda, ps, heads):
    """Rows behind the last one hold NaN, in K and V: the call gives the bits it gives over zeros there. Totals on
    both sides of the ends of pages, of 8 rows and of key tiles; many rows and few."""
    Nq, Nkv, H = heads
    for new in (40, 1):
        totals = [40, 41, 47, 48, 63, 64, 65, 71, 100, 120, 127, 128, 129, 136, 190, 200]
        a = _make(ps + H, "bf16", Nq, Nkv, H, ps, [t - new for t in totals], [new] * len(totals))
        b = dict(a, k=a["k"].clone(), v=a["v"].clone())
        for x, hole in ((a, 0.0), (b, float("nan"))):
            for n in ("k", "v"):
                mine = torch.zeros(x[n].shape[0], ps, dtype=torch.bool)
                for row, total in zip(x["table"], totals):
                    for j in range(total):
                        mine[row[j // ps], j % ps] = True
                x[n].masked_fill_(~mine[:, None, :, None], hole)
        want = _check(lib, a, cuda, f"{ps} {heads} {new}")
        assert torch.equal(_call(lib, b, cuda), want), new


@pytest.mark.parametrize("new", [1, 3, 20])
def test_more_sequences_than_are_dealt(lib, cuda, new):
    B = 1100
    a = _make(3, "f16", 8, 2, 64, 16, [(7 * b) % 90 for b in range(B)], [new if b % 7 else 0 for b in range(B)])
    _check(lib, a, cuda)


@pytest.mark.parametrize("Nq,Nkv,H,new", [
    (24, 1, 128, [1, 1]), (24, 1, 128, [1, 9]), (130, 1, 64, [1, 5]), (129, 1, 256, [1, 3]), (300, 1, 64, [1, 2]),
    (256, 1, 128, [1, 2]), (257, 1, 128, [2, 1]), (17, 1, 64, [1, 1]), (32, 2, 96, [1, 40])])
def test_wide_groups(lib, cuda, Nq, Nkv, H, new):
    for dtype in ("f16", "f32"):
        _check(lib, _make(4, dtype, Nq, Nkv, H, 16, [150, 77], new), cuda)


@pytest.mark.parametrize("shape", ["token", "chunk", "mixed"])
@pytest.mark.parametrize("which", ["q", "k", "v", "out"])
def test_unaligned_tensors(lib, cuda, shape, which):
    """2 bytes behind a 16-byte boundary: CUDA cores, the same definition."""
    a = _make(5, "f16", *SHAPES[shape])
    want, bound, _ = _want(a, cuda)
    kw = {}
    if which == "out":
        kw["out"] = _unaligned(torch.zeros_like(a["q"]).to(cuda))
    else:
        a = dict(a, **{which: _unaligned(a[which].to(cuda))})
    pu.close(_call(lib, a, cuda, **kw), want, bound)
    assert lib.last_kernel() == "paged_simple_kernel"


def test_unaligned_append_and_keep(lib, cuda):
    a = _append_case(6, "f16", *APPENDS["odd_heads"], norm=True)
    k, v = a["k"].to(cuda), a["v"].to(cuda)
    k2, v2 = _unaligned(k), _unaligned(v)
    q, q2 = _append(lib, a, cuda, k, v), _append(lib, a, cuda, k2, v2)
    assert torch.equal(v, v2)
    # Wide and narrow loads add a head's squares in different orders. The squares are exact in 32 bits and positive,
    # so the two sums differ by at most 2 H 2^-24 relative and the norms' factors by H 2^-24 + 4 2^-24 < 2^-16 for H <=
    # 250: x r rounds to the same float16 or the next (2^-10), that times w to within 2^-10 + 2 2^-11 = 2^-9, and a
    # rotated value, rounded on both sides, to within 2^-9 + 2 2^-11 < 2^-8 of |a cos| + |b sin|.
    Nq, Nkv, H = a["Nq"], a["Nkv"], a["k"].shape[3]
    assert H <= 250 and not a["inter"] and not a["rd"]
    x = a["q"].double().view(-1, Nq + 2 * Nkv, H)[:, :Nq + Nkv]
    z = (x / (x.square().mean(-1, keepdim=True) + 1e-6).sqrt()).abs()
    z[:, :Nq] *= a["qw"].double()
    z[:, Nq:] *= a["kw"].double()
    b, s = _tokens(a)
    row = torch.tensor(a["past"])[b] + s
    c, sn = a["cos"].double()[row][:, None].abs(), a["sin"].double()[row][:, None].abs()
    u, w = z[..., :H // 2], z[..., H // 2:]
    most = 2.0 ** -8 * torch.cat([u * c + w * sn, w * c + u * sn], -1)
    assert ((q.double() - q2.double()).abs().cpu() <= most[:, :Nq].reshape(q.shape)).all()
    page = torch.tensor([a["table"][int(i)][int(r) // k.shape[2]] for i, r in zip(b, row)])
    off = (k.double() - k2.double()).abs().cpu()
    assert (off[page, :, row % k.shape[2]] <= most[:, Nq:]).all()
    off[page, :, row % k.shape[2]] = 0.0
    assert not off.any()
    k, v = (torch.randn((6, 2, 16, 64), device=cuda).half() for _ in range(2))
    k2, v2 = _unaligned(k), _unaligned(v)
    for x, y in ((k, v), (k2, v2)):
        _keep(lib, cuda, x, y, [[0, 3], [5, 1]], [4, 10], [[1, 5], [0, 2, 9]])
    assert torch.equal(k, k2) and torch.equal(v, v2)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
def test_far_pages(lib, cuda, dtype):
    """Pages whose elements lie behind 2^31: the bits of the same rows in a small pool."""
    Nq, Nkv, H, ps = 8, 2, 128, 64
    far = (1 << 31) // (Nkv * ps * H) + 70
    big = [torch.zeros((far, Nkv, ps, H), dtype=T[dtype], device=cuda) for _ in range(2)]
    for new in ([1, 1], [90, 5]):
        a = _make(7, dtype, Nq, Nkv, H, ps, [300, 130], new)
        pages = a["k"].shape[0]
        for x, small in zip(big, (a["k"], a["v"])):
            x[far - pages:] = small.to(cuda)
        moved = [[p + far - pages if 0 <= p < pages else p for p in row] for row in a["table"]]
        want = _call(lib, a, cuda)
        assert torch.equal(_call(lib, dict(a, k=big[0], v=big[1], table=moved), cuda), want)
    b = _append_case(8, dtype, Nq, Nkv, H, ps, [300, 130], [20, 1])
    pages = b["k"].shape[0]
    for x, small in zip(big, (b["k"], b["v"])):
        x[far - pages:] = small.to(cuda)
    moved = [[p + far - pages if 0 <= p < pages else p for p in row] for row in b["table"]]
    k, v = b["k"].to(cuda), b["v"].to(cuda)
    assert torch.equal(_append(lib, b, cuda, k, v), _append(lib, dict(b, table=moved), cuda, *big))
    assert torch.equal(big[0][far - pages:], k) and torch.equal(big[1][far - pages:], v)
    _keep(lib, cuda, k, v, b["table"], [300, 130], [[0, 4, 19], [0]])
    _keep(lib, cuda, *big, moved, [300, 130], [[0, 4, 19], [0]])
    assert torch.equal(big[0][far - pages:], k) and torch.equal(big[1][far - pages:], v)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_pages(lib, cuda, dtype):
    """Sequences that begin alike share those pages."""
    for new in ([1, 1, 1], [1, 70, 2]):
        a = _make(9, dtype, 8, 2, 128, 16, [100, 100, 64], new)
        for row in a["table"][1:]:
            row[:4] = a["table"][0][:4]
        _check(lib, a, cuda)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_starts_that_do_not_ascend(lib, cuda, dtype):
    """Nothing outside the tensors is touched, and what no sequence names stays as it was."""
    a = _make(10, dtype, 8, 2, 64, 16, [20, 30, 10], [12, 12, 12], behind=6)
    a["starts"] = [4, 12, 9, 30]
    for most in (36, 21, 3):
        out = torch.full_like(a["q"], 7.0).to(cuda)
        got = _call(lib, a, cuda, out=out, max_query_len=most)
        assert torch.equal(got[:4], torch.full_like(got[:4], 7.0)) and torch.equal(got[30:], torch.full_like(got[30:], 7.0))
    want, bound, _ = _want(dict(a, starts=[4, 12, 12, 12]), cuda)
    got = _call(lib, a, cuda, max_query_len=36)
    pu.close(got[4:9], want[4:9], bound[4:9])  # tokens of one sequence alone


def test_most_is_not_given(lib, cuda):
    for shape in ("token", "mixed", "few"):
        a = _make(11, "bf16", *SHAPES[shape])
        want, bound, _ = _want(a, cuda)
        pu.close(_call(lib, a, cuda, max_query_len=None), want, bound)


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_lengths_change_between_replays(lib, cuda, dtype):
    """One captured call, planned for the most it has to take; lengths, starts, pages and queries are those of each
    replay."""
    Nq, Nkv, H, ps, B, tokens, width, most = 8, 2, 128, 16, 24, 340, 40, 300
    steps = [([0] * 24, [1] * 24), ([300 + b for b in range(24)], [1] * 23 + [300]), ([17 * b for b in range(24)], [0, 60] * 3 + [2] * 18),
             ([5] * 24, [0] * 24), ([600] * 24, [1] * 24)]
    q = torch.zeros((tokens, Nq * H), dtype=T[dtype], device=cuda)
    k, v = (torch.zeros((B * width, Nkv, ps, H), dtype=T[dtype], device=cuda) for _ in range(2))
    table, past, starts = torch.zeros((B, width), dtype=torch.int32, device=cuda), _i32([0] * B, cuda), _i32([0] * (B + 1), cuda)
    out = torch.zeros_like(q)

    def run():
        lib.kv_attention_paged(q, k, v, table, past, num_heads=Nq, query_starts=starts, max_query_len=most, out=out)

    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i, (p, n) in enumerate(steps):
        a = _make(20 + i, dtype, Nq, Nkv, H, ps, p, n, behind=tokens - sum(n))
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


def test_two_calls_at_a_time(lib, cuda):
    """Calls of both kernels on two streams side by side, each with a workspace of its own."""
    sides = [torch.cuda.Stream() for _ in range(2)]
    calls = [_make(30 + i, "bf16", *SHAPES[s]) for i, s in enumerate(("mixed_many", "mixed_narrow"))]
    want = [_call(lib, a, cuda) for a in calls]
    moved = []
    for a in calls:
        moved.append(dict(a, q=a["q"].to(cuda), k=a["k"].to(cuda), v=a["v"].to(cuda)))
    torch.cuda.synchronize()
    for _ in range(8):
        got = []
        for side, a in zip(sides, moved):
            with torch.cuda.stream(side):
                got.append(_call(lib, a, cuda))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("dtype,variant", [("f16", "auto"), ("f16", "simt"), ("f32", "auto")])
def test_the_next_kernel_sees_what_was_written(lib, cuda, dtype, variant):
    """Append, attention, keep and append again with nothing between them: what each writes is there for the next,
    although each kernel starts before the one in front of it ends."""
    Nq, Nkv, H, ps, B = 8, 2, 128, 16, 40
    b = _append_case(40, dtype, Nq, Nkv, H, ps, [11 * i % 300 for i in range(B)], [1] * (B - 1) + [200])
    starts, past, table = (_i32(b[n], cuda) for n in ("starts", "past", "table"))
    q, cos, sin = (b[n].to(cuda) for n in ("q", "cos", "sin"))
    kept, lens = _i32([[0]] * (B - 1) + [[5]], cuda), _i32([1] * B, cuda)

    def step(wait):
        k, v = b["k"].to(cuda), b["v"].to(cuda)
        outs = []
        for turn in range(3):
            qo = lib.rope_apply_qkv_paged(q + turn, cos, sin, num_heads=Nq, kv_num_heads=Nkv, k_pages=k, v_pages=v, page_table=table,
                                          past_seq_lens=past, query_starts=starts)
            wait()
            outs.append(lib.kv_attention_paged(qo, k, v, table, past, num_heads=Nq, query_starts=starts, max_query_len=200))
            wait()
            lib.kv_keep_paged(k, v, table, past, kept, lens)
            wait()
            outs.append(lib.kv_attention_paged(qo, k, v, table, past, num_heads=Nq, query_starts=starts, max_query_len=200))
            wait()
        return [*outs, k, v]

    with lib.variant(variant):
        want = step(torch.cuda.synchronize)
        for _ in range(5):
            for x, y in zip(step(lambda: None), want):
                assert torch.equal(x, y)


def test_append_kernels(lib, cuda):
    for shape, kernel in (((8, 2, 128, 16, [3, 9], [1, 70]), "paged_append_heads_kernel"),
                          ((8, 2, 19 * 2, 16, [3, 9], [1, 70]), "paged_append_kernel")):
        a = _append_case(41, "bf16", *shape)
        _append(lib, a, cuda, a["k"].to(cuda), a["v"].to(cuda))
        assert lib.last_kernel() == kernel


@pytest.mark.parametrize("H", [8, 16, 24, 40, 56, 104, 136, 200, 248])
def test_head_sizes(lib, cuda, H):
    """Multiples of 8 run padded on the tensor cores."""
    for new, kernel in (([1, 2, 1], "token"), ([70, 1, 30], "tile")):
        _check(lib, _make(H, "f16", 6, 3, H, 32, [150, 77, 40], new), cuda, f"{H} {new}")
        assert lib.last_kernel() == f"paged_{kernel}_kernel"


@pytest.mark.parametrize("width,window,cap", [(32, 0, 0.0), (34, 0, 0.0), (44, 0, 0.0), (46, 0, 0.0), (60, 0, 0.0), (200, 300, 0.0),
                                              (200, 700, 0.0), (20, 0, 30.0), (32, 0, 30.0)])
def test_split_or_not(lib, cuda, width, window, cap):
    """On both sides of the table widths and windows up to which no item is split, with a workspace and without."""
    a = _make(width + window, "f16", 4, 4, 64, 16, [150, 0, 200, 3, 190], [300, 17, 90, 1, 120], cap=cap, window=window)
    for row in a["table"]:
        row += [-3] * (width - len(row))
    want = _check(lib, a, cuda, "planned")
    none = torch.zeros(0, dtype=torch.uint8, device=cuda)
    _check(lib, a, cuda, "none", workspace=none)
    assert torch.equal(_call(lib, a, cuda), want)
