"""The measured cases of the paged-cache operators: append, attention (of plain batches and of draft trees), keep.

Four operators of one attention layer of a serving step, over caches held in pages that a page table deals to
the sequences, each sequence with any number of new tokens:

  rope_apply_qkv_paged   Q and K rotation (optionally QK-RMSNorm first) with the append of K and V to pages;
  kv_attention_paged     attention of each sequence's new tokens over its pages: single tokens, prompts, both in
                         one batch; with ``tree_masks`` the new tokens are trees of drafts, each seeing its
                         ancestors;
  kv_keep_paged          after verification: the rows of the accepted drafts move up behind the older ones.

Each case runs one call. ``own`` false computes it with elementary torch operations in 32 bits; ``own`` true calls
the package. A case fixes the lengths of its sequences; the seed deals them, the pages and the values.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SHORT = 64        # new tokens up to which the plain form pads sequences together
TREE_MOST = 64    # nodes of a tree: bits of a mask


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _case(name, op, dtype, heads, page, B, past, new=(1, 1), prompts=0, prompt=(0, 0), tree=False, norm=False,
          interleaved=False, rd=0, cap=0.0, window=0, alibi=False, kept=(0, 0)):
    """``past`` and ``new`` are the ends between which the sequences' older rows and new tokens lie; the first
    ``prompts`` sequences have ``prompt`` new tokens instead."""
    return {"name": name, "op": op, "dtype": dtype, "Nq": heads[0], "Nkv": heads[1], "H": heads[2], "page": page,
            "B": B, "past_lo": past[0], "past_hi": past[1], "new_lo": new[0], "new_hi": new[1], "prompts": prompts,
            "prompt_lo": prompt[0], "prompt_hi": prompt[1], "tree": tree, "norm": norm, "interleaved": interleaved,
            "rd": rd, "cap": cap, "window": window, "alibi": alibi, "kept_lo": kept[0], "kept_hi": kept[1]}


def listed():
    return [
        # one decode step of 256 sequences
        _case("append_decode_256", "append", "f16", (32, 8, 128), 16, 256, (0, 2047)),
        # chunks of seven prompts behind cached tokens, with QK-Norm
        _case("append_prompts_norm", "append", "bf16", (32, 8, 128), 64, 7, (0, 1500), prompts=7, prompt=(301, 2048),
              norm=True),
        # draft trees of a small model in 32 bits: positions by depth, partial interleaved rotation
        _case("append_tree_f32", "append", "f32", (28, 4, 64), 16, 5, (5, 900), new=(20, 61), tree=True,
              interleaved=True, rd=32),
        # one user's next token over a short chat: latency is all of it
        _case("decode_one", "attend", "f16", (32, 8, 128), 16, 1, (777, 777)),
        # a batch of next tokens over histories of every length
        _case("decode_batch", "attend", "bf16", (32, 8, 128), 64, 64, (1, 8190)),
        # prompts of odd lengths in a layer that sees the last 512 keys
        _case("prompts_window", "attend", "f16", (16, 16, 64), 16, 5, (0, 2401), prompts=5, prompt=(100, 1531),
              window=512),
        # a chunk of a prompt beside the next tokens of 95 sequences, with capped scores
        _case("mixed_capped", "attend", "bf16", (40, 8, 128), 16, 96, (0, 4000), prompts=1, prompt=(2048, 2048), cap=50.0),
        # a small model kept in 32 bits, pages of a size that is no power of two
        _case("prompts_f32", "attend", "f32", (8, 2, 64), 24, 3, (0, 100), prompts=3, prompt=(57, 301), cap=20.0),
        # one user's draft tree behind a long context
        _case("tree_one", "attend", "bf16", (32, 8, 128), 64, 1, (8000, 8000), new=(60, 60), tree=True),
        # draft trees of 32 sequences
        _case("tree_batch", "attend", "f16", (32, 8, 128), 16, 32, (1, 4096), new=(26, 64), tree=True),
        # the accepted paths of 64 sequences' trees
        _case("keep_64", "keep", "f16", (32, 8, 128), 16, 64, (0, 2000), new=(60, 60), tree=True, kept=(1, 7)),
        # the same of a few sequences of a small model, long paths
        _case("keep_long_paths", "keep", "bf16", (28, 4, 64), 64, 3, (100, 900), new=(64, 64), tree=True, kept=(13, 40)),
    ]


HEADS = [(32, 8, 128), (28, 4, 128), (40, 8, 128), (8, 1, 128), (16, 16, 64), (12, 2, 64), (6, 3, 32), (10, 5, 96),
         (16, 8, 256)]
PAGES = [16, 16, 32, 64, 64, 128, 8, 24, 20]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend", "tree", "keep"])
    heads = rng.choice(HEADS)
    dtype = rng.choice(["f16", "bf16", "f16", "bf16", "f16", "bf16", "f32"])
    page = rng.choice(PAGES)
    row = heads[1] * heads[2]
    more = {}
    if op == "append":
        kind = rng.choice(["token", "tree", "prompts"])
        hi = _spread(rng, 1, 3000)
        B = _spread(rng, 1, max(1, min(256, (1 << 27) // ((hi + 64) * row))))
        if kind == "tree":
            B = min(B, 64)
            more = dict(new=(rng.randint(1, 20), rng.randint(21, TREE_MOST)), tree=True)
        elif kind == "prompts":
            B = min(B, 8)
            more = dict(prompts=B, prompt=(rng.randint(1, 200), _spread(rng, 200, 1000)))
        more.update(norm=rng.random() < 0.4, interleaved=rng.random() < 0.4, rd=rng.choice([0, 0, heads[2] // 2]))
    elif op == "keep":
        hi = _spread(rng, 1, 2000)
        B = _spread(rng, 1, max(1, min(128, (1 << 27) // ((hi + 64) * row))))
        more = dict(new=(rng.randint(20, 50), rng.randint(50, TREE_MOST)), tree=True, kept=(rng.randint(0, 3), rng.randint(4, 20)))
    else:  # attention, of a plain batch or of trees
        more = dict(cap=rng.choice([0.0, 0.0, 30.0, 50.0]))
        kind = "tree" if op == "tree" else rng.choice(["token", "token", "few", "prompts", "mixed"])
        small = dtype == "f32" or page % 8 != 0  # these run on CUDA cores
        if small:
            hi, B = _spread(rng, 1, 400), rng.randint(1, 3)
            more.update(new=(1, rng.randint(1, 16)) if kind != "tree" else (rng.randint(1, 20), rng.randint(21, TREE_MOST)))
            if kind in ("prompts", "mixed"):
                more.update(prompts=1, prompt=(rng.randint(20, 60), rng.randint(61, 300)))
        elif kind in ("token", "few", "tree"):
            hi = _spread(rng, 8, 16384)
            if kind == "few":
                more.update(new=(1, rng.randint(2, 16)))
            if kind == "tree":
                more.update(new=(rng.randint(1, 30), rng.randint(31, TREE_MOST)))
            B = _spread(rng, 1, max(1, min(128 if kind == "token" else 32, (1 << 28) // (hi * row))))
        else:
            hi = _spread(rng, 1, 2048)
            long = _spread(rng, 70, 2000)
            n = rng.randint(1, 4) if long < 1000 else 1
            B = n if kind == "prompts" else n + _spread(rng, 1, max(1, min(64, (1 << 27) // (hi * row))))
            more.update(new=(1, 1), prompts=n, prompt=(rng.randint(65, long), long))
        more["tree"] = kind == "tree"
        if kind != "tree":
            more.update(window=rng.choice([0, 0, 0, _spread(rng, 1, 2000)]), alibi=rng.random() < 0.2)
        op = "attend"
    case = _case("", op, dtype, heads, page, B, (rng.randint(0, hi), hi), **more)
    return {k: v for k, v in case.items() if k != "name"}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _between(lo, hi, n):
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _lengths(c):
    """(older rows, new tokens) of each sequence, in an order that the case fixes."""
    B, P = c["B"], c["prompts"]
    past = _between(c["past_lo"], c["past_hi"], B)
    turn = max(1, B * 5 // 8) | 1
    past = [past[i * turn % B] for i in range(B)] if math.gcd(turn, B) == 1 else past
    return list(zip(past, _between(c["prompt_lo"], c["prompt_hi"], P) + _between(c["new_lo"], c["new_hi"], B - P)))


def _trees(sizes, host):
    """(masks, depths) of random trees: node 0 is a root, another's parent is one of the 12 before it."""
    masks, depths = [], []
    for n in sizes:
        pick = torch.rand(n, generator=host).tolist()
        word, depth = [1], [0]
        for i in range(1, n):
            parent = max(0, i - 12) + int(pick[i] * (i - max(0, i - 12)))
            word.append(word[parent] | 1 << i)
            depth.append(depth[parent] + 1)
        masks += [w - (1 << 64) if w >> 63 else w for w in word]
        depths += depth
    return masks, depths


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    T = DTYPES[case["dtype"]]
    B, Nq, Nkv, H, ps = (case[k] for k in ("B", "Nq", "Nkv", "H", "page"))

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(T)

    def ints(v, kind=torch.int32):
        return torch.tensor(v, dtype=kind, device=dev)

    lengths = _lengths(case)
    lengths = [lengths[i] for i in torch.randperm(B, generator=host).tolist()]
    past, new = [p for p, _ in lengths], [n for _, n in lengths]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    st = {"case": case, "past": ints(past), "starts": ints(starts), "most": max(new), "tokens": starts[-1]}
    # a pool of pages of which the sequences hold some, in no order, and a table as wide as the longest needs
    held = [-(-(p + n) // ps) for p, n in lengths]
    pages = sum(held) + 3
    order = torch.randperm(pages, generator=host, dtype=torch.int32).tolist()
    rows, at = [], 0
    for n in held:
        rows.append(order[at:at + n] + [0] * (max(held) - n))
        at += n
    st["table"], st["spare"] = ints(rows), order[-1]
    st["k_pages"], st["v_pages"] = normal(pages, Nkv, ps, H), normal(pages, Nkv, ps, H)
    if case["tree"]:
        masks, depths = _trees(new, host)
        st["masks"] = ints(masks, torch.int64)
        base = [p for p, n in lengths for _ in range(n)]
        st["positions"] = ints([p + d for p, d in zip(base, depths)], torch.int64)
    if case["op"] == "append":
        rd = case["rd"] or H
        inv = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=dev) / rd)
        angle = torch.arange(max(p + n for p, n in lengths), dtype=torch.float64, device=dev)[:, None] * inv
        st["cos"], st["sin"] = angle.cos().to(T), angle.sin().to(T)
        st["qkv"] = normal(starts[-1], (Nq + 2 * Nkv) * H)
        if case["norm"]:
            st["qw"], st["kw"] = ((torch.rand(H, generator=g, device=dev) + 0.5).to(T) for _ in range(2))
        return st
    if case["op"] == "keep":
        count = _between(case["kept_lo"], case["kept_hi"], B)
        count = [min(count[i], n) for i, n in zip(torch.randperm(B, generator=host).tolist(), new)]
        paths = [torch.randperm(n, generator=host)[:k].sort().values.tolist() for n, k in zip(new, count)]
        st["kept"] = ints([p + [0] * (max(1, case["kept_hi"]) - len(p)) for p in paths])
        st["kept_lens"] = ints(count)
        return st
    # rotated queries whose scores spread as in a trained model's heads (a few units)
    st["q"] = normal(starts[-1], Nq * H, scale=1.5)
    if case["alibi"]:
        st["slopes"] = 2.0 ** (-8.0 * (torch.arange(Nq, dtype=torch.float32, device=dev) + 1) / Nq)
    # the sequences that the plain form pads together: those with few new tokens, and the others
    for name, which in (("short", [b for b in range(B) if new[b] <= SHORT]), ("long", [b for b in range(B) if new[b] > SHORT])):
        if which:
            pad = max(new[b] for b in which)
            st[name] = {"which": ints(which, torch.int64), "pad": pad, "keys": max(past[b] + new[b] for b in which),
                        "tokens": ints([t for b in which for t in range(starts[b], starts[b + 1])], torch.int64),
                        "places": ints([i * pad + s for i, b in enumerate(which) for s in range(new[b])], torch.int64)}
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op == "attend":
        return _own_attend(state) if own else _plain_attend(state)
    if op == "append":
        q = _own_append(state) if own else _plain_append(state)
        return {"q": q, "k_pages": state["k_pages"], "v_pages": state["v_pages"]}
    (_own_keep if own else _plain_keep)(state)
    return {"k_pages": state["k_pages"], "v_pages": state["v_pages"]}


def _own_append(st):
    import rotary_position_embedding_gb300 as rp

    c = st["case"]
    return rp.rope_apply_qkv_paged(st["qkv"], st["cos"], st["sin"], st.get("positions"), num_heads=c["Nq"],
                                   kv_num_heads=c["Nkv"], k_pages=st["k_pages"], v_pages=st["v_pages"],
                                   page_table=st["table"], past_seq_lens=st["past"], query_starts=st["starts"],
                                   interleaved=int(c["interleaved"]), rotary_embedding_dim=c["rd"],
                                   q_norm_weight=st.get("qw"), k_norm_weight=st.get("kw"))


def _own_attend(st):
    import rotary_position_embedding_gb300 as rp

    c = st["case"]
    return rp.kv_attention_paged(st["q"], st["k_pages"], st["v_pages"], st["table"], st["past"], num_heads=c["Nq"],
                                 query_starts=st["starts"], max_query_len=st["most"], softcap=c["cap"],
                                 window=c["window"], alibi_slopes=st.get("slopes"),
                                 tree_masks=st["masks"] if c["tree"] else None)


def _own_keep(st):
    import rotary_position_embedding_gb300 as rp

    rp.kv_keep_paged(st["k_pages"], st["v_pages"], st["table"], st["past"], st["kept"], st["kept_lens"])


def _sequence_of(st):
    """(sequence, index in it) of each token."""
    at = torch.arange(st["tokens"], device=st["starts"].device)
    b = torch.searchsorted(st["starts"][1:].long(), at, right=True)
    return b, at - st["starts"].long()[b]


def _plain_append(st):
    """The definition step by step: QK-Norm and the rotation round to the storage type where the package's Q/K
    operators do (each a part of their definition)."""
    c = st["case"]
    T = DTYPES[c["dtype"]]
    Nq, Nkv, H, ps = (c[k] for k in ("Nq", "Nkv", "H", "page"))
    rd = c["rd"] or H
    b, s = _sequence_of(st)
    row = st["past"].long()[b] + s
    position = st["positions"] if c["tree"] else row
    x = st["qkv"].float().view(-1, Nq + 2 * Nkv, H)
    qk = x[:, :Nq + Nkv]
    if c["norm"]:
        r = torch.rsqrt(qk.square().mean(-1, keepdim=True) + 1e-6)
        w = torch.cat([st["qw"].expand(Nq, H), st["kw"].expand(Nkv, H)]).float()
        qk = ((qk * r).to(T).float() * w).to(T).float()
    cos, sin = st["cos"][position].float()[:, None], st["sin"][position].float()[:, None]
    turned, tail = qk[..., :rd], qk[..., rd:]
    if c["interleaved"]:
        u, w = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([u * cos - w * sin, w * cos + u * sin], -1).flatten(-2)
    else:
        u, w = turned[..., :rd // 2], turned[..., rd // 2:]
        turned = torch.cat([u * cos - w * sin, w * cos + u * sin], -1)
    qk = torch.cat([turned, tail], -1).to(T)
    page = st["table"].long()[b, row // ps]
    st["k_pages"][page, :, row % ps] = qk[:, Nq:]
    st["v_pages"][page, :, row % ps] = x[:, Nq + Nkv:].to(T)
    return qk[:, :Nq].reshape(-1, Nq * H)


def _plain_attend(st):
    out = torch.empty_like(st["q"])
    if "short" in st:
        _plain_group(st, st["short"], out)
    if "long" in st:
        _plain_group(st, st["long"], out)
    return out


def _plain_group(st, group, out):
    """Sequences padded to as many tokens and keys as the longest has."""
    c = st["case"]
    Nq, Nkv, H, ps = (c[k] for k in ("Nq", "Nkv", "H", "page"))
    G, S, n, which = Nq // Nkv, group["pad"], group["keys"], group["which"]
    j = torch.arange(n, device=which.device)
    page = st["table"].long()[which][:, j // ps]
    k = st["k_pages"][page, :, j % ps].float().transpose(1, 2)
    v = st["v_pages"][page, :, j % ps].float().transpose(1, 2)
    token = (st["starts"].long()[which][:, None] + torch.arange(S, device=which.device)).clamp(max=st["tokens"] - 1)
    q = st["q"][token].float().view(-1, S, Nkv, G, H).permute(0, 2, 3, 1, 4).reshape(-1, Nkv, G * S, H)
    s = torch.matmul(q * H ** -0.5, k.transpose(2, 3)).view(-1, Nkv, G, S, n)
    if c["cap"]:
        s.div_(c["cap"]).tanh_().mul_(c["cap"])
    past = st["past"].long()[which][:, None, None]
    i = past + torch.arange(S, device=which.device)[:, None]
    if c["alibi"]:
        s.sub_(st["slopes"].view(Nkv, G, 1, 1) * (i - j).abs().float()[:, None, None])
    if c["tree"]:
        bit = j - past
        seen = (bit < 0) | ((bit < TREE_MOST) & (st["masks"][token][:, :, None] >> bit.clamp(0, 63) & 1).bool())
    else:
        seen = j <= i
        if c["window"]:
            seen = seen & (j > i - c["window"])
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(s.view(-1, Nkv, G * S, n), v) / s.sum(-1).view(-1, Nkv, G * S, 1)
    o = o.view(-1, Nkv, G, S, H).permute(0, 3, 1, 2, 4).reshape(-1, Nq * H)
    out[group["tokens"]] = o[group["places"]].to(out.dtype)


def _plain_keep(st):
    c = st["case"]
    ps = c["page"]
    i = torch.arange(st["kept"].shape[1], device=st["kept"].device)
    past = st["past"].long()[:, None]
    on = i < st["kept_lens"][:, None]
    table = st["table"].long()

    def place(row):
        """(page, row of it); what is not kept goes from a row that no sequence holds to itself."""
        page = table.gather(1, torch.where(on, row // ps, 0))
        return torch.where(on, page, st["spare"]), torch.where(on, row % ps, 0)

    page, row = place(past + st["kept"].long())
    to_page, to_row = place(past + i)
    k, v = st["k_pages"][page, :, row], st["v_pages"][page, :, row]
    st["k_pages"][to_page, :, to_row] = k
    st["v_pages"][to_page, :, to_row] = v


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    es = torch.finfo(DTYPES[case["dtype"]]).bits // 8
    B, Nq, Nkv, H = (case[k] for k in ("B", "Nq", "Nkv", "H"))
    lengths = _lengths(case)
    tokens = sum(n for _, n in lengths)
    if case["op"] == "append":
        rd = case["rd"] or H
        table = min(max(p + n for p, n in lengths), tokens)
        return {"bytes": (2 * tokens * (Nq + 2 * Nkv) * H + table * rd) * es, "flops": tokens * (Nq + Nkv) * 3 * rd}
    if case["op"] == "keep":
        rows = sum(min(k, n) for k, (_, n) in zip(_between(case["kept_lo"], case["kept_hi"], B), lengths))
        return {"bytes": 4 * rows * Nkv * H * es, "flops": 0}
    pairs = keys = 0
    for p, n in lengths:
        w = case["window"] or p + n
        # token s sees min(p + s + 1, w) keys; nodes of a tree are taken to see half of the tree's older nodes
        full = max(0, min(n, p + n - w))  # tokens that see w keys
        pairs += full * w + (n - full) * p + (n - full) * (n - full + 1) / 2
        if case["tree"]:
            pairs -= n * (n - 1) / 4
        keys += min(p + n, w + n - 1)
    return {"bytes": (2 * tokens * Nq + 2 * keys * Nkv) * H * es, "flops": 4 * pairs * Nq * H}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(st, case)
    pages = {name: st[name].double() for name in ("k_pages", "v_pages")}
    if case["op"] == "append":
        return {"q": _exact_append(st, case, pages), **pages}
    table, past = st["table"].tolist(), st["past"].tolist()
    for b, n in enumerate(st["kept_lens"].tolist()):
        path = st["kept"][b].tolist()
        for name in pages:
            rows = [st[name][table[b][(past[b] + k) // case["page"]], :, (past[b] + k) % case["page"]] for k in path[:n]]
            for i, row in enumerate(rows):
                pages[name][table[b][(past[b] + i) // case["page"]], :, (past[b] + i) % case["page"]] = row.double()
    return pages


def _exact_append(st, c, pages):
    """One sequence at a time."""
    T = DTYPES[c["dtype"]]
    Nq, Nkv, H, ps = (c[k] for k in ("Nq", "Nkv", "H", "page"))
    rd = c["rd"] or H
    first = torch.arange(0, rd, 2, device=st["qkv"].device) if c["interleaved"] else torch.arange(rd // 2, device=st["qkv"].device)
    second = first + (1 if c["interleaved"] else rd // 2)
    starts, past = st["starts"].tolist(), st["past"].tolist()
    q = torch.empty((st["tokens"], Nq, H), dtype=torch.float64, device=st["qkv"].device)
    for b in range(c["B"]):
        lo, hi = starts[b], starts[b + 1]
        rows = torch.arange(past[b], past[b] + hi - lo, device=q.device)
        at = st["positions"][lo:hi] if c["tree"] else rows
        z = st["qkv"][lo:hi].double().view(hi - lo, Nq + 2 * Nkv, H)
        if c["norm"]:
            for u, w, weight in ((0, Nq, st["qw"]), (Nq, Nq + Nkv, st["kw"])):
                part = z[:, u:w]
                r = 1.0 / torch.sqrt((part ** 2).sum(-1, keepdim=True) / H + 1e-6)
                z[:, u:w] = ((part * r).to(T).double() * weight.double()).to(T).double()
        cos, sin = st["cos"].double()[at][:, None], st["sin"].double()[at][:, None]
        y = z.clone()
        y[..., first] = z[..., first] * cos - z[..., second] * sin
        y[..., second] = z[..., second] * cos + z[..., first] * sin
        y[:, Nq + Nkv:] = z[:, Nq + Nkv:]
        q[lo:hi] = y[:, :Nq]
        where = st["table"][b].long()[rows // ps]
        pages["k_pages"][where, :, rows % ps] = y[:, Nq:Nq + Nkv]
        pages["v_pages"][where, :, rows % ps] = y[:, Nq + Nkv:]
    return q.view(-1, Nq * H)


def _exact_attend(st, c):
    """One sequence and key/value head at a time."""
    Nq, Nkv, H, ps = (c[k] for k in ("Nq", "Nkv", "H", "page"))
    G = Nq // Nkv
    starts, past = st["starts"].tolist(), st["past"].tolist()
    q = st["q"].double().view(-1, Nkv, G, H)
    out = torch.zeros_like(q)
    for b in range(c["B"]):
        lo, n = starts[b], starts[b + 1] - starts[b]
        total = past[b] + n
        pages = st["table"][b, :-(-total // ps)].long()
        pos = torch.arange(past[b], total, device=q.device)[:, None]
        key = torch.arange(total, device=q.device)[None]
        if c["tree"]:
            hidden = torch.zeros((n, total), dtype=torch.bool, device=q.device)
            words = st["masks"][lo:lo + n]
            for t in range(n):
                hidden[:, past[b] + t] = (words >> t & 1) == 0
        else:
            hidden = key > pos
            if c["window"]:
                hidden |= pos - key >= c["window"]
        k = st["k_pages"][pages].double().transpose(0, 1).reshape(Nkv, -1, H)[:, :total]
        v = st["v_pages"][pages].double().transpose(0, 1).reshape(Nkv, -1, H)[:, :total]
        for h in range(Nkv):
            s = torch.einsum("sgh,th->gst", q[lo:lo + n, h], k[h]) / math.sqrt(H)
            if c["cap"]:
                s = c["cap"] * torch.tanh(s / c["cap"])
            if c["alibi"]:
                s = s - st["slopes"][h * G:(h + 1) * G].double()[:, None, None] * (pos - key).abs().double()
            p = torch.softmax(s.masked_fill(hidden, float("-inf")), -1)
            out[lo:lo + n, h] = torch.einsum("gst,th->sgh", p, v[h])
    return out.view(-1, Nq * H)
