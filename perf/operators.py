"""The measured cases of the cache operators: the 8-bit append and the attention over the caches.

Three operators of one attention layer, in the order in which a serving step calls them:

  rope_apply_qkv_fp8   Q and K rotation (optionally QK-RMSNorm first) with the append of K and V to
                       caches held in 8 bits, one power-of-two scale for each block of 16 rows and head;
  kv_attention         attention of the new tokens over the caches in the storage type;
  kv_attention_fp8     the same over the 8-bit caches.

Each case runs one call. ``own`` false computes it with elementary torch operations in 32 bits; ``own``
true calls the package. Past lengths are spread evenly between a case's two ends and dealt to the
sequences by the seed, documents likewise, so the work of a case does not depend on the seed.
"""

import math

import torch

own = False

BLOCK = 16        # rows of a cache that share a scale
TINY = -120       # exponent of the scale of a block of zeros
DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _append(name, dtype, B, S, Nq, Nkv, H, max_len, lo, hi, norm=False, interleaved=False, rd=0):
    return {"name": name, "op": "append", "dtype": dtype, "B": B, "S": S, "Nq": Nq, "Nkv": Nkv, "H": H,
            "max_len": max_len, "past_lo": lo, "past_hi": hi, "norm": norm, "interleaved": interleaved, "rd": rd}


def _attend(name, op, dtype, B, S, Nq, Nkv, H, max_len, lo, hi, cap=0.0, alibi=False, documents=0, prefix=0):
    return {"name": name, "op": op, "dtype": dtype, "B": B, "S": S, "Nq": Nq, "Nkv": Nkv, "H": H,
            "max_len": max_len, "past_lo": lo, "past_hi": hi, "cap": cap, "alibi": alibi, "documents": documents,
            "prefix": prefix}


def listed():
    return [
        # one decode step of 256 sequences: most of them append inside a block that older tokens scaled
        _append("append_decode_256", "f16", 256, 1, 32, 8, 128, 4096, 0, 4095),
        # a chunk of four prompts behind cached tokens, with QK-Norm
        _append("append_prompt_norm", "bf16", 4, 2048, 32, 8, 128, 4096, 0, 2047, norm=True),
        # a short draft of a small model: partial interleaved rotation, odd lengths
        _append("append_short_odd", "bf16", 3, 37, 28, 4, 64, 1000, 5, 900, interleaved=True, rd=32),
        # one user's next token over a short chat, with a bias by distance: latency is all of it
        _attend("decode_one", "attend", "f16", 1, 1, 32, 8, 128, 4096, 777, 777, alibi=True),
        # a batch of next tokens over histories of every length, with capped scores
        _attend("decode_batch_capped", "attend", "bf16", 64, 1, 32, 8, 128, 8192, 1, 8190, cap=50.0),
        # a chunk of four prompts behind cached tokens, with capped scores
        _attend("prompt_capped", "attend", "f16", 4, 2048, 32, 8, 128, 4096, 0, 2047, cap=30.0),
        # documents packed into one long row
        _attend("prompt_documents", "attend", "bf16", 1, 8192, 28, 4, 128, 8192, 0, 0, documents=11),
        # prompts whose first part is seen by all their tokens, with a bias by distance; odd lengths
        _attend("prompt_prefix_odd", "attend", "bf16", 3, 1531, 16, 16, 64, 2048, 0, 401, alibi=True, prefix=300),
        # a small model kept in 32 bits
        _attend("prompt_f32", "attend", "f32", 2, 301, 8, 2, 64, 512, 0, 100, cap=20.0),
        # a batch of next tokens over 8-bit caches
        _attend("fp8_decode_256", "attend_fp8", "f16", 256, 1, 32, 8, 128, 4096, 0, 4095),
        # one user's next token over a very long context
        _attend("fp8_decode_long", "attend_fp8", "bf16", 1, 1, 32, 8, 128, 131072, 131000, 131000),
        # a chunk of two prompts behind long cached contexts, with capped scores
        _attend("fp8_prompt_chunk", "attend_fp8", "bf16", 2, 1024, 32, 8, 128, 8192, 5000, 7100, cap=50.0),
    ]


HEADS = [(32, 8, 128), (28, 4, 128), (40, 8, 128), (8, 1, 128), (16, 16, 64), (12, 2, 64), (6, 3, 32), (10, 5, 96),
         (16, 8, 256)]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "attend_fp8", "attend_fp8"])
    Nq, Nkv, H = rng.choice(HEADS)
    dtype = rng.choice(["f16", "bf16"])
    if op == "append":
        S = rng.choice([1, rng.randint(2, 17), _spread(rng, 18, 2048)])
        B = _spread(rng, 1, max(1, min(256, 8192 // S)))
        hi = _spread(rng, 1, 4000)
        return {k: v for k, v in _append("", dtype, B, S, Nq, Nkv, H, hi + S + rng.randint(0, 100), rng.randint(0, hi),
                                         hi, norm=rng.random() < 0.4, interleaved=rng.random() < 0.4,
                                         rd=rng.choice([0, 0, H // 2])).items() if k != "name"}
    if op == "attend" and rng.random() < 0.1:
        dtype, H = "f32", 64
    kind = rng.choice(["token", "few", "prompt"])
    if dtype == "f32":
        S, B, hi = rng.choice([1, rng.randint(2, 300)]), rng.randint(1, 2), _spread(rng, 1, 200)
    elif kind == "token":
        S = 1
        hi = _spread(rng, 8, 32768)
        B = _spread(rng, 1, max(1, min(256, (1 << 28) // (hi * Nkv * H))))
    elif kind == "few":
        S = rng.randint(2, 20)
        hi = _spread(rng, 8, 32768)
        B = _spread(rng, 1, max(1, min(64, (1 << 27) // (hi * Nkv * H))))
    else:
        S = _spread(rng, 21, 3000)
        hi = _spread(rng, 1, 2048)
        B = _spread(rng, 1, max(1, min(8, (1 << 23) // (S * (S + hi)))))
    case = _attend("", op, dtype, B, S, Nq, Nkv, H, hi + S + rng.randint(0, 60), rng.randint(0, hi), hi,
                   cap=rng.choice([0.0, 0.0, 30.0, 50.0]), alibi=rng.random() < 0.25,
                   documents=rng.choice([0, 0, 0, rng.randint(2, 12)]),
                   prefix=rng.choice([0, 0, 0, rng.randint(1, hi + S)]))
    return {k: v for k, v in case.items() if k != "name"}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _past_sorted(c):
    B = c["B"]
    return [c["past_lo"] + (c["past_hi"] - c["past_lo"]) * b // max(1, B - 1) for b in range(B)]


def _document_lengths(c):
    """Lengths, one for each document of a row of the cache, growing from the first to the last."""
    n, T = c["documents"], c["max_len"]
    cuts = [T * i * (i + 1) // (n * (n + 1)) for i in range(n + 1)]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _quantised(x):
    """(codes, scales) of x (B, Nkv, L, H), as the append leaves a cache whose blocks were filled at once."""
    B, N, L, H = x.shape
    nb = -(-L // BLOCK)
    p = torch.zeros((B, N, nb * BLOCK, H), dtype=torch.float32, device=x.device)
    p[:, :, :L] = x
    p = p.view(B, N, nb, BLOCK, H)
    scale = _scale_of(p.abs().amax(dim=(3, 4)))
    q = (p / scale[..., None, None]).to(torch.float8_e4m3fn).view(B, N, nb * BLOCK, H)[:, :, :L]
    return q.contiguous(), scale


def _scale_of(amax):
    """The smallest power of two by which amax fits the largest 8-bit value, 448 = 0.875 * 2**9."""
    m, e = torch.frexp(amax.float())
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(amax > 0, e.clamp(min=TINY), torch.full_like(e, TINY))
    return torch.ldexp(torch.ones_like(amax, dtype=torch.float32), e)


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    host = torch.Generator()
    host.manual_seed(seed)
    T = DTYPES[case["dtype"]]
    B, S, Nq, Nkv, H, L = (case[k] for k in ("B", "S", "Nq", "Nkv", "H", "max_len"))

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale)

    lengths = torch.tensor(_past_sorted(case), dtype=torch.int32)[torch.randperm(B, generator=host)]
    st = {"case": case, "past": lengths.to(dev), "longest": int(case["past_hi"]) + S}
    if case["op"] == "append":
        rd = case["rd"] or H
        inv = 10000.0 ** (-torch.arange(0, rd, 2, dtype=torch.float64, device=dev) / rd)
        angle = torch.arange(L, dtype=torch.float64, device=dev)[:, None] * inv
        st["cos"], st["sin"] = angle.cos().to(T), angle.sin().to(T)
        st["qkv"] = normal(B, S, (Nq + 2 * Nkv) * H).to(T)
        # the caches of a running program: what older tokens left, of another magnitude than the new ones
        st["k_cache"], st["k_scale"] = _quantised(normal(B, Nkv, L, H, scale=0.7))
        st["v_cache"], st["v_scale"] = _quantised(normal(B, Nkv, L, H, scale=0.4))
        if case["norm"]:
            st["qw"], st["kw"] = ((torch.rand(H, generator=g, device=dev) + 0.5).to(T) for _ in range(2))
        return st
    # rotated queries and keys whose scores spread as in a trained model's heads (a few units)
    st["q"] = normal(B, S, Nq * H, scale=1.5).to(T)
    k, v = normal(B, Nkv, L, H), normal(B, Nkv, L, H)
    if case["op"] == "attend":
        st["k_cache"], st["v_cache"] = k.to(T), v.to(T)
    else:
        st["k_cache"], st["k_scale"] = _quantised(k)
        st["v_cache"], st["v_scale"] = _quantised(v)
    if case["alibi"]:
        st["slopes"] = 2.0 ** (-8.0 * (torch.arange(Nq, dtype=torch.float32, device=dev) + 1) / Nq)
    if case["documents"]:
        n = torch.tensor(_document_lengths(case))
        ids = [torch.repeat_interleave(torch.arange(len(n), dtype=torch.int32), n[torch.randperm(len(n), generator=host)])
               for _ in range(B)]
        st["documents"] = torch.stack(ids).to(dev)
    if case["prefix"]:
        st["prefix"] = torch.randint(case["prefix"] // 2, case["prefix"] + 1, (B,), generator=host).to(torch.int32).to(dev)
    return st


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if case["op"] == "append":
        q = _own_append(state) if own else _plain_append(state)
        # the codes as 8-bit floating values, with their scales
        return {"q": q, "k_cache": state["k_cache"], "v_cache": state["v_cache"], "k_scale": state["k_scale"],
                "v_scale": state["v_scale"]}
    return _own_attend(state) if own else _plain_attend(state)


def _own_append(st):
    import rotary_position_embedding_gb300 as rp

    c = st["case"]
    return rp.rope_apply_qkv_fp8(st["qkv"], st["cos"], st["sin"], None, num_heads=c["Nq"], kv_num_heads=c["Nkv"],
                                 k_cache=st["k_cache"], v_cache=st["v_cache"], k_scale=st["k_scale"],
                                 v_scale=st["v_scale"], past_seq_lens=st["past"],
                                 interleaved=int(c["interleaved"]), rotary_embedding_dim=c["rd"],
                                 q_norm_weight=st.get("qw"), k_norm_weight=st.get("kw"))


def _own_attend(st):
    import rotary_position_embedding_gb300 as rp

    c = st["case"]
    more = dict(num_heads=c["Nq"], softcap=c["cap"], alibi_slopes=st.get("slopes"), document_ids=st.get("documents"),
                prefix_lens=st.get("prefix"))
    if c["op"] == "attend":
        return rp.kv_attention(st["q"], st["k_cache"], st["v_cache"], st["past"], **more)
    return rp.kv_attention_fp8(st["q"], st["k_cache"], st["v_cache"], st["k_scale"], st["v_scale"], st["past"], **more)


def _plain_append(st):
    """The definition step by step: QK-Norm and the rotation round to the storage type where the
    package's Q/K operators do (each a part of their definition), the 8-bit codes are rounded from that."""
    c = st["case"]
    T = DTYPES[c["dtype"]]
    B, S, Nq, Nkv, H, L = (c[k] for k in ("B", "S", "Nq", "Nkv", "H", "max_len"))
    rd = c["rd"] or H
    x = st["qkv"].float().view(B, S, Nq + 2 * Nkv, H)
    row = st["past"].long()[:, None] + torch.arange(S, device=x.device)
    qk, v = x[:, :, :Nq + Nkv], x[:, :, Nq + Nkv:]
    if c["norm"]:
        r = torch.rsqrt(qk.square().mean(-1, keepdim=True) + 1e-6)
        w = torch.cat([st["qw"].expand(Nq, H), st["kw"].expand(Nkv, H)]).float()
        qk = ((qk * r).to(T).float() * w).to(T).float()
    cos, sin = st["cos"][row].float()[:, :, None], st["sin"][row].float()[:, :, None]
    turned, tail = qk[..., :rd], qk[..., rd:]
    if c["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turned[..., :rd // 2], turned[..., rd // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    qk = torch.cat([turned, tail], -1).to(T)
    _plain_store(qk[:, :, Nq:].float(), row, st["past"].long(), st["k_cache"], st["k_scale"])
    _plain_store(v, row, st["past"].long(), st["v_cache"], st["v_scale"])
    return qk[:, :, :Nq].reshape(B, S, Nq * H)


def _plain_store(x, row, past, cache, scale):
    """Rows x (B, S, Nkv, H) to `row` of an 8-bit cache, whose block scales and older rows follow."""
    B, S, N, H = x.shape
    x = x.transpose(1, 2)
    codes = cache.view(torch.uint8)
    at = torch.arange(B, device=x.device)
    where = (row // BLOCK)[:, None].expand(B, N, S)
    need = torch.zeros_like(scale).scatter_reduce(2, where, x.abs().amax(-1), "amax")
    fresh = _scale_of(need)
    touched = torch.zeros_like(scale, dtype=torch.bool).scatter(2, where, True)
    first = (past // BLOCK)[:, None, None].expand(B, N, 1)
    older = (past % BLOCK > 0)[:, None, None]
    was = scale.gather(2, first)
    fresh = fresh.scatter(2, first, torch.where(older, torch.maximum(was, fresh.gather(2, first)), fresh.gather(2, first)))
    new = torch.where(touched, fresh, scale)
    # older rows of the first block, rounded again by its new scale; its other rows keep their codes
    block = (past // BLOCK * BLOCK)[:, None] + torch.arange(BLOCK, device=x.device)
    inside = block.clamp(max=cache.shape[2] - 1)
    held = cache.view(torch.uint8)[at[:, None], :, inside]
    values = held.view(torch.float8_e4m3fn).float() * (was / new.gather(2, first))[:, None, :, 0, None]
    again = values.to(torch.float8_e4m3fn).view(torch.uint8)
    codes[at[:, None], :, inside] = torch.where((block < past[:, None])[:, :, None, None], again, held)
    mine = (x / new.gather(2, where)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[at[:, None], :, row] = mine.transpose(1, 2)
    scale.copy_(new)


def _values(codes, scale, n):
    """The first n rows that an 8-bit cache stands for."""
    by_row = scale.repeat_interleave(BLOCK, dim=2)[:, :, :n, None]
    return codes[:, :, :n].float() * by_row


def _plain_attend(st):
    c = st["case"]
    B, S, Nq, Nkv, H = (c[k] for k in ("B", "S", "Nq", "Nkv", "H"))
    n = st["longest"]
    if c["op"] == "attend":
        k, v = st["k_cache"][:, :, :n].float(), st["v_cache"][:, :, :n].float()
    else:
        k, v = _values(st["k_cache"], st["k_scale"], n), _values(st["v_cache"], st["v_scale"], n)
    q = st["q"].float().view(B, S, Nkv, Nq // Nkv, H).permute(0, 2, 3, 1, 4).reshape(B, Nkv, -1, H)
    s = torch.matmul(q * H ** -0.5, k.transpose(2, 3)).view(B, Nkv, Nq // Nkv, S, n)
    if c["cap"]:
        s.div_(c["cap"]).tanh_().mul_(c["cap"])
    i = (st["past"].long()[:, None] + torch.arange(S, device=q.device))[:, :, None]
    j = torch.arange(n, device=q.device)
    if c["alibi"]:
        s.sub_(st["slopes"].view(Nkv, -1, 1, 1) * (i - j).abs().float()[:, None, None])
    seen = j <= i
    if c["prefix"]:
        seen = seen | ((j < st["prefix"][:, None, None]) & (j < (st["past"].long() + S)[:, None, None]))
    if c["documents"]:
        ids = st["documents"]
        seen = seen & (ids.gather(1, i[:, :, 0])[:, :, None] == ids[:, None, :n])
    s.masked_fill_(~seen[:, None, None], float("-inf"))
    s.sub_(s.amax(-1, keepdim=True)).exp_()
    out = torch.matmul(s.view(B, Nkv, -1, n), v) / s.sum(-1).view(B, Nkv, -1, 1)
    out = out.view(B, Nkv, Nq // Nkv, S, H).permute(0, 3, 1, 2, 4).reshape(B, S, Nq * H)
    return out.to(DTYPES[c["dtype"]])


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    es = torch.finfo(DTYPES[case["dtype"]]).bits // 8
    B, S, Nq, Nkv, H = (case[k] for k in ("B", "S", "Nq", "Nkv", "H"))
    past = _past_sorted(case)
    if case["op"] == "append":
        rd = case["rd"] or H
        rows = B * S
        table = max(past) + S - min(past)
        read = rows * (Nq + 2 * Nkv) * H * es + min(table, rows) * rd * es
        written = rows * (Nq * es + 2 * Nkv) * H
        scales = 2 * B * Nkv * (S // BLOCK + 1) * 4
        return {"bytes": read + written + scales, "flops": rows * (Nq + Nkv) * 3 * rd}
    kv = 1 + 4.0 / (BLOCK * H) if case["op"] == "attend_fp8" else es
    pairs = keys = 0.0
    share = 1.0
    if case["documents"]:  # of the pairs below the diagonal, those inside a document
        share = sum(n * n for n in _document_lengths(case)) / float(case["max_len"]) ** 2
    for p in past:
        own_rows = S * p + S * (S + 1) / 2
        prefix = min(0.75 * case["prefix"], p + S)
        ahead = max(0.0, prefix - p) ** 2 / 2
        pairs += (own_rows + ahead) * share
        keys += p + S
    return {"bytes": 2 * B * S * Nq * H * es + 2 * keys * Nkv * H * kv, "flops": 4 * pairs * Nq * H}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(st, case)
    return _exact_attend(st, case)


def _to_codes(x, scale):
    return (x / scale).float().to(torch.float8_e4m3fn)


def _exact_append(st, c):
    """Token by token of the definition for each sequence; caches sliced where the append touches them."""
    T = DTYPES[c["dtype"]]
    B, S, Nq, Nkv, H = (c[k] for k in ("B", "S", "Nq", "Nkv", "H"))
    rd = c["rd"] or H
    h = rd // 2
    x = st["qkv"].double().view(B, S, Nq + 2 * Nkv, H)
    first = torch.arange(0, rd, 2, device=x.device) if c["interleaved"] else torch.arange(h, device=x.device)
    second = first + (1 if c["interleaved"] else h)
    q_all = torch.empty((B, S, Nq, H), dtype=torch.float64, device=x.device)
    for b in range(B):
        past = int(st["past"][b])
        z = x[b].clone()
        if c["norm"]:
            for lo, hi, w in ((0, Nq, st["qw"]), (Nq, Nq + Nkv, st["kw"])):
                part = z[:, lo:hi]
                r = 1.0 / torch.sqrt((part ** 2).sum(-1, keepdim=True) / H + 1e-6)
                z[:, lo:hi] = ((part * r).to(T).double() * w.double()).to(T).double()
        cos, sin = (st[k][past:past + S].double()[:, None, :] for k in ("cos", "sin"))
        y = z.clone()
        y[..., first] = z[..., first] * cos - z[..., second] * sin
        y[..., second] = z[..., second] * cos + z[..., first] * sin
        q_all[b] = y[:, :Nq]
        for rows, cache, scale in ((y[:, Nq:Nq + Nkv].to(T).double(), st["k_cache"], st["k_scale"]),
                                   (x[b][:, Nq + Nkv:], st["v_cache"], st["v_scale"])):
            for blk in range(past // BLOCK, (past + S - 1) // BLOCK + 1):
                r0, r1 = max(past, blk * BLOCK), min(past + S, (blk + 1) * BLOCK)
                new = rows[r0 - past:r1 - past].transpose(0, 1)
                need = _scale_of(new.abs().amax(dim=(1, 2))).double()
                if blk * BLOCK < past:
                    was = scale[b, :, blk].double()
                    need = torch.maximum(need, was)
                    old = cache[b, :, blk * BLOCK:past].float().double() * was[:, None, None]
                    cache.view(torch.uint8)[b, :, blk * BLOCK:past] = _to_codes(old, need[:, None, None]).view(torch.uint8)
                cache.view(torch.uint8)[b, :, r0:r1] = _to_codes(new, need[:, None, None]).view(torch.uint8)
                scale[b, :, blk] = need.float()
    return {"q": q_all.view(B, S, Nq * H), "k_cache": st["k_cache"].float().double(), "v_cache": st["v_cache"].float().double(),
            "k_scale": st["k_scale"].double(), "v_scale": st["v_scale"].double()}


def _exact_attend(st, c):
    """One sequence and key/value head at a time."""
    B, S, Nq, Nkv, H = (c[k] for k in ("B", "S", "Nq", "Nkv", "H"))
    G = Nq // Nkv
    q = st["q"].double().view(B, S, Nkv, G, H)
    out = torch.zeros((B, S, Nkv, G, H), dtype=torch.float64, device=q.device)
    for b in range(B):
        past = int(st["past"][b])
        total = past + S
        pos = torch.arange(past, total, device=q.device)[:, None]
        key = torch.arange(total, device=q.device)[None]
        hidden = key > pos
        if c["prefix"]:
            hidden &= key >= int(st["prefix"][b])
        if c["documents"]:
            hidden |= st["documents"][b, past:total, None] != st["documents"][b, None, :total]
        for h in range(Nkv):
            k, v = st["k_cache"][b, h, :total].double(), st["v_cache"][b, h, :total].double()
            if c["op"] == "attend_fp8":
                blk = torch.arange(total, device=q.device) // BLOCK
                k = k * st["k_scale"][b, h].double()[blk, None]
                v = v * st["v_scale"][b, h].double()[blk, None]
            s = torch.einsum("sgh,th->gst", q[b, :, h], k) / math.sqrt(H)
            if c["cap"]:
                s = c["cap"] * torch.tanh(s / c["cap"])
            if c["alibi"]:
                s = s - st["slopes"][h * G:(h + 1) * G].double()[:, None, None] * (pos - key).abs().double()
            p = torch.softmax(s.masked_fill(hidden, float("-inf")), -1)
            out[b, :, h] = torch.einsum("gst,th->sgh", p, v)
    return out.view(B, S, Nq * H)
