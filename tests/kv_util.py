"""The cache operators in 64 bits, for the tests: plain loops over sequences and heads, and the
bounds that the storage types allow."""

import math

import numpy as np
import torch

BLOCK = 16
EPS = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}  # half a step, relative
SMALLEST = {torch.float32: 2.0 ** -149, torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -133}


def visible(past, S, L, s, prefix=None, docs=None):
    """Truth values over the L cache rows: what token s of one sequence sees."""
    i = past + s
    j = np.arange(L)
    seen = j <= i
    if prefix is not None:
        seen |= j < prefix
    seen &= j < past + S
    if docs is not None:
        seen &= (docs == docs[i]) if 0 <= i < L else False
    return seen


def attention(q, k, v, past, num_heads, scale, cap=0.0, slopes=None, docs=None, prefix=None, weight_eps=0.0):
    """(out, bound) in float64 for q (B, S, Nq*H), k and v (B, Nkv, L, H) float64 tensors.

    bound: what float32 sums, weights rounded to ``weight_eps`` and nothing else may add up to. Each of a
    score's H products and additions is off by at most 2^-23 of the sum of magnitudes (a tensor core may
    truncate where an FMA rounds), its scaling, cap and bias by a few more roundings, so a score is off by
    at most d and a weight by a factor e^(2 d) (its own and the sum's); the weights are rounded once, the
    sum of them at most by the same, and the n products with V are added with 2^-23 each."""
    B, S, _ = q.shape
    _, N, L, H = k.shape
    G = num_heads // N
    out = torch.zeros((B, S, num_heads, H), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    qh = q.view(B, S, num_heads, H)
    for b in range(B):
        for s in range(S):
            seen = visible(int(past[b]), S, L, s, None if prefix is None else int(prefix[b]),
                           None if docs is None else docs[b])
            idx = torch.from_numpy(np.nonzero(seen)[0]).to(q.device)
            if idx.numel() == 0:
                continue
            dist = (int(past[b]) + s - idx).abs().double()
            for n in range(N):
                kk, vv = k[b, n, idx], v[b, n, idx]
                rows = qh[b, s, n * G:(n + 1) * G]
                y = rows @ kk.T * scale
                size = rows.abs() @ kk.abs().T * abs(scale)
                d = (H + 8) * 2.0 ** -23 * size
                if cap:
                    d = d + 8 * 2.0 ** -23 * cap
                    y = cap * torch.tanh(y / cap)
                if slopes is not None:
                    y = y - slopes[n * G:(n + 1) * G, None].double() * dist
                    d = d + 4 * 2.0 ** -23 * slopes[n * G:(n + 1) * G, None].double() * dist
                d = d + 4 * 2.0 ** -23 * y.abs()
                p = torch.softmax(y, -1)
                off = p * torch.expm1(2 * d.clamp(max=50.0))
                mean = p @ vv.abs()
                c = 2 * weight_eps + (idx.numel() + 16) * 2.0 ** -23
                total = c * mean + off @ vv.abs() + off.sum(-1, keepdim=True) * mean
                # weights below the smallest normal value of a 16-bit type lose up to half its smallest step
                if weight_eps > 2.0 ** -20:
                    total = total + idx.numel() * 2.0 ** -25 * vv.abs().amax()
                out[b, s, n * G:(n + 1) * G] = p @ vv
                bound[b, s, n * G:(n + 1) * G] = total
    return out.view(B, S, -1), bound.view(B, S, -1)


def close(got, want, bound, what=""):
    T = got.dtype
    got = got.double()
    limit = want.abs() * EPS[T] + bound * (1 + EPS[T]) + SMALLEST[T]
    bad = ~((got - want).abs() <= limit)
    if bad.any():
        at = int(bad.flatten().nonzero()[0])
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} outside, first {at}: {got.flatten()[at]} against "
            f"{want.flatten()[at]}, limit {limit.flatten()[at]}")


# --------------------------------------------------------------------------
# e4m3 by its definition
# --------------------------------------------------------------------------

def e4m3_table():
    """The value of every code."""
    t = np.zeros(256)
    for c in range(256):
        sign, e, m = -1.0 if c & 128 else 1.0, (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        t[c] = sign * (math.nan if (c & 127) == 127 else x)
    return t


_VALUES = e4m3_table()
_POSITIVE = _VALUES[:127]


def e4m3(x):
    """Codes of float64 values: the nearest, of two equally near the even one; beyond 448: 448; NaN: NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(_POSITIVE, np.nan_to_num(a, nan=0.0)).clip(0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POSITIVE[lo], _POSITIVE[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.isnan(x), 127, code)
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def values(codes, scale):
    """Float64 values of 8-bit caches: codes uint8 (B, N, L, H), scale (B, N, ceil(L/16))."""
    by_row = np.repeat(scale.astype(np.float64), BLOCK, axis=2)[:, :, :codes.shape[2], None]
    return _VALUES[codes] * by_row


def scale_of(amax):
    if amax <= 0:
        return 2.0 ** -120
    s = 2.0 ** -120
    while s * 448.0 < amax:
        s *= 2.0
    return s


def append(codes, scale, new, past):
    """Rows new (B, S, N, H) float64 appended to codes and scale (numpy, in place)."""
    B, S, N, H = new.shape
    L = codes.shape[2]
    for b in range(B):
        p = int(past[b])
        for n in range(N):
            for blk in range(-(-L // BLOCK)):
                rows = [r for r in range(max(blk * BLOCK, p, 0), min((blk + 1) * BLOCK, p + S, L))]
                if not rows:
                    continue
                x = new[b, [r - p for r in rows], n]
                finite = np.abs(x[np.isfinite(x)])
                need = scale_of(finite.max() if finite.size else 0.0)
                if blk * BLOCK < p:
                    was = float(scale[b, n, blk])
                    need = max(need, was)
                    if need > was:
                        codes[b, n, blk * BLOCK:p] = e4m3(_VALUES[codes[b, n, blk * BLOCK:p]] * (was / need))
                codes[b, n, rows] = e4m3(x / need)
                scale[b, n, blk] = need
