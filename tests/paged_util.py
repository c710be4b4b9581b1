"""The paged-cache operators in 64 bits, for the tests: one sequence at a time, page by page."""

import numpy as np
import torch

import kv_util as ku


def rows_of(pages, table, count):
    """The first `count` rows (Nkv, count, H) float64 of the sequence with this row of the page table (a list).
    A page outside the pool holds zeros."""
    P, N, ps, H = pages.shape
    out = torch.zeros((N, count, H), dtype=torch.float64, device=pages.device)
    for i in range(-(-count // ps)):
        n = min(ps, count - i * ps)
        if 0 <= table[i] < P:
            out[:, i * ps:i * ps + n] = pages[table[i], :, :n].double()
    return out


def visible(past, n, total, s, window=0, word=None):
    """Truth values over the rows below `total`: what new token s sees."""
    i, j = past + s, np.arange(total)
    if word is None:
        seen = j <= i
        return seen & (j > i - window) if window else seen
    bit = j - past
    return (bit < 0) | ((bit < 64) & np.array([(int(word) >> min(max(int(b), 0), 63)) & 1 for b in bit], dtype=bool))


def attention(q, k_pages, v_pages, table, past, starts, num_heads, scale, cap=0.0, window=0, slopes=None, masks=None,
              weight_eps=0.0, most=None):
    """(out, bound, owned) for q (tokens, Nq*H): float64 tensors, and which tokens are some sequence's.

    The bound is kv_util.attention's, by the same count of roundings."""
    T = q.shape[0]
    N, ps, H = k_pages.shape[1:]
    G = num_heads // N
    out = torch.zeros((T, num_heads, H), dtype=torch.float64, device=q.device)
    bound = torch.zeros_like(out)
    owned = torch.zeros(T, dtype=torch.bool, device=q.device)
    qh = q.double().view(T, N, G, H)
    for b in range(len(past)):
        t0, n = starts[b], starts[b + 1] - starts[b]
        if n == 0 or (most is not None and n > most):
            continue
        owned[t0:t0 + n] = True
        total = max(0, min(past[b] + n, len(table[b]) * ps))
        if total == 0:
            continue
        k, v = (rows_of(x, table[b], total) for x in (k_pages, v_pages))
        seen = torch.from_numpy(np.stack([visible(past[b], n, total, s, window, None if masks is None else masks[t0 + s])
                                          for s in range(n)])).to(q.device)
        dist = (torch.arange(n, device=q.device)[:, None] + past[b] - torch.arange(total, device=q.device)).abs().double()
        for h in range(N):
            rows = qh[t0:t0 + n, h].transpose(0, 1)                      # (G, n, H)
            # what nobody sees may be NaN: it takes no part
            some = seen.any(0)
            kk = torch.where(some[:, None], k[h], 0.0)
            vv = torch.where(some[:, None], v[h], 0.0)
            y = rows @ kk.T * scale
            d = (H + 8) * 2.0 ** -23 * (rows.abs() @ kk.abs().T) * abs(scale)
            if cap:
                d = d + 8 * 2.0 ** -23 * cap
                y = cap * torch.tanh(y / cap)
            if slopes is not None:
                by = slopes[h * G:(h + 1) * G].double()[:, None, None] * dist
                y = y - by
                d = d + 4 * 2.0 ** -23 * by
            d = d + 4 * 2.0 ** -23 * y.abs()
            y = y.masked_fill(~seen, float("-inf"))
            p = torch.softmax(y, -1)
            p = torch.where(seen.any(1)[:, None], p, torch.zeros_like(p))
            off = torch.where(seen, p * torch.expm1(2 * d.clamp(max=50.0)), torch.zeros_like(p))
            mean = p @ vv.abs()
            count = seen.sum(1).double()[:, None]
            c = 2 * weight_eps + (count + 16) * 2.0 ** -23
            total_off = c * mean + off @ vv.abs() + off.sum(-1, keepdim=True) * mean
            if weight_eps > 2.0 ** -20:
                total_off = total_off + count * 2.0 ** -25 * vv.abs().amax()
            out[t0:t0 + n, h * G:(h + 1) * G] = (p @ vv).transpose(0, 1)
            bound[t0:t0 + n, h * G:(h + 1) * G] = total_off.transpose(0, 1)
    return out.view(T, -1), bound.view(T, -1), owned


def random_trees(sizes, rng):
    """(masks, depths): a random tree for each size, node 0 its root."""
    masks, depths = [], []
    for n in sizes:
        word, depth = [], []
        for i in range(n):
            parent = int(rng.integers(max(0, i - 5), i)) if i else -1
            word.append((word[parent] if i else 0) | 1 << i)
            depth.append(depth[parent] + 1 if i else 0)
        masks += [w - (1 << 64) if w >> 63 else w for w in word]
        depths += depth
    return masks, depths


def table_for(rng, lengths, ps, pages=None, width=None):
    """(page table as lists, pages of the pool): each sequence's pages in no order; behind them junk that must
    not be looked at."""
    held = [max(0, -(-n // ps)) for n in lengths]
    pages = max(1, sum(held) + 2) if pages is None else pages
    order = rng.permutation(pages).tolist()
    width = max(held + [1]) if width is None else width
    rows, at = [], 0
    for n in held:
        rows.append(order[at:at + n] + [int(x) for x in rng.integers(-2 ** 31, 2 ** 31 - 1, width - n)])
        at += n
    return rows, pages


def close(got, want, bound, what=""):
    ku.close(got, want, bound, what)
