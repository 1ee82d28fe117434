"""Plain float64 forms of the operators around the 4-bit paged KV cache: its
write with the position rotation, the attention over it, and the log
probabilities of given tokens.

TEST INFRASTRUCTURE ONLY: see the package docstring.
"""

import numpy as np

from .lowbit import BAD_INPUT, BAD_PAGE, CAPACITY, PAGE


def bf16(x):
    """The nearest bf16 value of each float64 (ties to even), as float64."""
    x = np.asarray(x, dtype=np.float64)
    m, e = np.frexp(x)
    step = np.exp2(np.maximum(e, -125).astype(np.float64) - 8)
    with np.errstate(invalid="ignore"):
        y = np.rint(x / step) * step
    return np.where(np.isfinite(x), np.where(np.abs(y) > 3.3895313892515355e38, np.copysign(np.inf, x), y), x)


def rotate(x, position, theta):
    """Row x [..., hd] at a position: dimensions i and i + hd/2 turned by position * theta^(-2i/hd)."""
    x = np.asarray(x, dtype=np.float64)
    if theta == 0:
        return x
    half = x.shape[-1] // 2
    angle = position * float(theta) ** (-np.arange(half, dtype=np.float64) / half)
    c, s = np.cos(angle), np.sin(angle)
    a, b = x[..., :half], x[..., half:]
    return np.concatenate([a * c - b * s, b * c + a * s], axis=-1)


def quantise(x):
    """(codes [..., hd] 0..15, scale [...], base [...], quotient (x - base) / scale before it is rounded)."""
    x = np.asarray(x, dtype=np.float64)
    whole = np.isfinite(x).all(-1)
    y = np.where(whole[..., None], x, 0.0)
    base = bf16(y.min(-1))
    scale = bf16(np.maximum(y.max(-1) - base, 0) / 15)
    part = (y - base[..., None]) / np.where(scale > 0, scale, 1.0)[..., None]
    part = np.where((scale > 0)[..., None], part, 0.0)
    codes = np.clip(np.rint(part), 0, 15).astype(np.uint8)
    return codes, np.where(whole, scale, np.nan), np.where(whole, base, np.nan), part


def pack(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpack(packed):
    return np.stack([packed & 15, packed >> 4], axis=-1).reshape(*packed.shape[:-1], -1)


def request(S, n, n_max, max_pages, num_pages, row, first=0):
    """(status, pages that the n new rows fall into) of a request."""
    if S < 0 or n < 0 or n > n_max or first < 0 or first + n > 2 ** 31 - 1:
        return BAD_INPUT, []
    if S + n > max_pages * PAGE:
        return CAPACITY, []
    pages = list(range(S // PAGE, -(-(S + n) // PAGE))) if n else []
    if any(not 0 <= int(row[p]) < num_pages for p in pages):
        return BAD_PAGE, []
    return 0, pages


def append(q, k, v, seq_lens, rows, positions, theta, page_table, num_pages):
    """What is written: a list of (side, page, head, slot, codes, scale, base, part), q turned (zero where there is
    no row; None without q) and status [B]."""
    B, n_max = k.shape[:2]
    out = None if q is None else np.zeros(q.shape)
    status, wrote = np.zeros(B, dtype=np.int32), []
    for b in range(B):
        S, n = int(seq_lens[b]), n_max if rows is None else int(rows[b])
        first = S if positions is None else int(positions[b])
        status[b], _ = request(S, n, n_max, page_table.shape[1], num_pages, page_table[b], first if theta else 0)
        if status[b]:
            continue
        for j in range(n):
            at, slot = int(page_table[b, (S + j) // PAGE]), (S + j) % PAGE
            if q is not None:
                out[b, j] = rotate(q[b, j], first + j, theta)
            for side, x in ((0, rotate(k[b, j], first + j, theta)), (1, v[b, j])):
                codes, scale, base, part = quantise(x)
                for h in range(k.shape[2]):
                    wrote.append((side, at, h, slot, codes[h], scale[h], base[h], part[h]))
    return wrote, out, status


def values(codes, params):
    """(values [..., hd], |scale| |n - 8| + |base + 8 scale|: what roundings of them are relative to)."""
    n, s, b = unpack(codes).astype(np.float64), params[..., :1].astype(np.float64), params[..., 1:].astype(np.float64)
    return b + s * n, np.abs(s * (n - 8)) + np.abs(b + 8 * s)


def attention(q, seq_lens, rows, page_table, codes, params, scale):
    """(out, status, size, reach): size = sum_e w |v|' / sum_e w and reach the largest scale |q| . |k|' that a row
    meets, with |x|' as `values` has it. codes, params: of K and V."""
    B, K, nq, hd = q.shape
    num_pages, nkv = codes[0].shape[:2]
    out, size, reach = np.zeros(q.shape), np.zeros(q.shape), np.zeros((B, K, nq))
    status = np.zeros(B, dtype=np.int32)
    for b in range(B):
        S, n = int(seq_lens[b]), K if rows is None else int(rows[b])
        status[b], _ = request(S, n, K, page_table.shape[1], num_pages, page_table[b])
        if status[b] or n == 0:
            continue
        ids = page_table[b, :-(-(S + n) // PAGE)]
        if ((ids < 0) | (ids >= num_pages)).any():
            status[b] = BAD_PAGE
            continue
        (kk, ka), (vv, va) = (values(c[ids], p[ids]) for c, p in zip(codes, params))
        for h in range(nq):
            g = h * nkv // nq
            flat = lambda x: x[:, g].reshape(-1, hd)
            for j in range(n):
                seen = slice(0, S + j + 1)
                row = np.asarray(q[b, j, h], dtype=np.float64)
                x = scale * (flat(kk)[seen] @ row)
                w = np.exp(x - x.max())
                w /= w.sum()
                out[b, j, h] = w @ flat(vv)[seen]
                size[b, j, h] = w @ flat(va)[seen]
                reach[b, j, h] = abs(scale) * (flat(ka)[seen] @ np.abs(row)).max()
    return out, status, size, reach


def token_logprobs(logits, tokens, top, temperature):
    """(logprobs [R], entropy [R], top_tokens [R, top], top_logprobs [R, top])."""
    x = np.asarray(logits, dtype=np.float64)
    R, V = x.shape
    with np.errstate(all="ignore"):
        y = (x - x.max(1, keepdims=True)) / temperature
        e = np.exp(y)
        z = e.sum(1)
        p = y - np.log(z)[:, None]
        h = np.log(z) - np.where(e > 0, e * y, e).sum(1) / z
    at = np.array([p[r, t] if 0 <= t < V else np.nan for r, t in enumerate(np.asarray(tokens))])
    # NaN behind everything, then by value, then by index
    order = np.lexsort((np.broadcast_to(np.arange(V), x.shape), -np.where(np.isnan(x), 0, x), np.isnan(x)), axis=1)[:, :top]
    return at, h, order, np.take_along_axis(p, order, axis=1)
