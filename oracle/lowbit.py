"""Plain float64 forms of the low-bit serving operators: pages for a growing
batch, the 8-bit paged KV cache, the linear layer with 4-bit weights.

TEST INFRASTRUCTURE ONLY: see the package docstring.
"""

import math

import numpy as np

from .fp8 import E4M3_MAX, e4m3_decode

PAGE = 16
OK, CAPACITY, BAD_PAGE, BAD_INPUT = 0, 1, 2, 3

_GRID = e4m3_decode(np.arange(127, dtype=np.uint8))   # the finite magnitudes by code


def e4m3_encode(x):
    """Nearest E4M3 code of each float64 (ties to the even code), magnitudes past 448 saturate, NaN -> 0x7F."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(np.where(np.isnan(x), 0.0, x)), E4M3_MAX)
    hi = np.clip(np.searchsorted(_GRID, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    up, down = _GRID[hi] - a, a - _GRID[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = code | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def kv8_scale(x):
    """The smallest power of two (2^-126 at least) under which the finite values of x are at most 448."""
    x = np.abs(np.asarray(x, dtype=np.float64))
    top = x[np.isfinite(x)].max(initial=0.0)
    s = 2.0 ** -126
    if top > 0:
        s = max(s, 2.0 ** (math.frexp(top)[1] - 9))
        while top > E4M3_MAX * s:
            s *= 2
    return s


def kv8_append(k, v, seq_lens, rows, page_table, k_codes, v_codes, k_scale, v_scale):
    """New rows k, v [B, n, nkv, hd] into copies of the cache; returns the four arrays and status [B]."""
    num_pages, nkv = k_codes.shape[:2]
    out = [a.copy() for a in (k_codes, v_codes, k_scale, v_scale)]
    status = np.zeros(len(seq_lens), dtype=np.int32)
    for b, S in enumerate(map(int, seq_lens)):
        n = k.shape[1] if rows is None else int(rows[b])
        if S < 0 or n < 0 or n > k.shape[1]:
            status[b] = BAD_INPUT
            continue
        if S + n > page_table.shape[1] * PAGE:
            status[b] = CAPACITY
            continue
        pages = list(range(S // PAGE, -(-(S + n) // PAGE))) if n else []
        if any(not 0 <= int(page_table[b, p]) < num_pages for p in pages):
            status[b] = BAD_PAGE
            continue
        for p in pages:
            at = int(page_table[b, p])
            for x, codes, scale in ((k, out[0], out[2]), (v, out[1], out[3])):
                for h in range(nkv):
                    e0, e1 = max(S, p * PAGE), min(S + n, (p + 1) * PAGE)
                    new = np.asarray(x[b, e0 - S:e1 - S, h], dtype=np.float64)
                    s = kv8_scale(new)
                    old = e0 - p * PAGE
                    if old and scale[at, h] >= s:
                        s = float(scale[at, h])
                    elif old:
                        had = e4m3_decode(codes[at, h, :old]) * float(scale[at, h])
                        codes[at, h, :old] = e4m3_encode(had / s)
                    codes[at, h, old:e1 - p * PAGE] = e4m3_encode(new / s)
                    scale[at, h] = s
    return (*out, status)


def attention_kv8(q, seq_lens, rows, page_table, k_codes, v_codes, k_scale, v_scale, scale):
    """(out [B, K, nq, hd], status [B], weight) with weight[b, j, h] = sum_e w_e |v_e| / sum_e w_e, the size that
    errors of the weights are relative to."""
    B, K, nq, hd = q.shape
    num_pages, nkv = k_codes.shape[:2]
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    status = np.zeros(B, dtype=np.int32)
    for b in range(B):
        S, n = int(seq_lens[b]), K if rows is None else int(rows[b])
        if S < 0 or n < 0 or n > K:
            status[b] = BAD_INPUT
            continue
        if S + n > page_table.shape[1] * PAGE:
            status[b] = CAPACITY
            continue
        if n == 0:
            continue
        ids = page_table[b, :-(-(S + n) // PAGE)]
        if ((ids < 0) | (ids >= num_pages)).any():
            status[b] = BAD_PAGE
            continue
        kk = e4m3_decode(k_codes[ids]) * k_scale[ids].astype(np.float64)[:, :, None, None]
        vv = e4m3_decode(v_codes[ids]) * v_scale[ids].astype(np.float64)[:, :, None, None]
        for h in range(nq):
            g = h * nkv // nq
            ke, ve = kk[:, g].reshape(-1, hd), vv[:, g].reshape(-1, hd)
            for j in range(n):
                seen = slice(0, S + j + 1)
                x = scale * (ke[seen] @ np.asarray(q[b, j, h], dtype=np.float64))
                w = np.exp(x - x.max())
                w /= w.sum()
                out[b, j, h] = w @ ve[seen]
                size[b, j, h] = w @ np.abs(ve[seen])
    return out, status, size


def unpack_w4(codes, scale, zeros, group):
    """(W [M, Kd] float64, |c| s + z s [M, Kd]: what rounding errors of a product with it are relative to)."""
    M, half = codes.shape
    c = np.empty((M, 2 * half))
    c[:, 0::2], c[:, 1::2] = codes & 15, codes >> 4
    s = np.repeat(np.asarray(scale, dtype=np.float64), group, axis=1)[:, :2 * half]
    z = 8.0 if zeros is None else np.repeat(zeros.astype(np.float64), group, axis=1)[:, :2 * half]
    return (c - z) * s, (c + z) * np.abs(s)


def assign_pages(seq_lens, new_lens, counts, table, free, free_count, num_pages, n_max):
    """(slot_mapping, counts, table, free_count, status) after each request in turn has taken its pages."""
    B, max_pages = table.shape
    table, counts = table.copy(), counts.copy()
    slots = np.full((B, n_max), -1, dtype=np.int32)
    status = np.zeros(B, dtype=np.int32)
    left = max(0, min(int(free_count), len(free)))
    dry = False
    for b in range(B):
        S, n, c = int(seq_lens[b]), int(new_lens[b]), int(counts[b])
        if S < 0 or n < 0 or n > n_max or c < 0 or c > max_pages or S > c * PAGE:
            status[b] = BAD_INPUT
            continue
        need = -(-(S + n) // PAGE)
        if need > max_pages:
            status[b] = CAPACITY
            continue
        grow = max(0, need - c)
        if grow and (dry or grow > left):
            dry = True
            status[b] = CAPACITY
            continue
        for i in range(grow):
            left -= 1
            table[b, c + i] = free[left]
        counts[b] = c + grow
        ids = [int(table[b, (S + i) // PAGE]) for i in range(n)]
        if any(not 0 <= p < num_pages for p in ids):
            status[b] = BAD_PAGE
            continue
        slots[b, :n] = [p * PAGE + (S + i) % PAGE for i, p in enumerate(ids)]
    return slots, counts, table, left, status


def release_pages(keep_lens, counts, table, free, free_count, num_pages):
    """(counts, table, free, free_count, status) after each request in turn has given back its pages."""
    B, max_pages = table.shape
    table, counts, free = table.copy(), counts.copy(), free.copy()
    status = np.zeros(B, dtype=np.int32)
    have = max(0, min(int(free_count), len(free)))
    full = False
    for b in range(B):
        n, c = int(keep_lens[b]), int(counts[b])
        if n < 0 or c < 0 or c > max_pages or n > c * PAGE:
            status[b] = BAD_INPUT
            continue
        keep = -(-n // PAGE)
        ids = table[b, keep:c].copy()
        if ((ids < 0) | (ids >= num_pages)).any():
            status[b] = BAD_PAGE
            continue
        if len(ids) and (full or have + len(ids) > len(free)):
            full = True
            status[b] = CAPACITY
            continue
        free[have:have + len(ids)] = ids
        have += len(ids)
        table[b, keep:c] = -1
        counts[b] = keep
    return counts, table, free, have, status
