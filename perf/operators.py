"""Cases of the low-bit serving operators: pages for a growing batch, the 8-bit paged KV cache's write and
attention, and the linear layer with 4-bit weights.

Four operators, picked by a case's "op":

  pages    a batch of requests grows by new_lens entries each: pages are taken from a stack of free ones and put into
           the page table, and every new entry gets its physical slot
  append   new key and value rows are stored in a paged cache of E4M3 codes with one scale for each (page, head)
  attend   grouped-query attention of K rows per request over that cache
  linear   y = x W^T with 4-bit weights and a scale (and a zero point) for each group of columns

`run` computes them in their plain form, or, where `own` is true, with the calls of the package.
"""

import math

import torch

own = False

PAGE = 16          # cache entries in a page
E4M3_MAX = 448.0   # largest E4M3 value


# ---------------------------------------------------------------- cases

def listed():
    return [
        # every decoding step of a busy server: each request gets room for its next eight drafts
        dict(name="pages step", op="pages", B=64, lo=16, hi=4096, n_max=8, max_pages=512),
        # a wave of prompts is admitted at once
        dict(name="pages prompts", op="pages", B=256, lo=0, hi=0, n_max=2048, max_pages=256),
        # a draft pass of 32 requests writes its rows behind the committed entries
        dict(name="append drafts", op="append", B=32, nkv=4, hd=128, lo=0, hi=511, n_max=8, ragged=False),
        # prompts of up to 2048 tokens, ragged, are stored in one call
        dict(name="append prompts", op="append", B=8, nkv=8, hd=64, lo=0, hi=40, n_max=2048, ragged=True),
        # the draft pass of a single user: latency counts
        dict(name="attend B1 K7", op="attend", B=1, K=7, nq=32, nkv=4, hd=128, lo=2048, hi=2048, ragged=False),
        # a decoding step of single tokens over a ragged batch
        dict(name="attend B64 tokens", op="attend", B=64, K=1, nq=32, nkv=4, hd=128, lo=512, hi=8192, ragged=False),
        # the draft pass of a full server, 88 query rows for each KV head
        dict(name="attend B128 K11", op="attend", B=128, K=11, nq=32, nkv=4, hd=128, lo=512, hi=8192, ragged=False),
        # 64-wide heads, some rows of each request padded away
        dict(name="attend hd64 K10", op="attend", B=64, K=10, nq=64, nkv=8, hd=64, lo=1024, hi=4096, ragged=True),
        # one user with a long document: the cache is split over the whole card
        dict(name="attend long", op="attend", B=1, K=1, nq=32, nkv=4, hd=128, lo=131072, hi=131072, ragged=False),
        # the output projection for one token
        dict(name="linear one row", op="linear", M=2048, N=1, Kd=4096, group=128, zeros=False, scale="bf16"),
        # the gate projection for the rows of one draft pass, asymmetric codes in small groups
        dict(name="linear draft rows", op="linear", M=6144, N=11, Kd=2048, group=32, zeros=True, scale="bf16"),
        # the LM head for the rows of one draft pass
        dict(name="linear LM head", op="linear", M=151936, N=8, Kd=2048, group=128, zeros=False, scale="f32"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["pages", "append", "attend", "attend", "linear", "linear"])
    if op == "pages":
        if rng.random() < 0.5:
            hi = _log(rng, 16, 8192)
            n_max = _log(rng, 1, 32)
            lo = rng.randint(0, hi)
        else:
            lo, hi, n_max = 0, rng.randint(0, 40), _log(rng, 33, 2048)
        max_pages = -(-(hi + n_max) // PAGE) + rng.randint(0, 40)
        return dict(op=op, B=_log(rng, 1, 256), lo=lo, hi=hi, n_max=n_max, max_pages=max_pages)
    if op == "append":
        hd = rng.choice([64, 128])
        if rng.random() < 0.6:
            B, n_max, hi = _log(rng, 1, 128), rng.randint(1, 16), rng.randint(0, 600)
        else:
            B, n_max, hi = rng.randint(1, 8), _log(rng, 17, 2048), rng.randint(0, 40)
        return dict(op=op, B=B, nkv=rng.choice([1, 2, 4, 8]), hd=hd, lo=rng.randint(0, hi), hi=hi, n_max=n_max,
                    ragged=rng.random() < 0.5)
    if op == "attend":
        hd = rng.choice([64, 128])
        nkv = rng.choice([1, 2, 4, 8])
        G = rng.choice([1, 2, 4, 5, 8, 16])
        K = rng.randint(1, min(16, 128 // G)) if rng.random() < 0.6 else 1
        B = _log(rng, 1, 128)
        # entries of all requests together stay below those of the largest listed case
        top = max(64, min(131072, 8192 * 40 * 4 // (B * nkv)))
        hi = _log(rng, 8, top)
        lo = hi if rng.random() < 0.3 else _log(rng, 1, hi) - 1
        return dict(op=op, B=B, K=K, nq=nkv * G, nkv=nkv, hd=hd, lo=lo, hi=hi, ragged=rng.random() < 0.4)
    group = rng.choice([32, 64, 128])
    Kd = 32 * _log(rng, 4, 270)
    M = _log(rng, 256, 9000) if rng.random() < 0.7 else _log(rng, 9000, 150000)
    while M * Kd > 151936 * 2048:
        M //= 2
    return dict(op=op, M=M, N=rng.choice([1, 1, 2, 3, 5, 7, 8, 11, 16]), Kd=Kd, group=group,
                zeros=rng.random() < 0.5, scale=rng.choice(["bf16", "f32"]))


# ---------------------------------------------------------------- inputs

def _lens(c):
    """The requests' lengths: evenly spread from lo to hi, so that their sum depends on the case alone."""
    B = c["B"]
    return [c["lo"] + (c["hi"] - c["lo"]) * b // max(1, B - 1) for b in range(B)] if B > 1 else [c["hi"]]


def _rows(c, n):
    """New rows of each request: n, or from none to n where the case is ragged."""
    return [(7 * b + n) % (n + 1) if c["ragged"] and b else n for b in range(c["B"])]


def _perm(n, g):
    return torch.randperm(n, generator=g, device="cuda")


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(need, max_pages, g, free=0):
    """A page table of randomly placed pages, -1 where a request has none, the number of pages in all and the free
    ones; where none are asked for, the last page belongs to nobody."""
    total, spare = int(sum(need)), max(1, free)
    n = torch.tensor(need, device="cuda")
    ids = _perm(total + free, g).to(torch.int32)
    ids = ids if free else torch.cat([ids, _i32([total])])
    at = torch.arange(max_pages, device="cuda")[None, :]
    first = (n.cumsum(0) - n)[:, None]
    table = torch.where(at < n[:, None], ids[(first + at).clamp_max(total + spare - 1)], -1)
    return table.contiguous(), total + spare, ids[total:].contiguous()


def _pow2_scale(amax):
    """The smallest power of two s with amax <= 448 s (2^-126 at least), for float32 amax >= 0."""
    m, e = torch.frexp(amax)
    k = torch.where(m > 0.875, e - 8, e - 9).clamp(-126, 120)
    k = torch.where(amax > 0, k, torch.full_like(k, -126))
    return torch.ldexp(torch.ones_like(amax), k)


def _cache(pages, nkv, hd, g):
    """Random codes with a scale for each (page, head), and the odd page of larger values."""
    x = torch.randn(pages, nkv, PAGE, hd, generator=g, device="cuda")
    x *= 1.0 + 3.0 * (torch.rand(pages, nkv, 1, 1, generator=g, device="cuda") < 0.05)
    s = _pow2_scale(x.abs().amax(dim=(2, 3)))
    return (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c, op = case, case["op"]
    if op == "pages":
        S = _lens(c)
        order = _perm(c["B"], g)
        need = [-(-s // PAGE) for s in S]
        grow = c["B"] * (-(-c["n_max"] // PAGE) + 1)
        table, num_pages, free = _table(need, c["max_pages"], g, grow)
        new = torch.randint(max(1, c["n_max"] // 2), c["n_max"] + 1, (c["B"],), generator=g, device="cuda")
        return dict(c=c, seq_lens=_i32(S)[order], new_lens=new.to(torch.int32), page_counts=_i32(need)[order],
                    page_table=table[order].contiguous(), free_pages=free, free_count=_i32([free.numel()]),
                    num_pages=num_pages)
    if op == "append":
        B, n, nkv, hd = c["B"], c["n_max"], c["nkv"], c["hd"]
        S, rows = _lens(c), _rows(c, c["n_max"])
        need = [-(-(s + r) // PAGE) for s, r in zip(S, rows)]
        table, num_pages, _ = _table(need, max(1, max(need)), g)
        kc, ks = _cache(num_pages, nkv, hd, g)
        vc, vs = _cache(num_pages, nkv, hd, g)
        # keys and values are columns of a fused projection's output, as in a decoder layer
        qkv = torch.randn(B, n, 4 * nkv * hd, generator=g, device="cuda")
        qkv *= 1.0 + 4.0 * (torch.rand(B, n, 1, generator=g, device="cuda") < 0.1)
        qkv = qkv.to(torch.bfloat16)
        k = qkv[..., 2 * nkv * hd:3 * nkv * hd].unflatten(-1, (nkv, hd))
        v = qkv[..., 3 * nkv * hd:].unflatten(-1, (nkv, hd))
        return dict(c=c, k=k, v=v, seq_lens=_i32(S), rows=_i32(rows), page_table=table, kc=kc, vc=vc, ks=ks, vs=vs)
    if op == "attend":
        B, K, nq, nkv, hd = c["B"], c["K"], c["nq"], c["nkv"], c["hd"]
        S, rows = _lens(c), _rows(c, c["K"])
        order = _perm(B, g).tolist()
        S, rows = [S[i] for i in order], [rows[i] for i in order]
        need = [-(-(s + K) // PAGE) for s in S]
        table, num_pages, _ = _table(need, max(need), g)
        kc, ks = _cache(num_pages, nkv, hd, g)
        vc, vs = _cache(num_pages, nkv, hd, g)
        q = (1.5 * torch.randn(B, K, nq, hd, generator=g, device="cuda")).to(torch.bfloat16)
        return dict(c=c, q=q, seq_lens=_i32(S), rows=_i32(rows) if c["ragged"] else None, page_table=table, kc=kc,
                    vc=vc, ks=ks, vs=vs)
    M, N, Kd, group = c["M"], c["N"], c["Kd"], c["group"]
    ng = -(-Kd // group)
    w = torch.randint(0, 256, (M, Kd // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = (0.5 + torch.rand(M, ng, generator=g, device="cuda")) * (0.3 / math.sqrt(Kd))
    s = s.to(torch.bfloat16) if c["scale"] == "bf16" else s
    z = torch.randint(5, 12, (M, ng), generator=g, device="cuda", dtype=torch.uint8) if c["zeros"] else None
    x = torch.randn(N, Kd, generator=g, device="cuda").to(torch.bfloat16)
    return dict(c=c, w=w, s=s, z=z, x=x)


# ---------------------------------------------------------------- one pass

def run(state):
    op = state["c"]["op"]
    if own:
        return _own(state)
    return {"pages": _pages, "append": _append, "attend": _attend, "linear": _linear}[op](state)


def _own(st):
    from speculative_drafting_pe_gb300 import binding
    op = st["c"]["op"]
    if op == "pages":
        o = binding.assign_pages(st["seq_lens"], st["new_lens"], st["page_counts"], st["page_table"],
                                 st["free_pages"], st["free_count"], st["num_pages"], st["c"]["n_max"])
        return [st["page_table"], o["slot_mapping"], o["page_counts"], o["free_count"], o["status"]]
    if op == "append":
        status = binding.kv8_append(st["k"], st["v"], st["seq_lens"], st["page_table"], st["kc"], st["vc"], st["ks"],
                                    st["vs"], rows=st["rows"])
        return [st["kc"].view(torch.float8_e4m3fn), st["vc"].view(torch.float8_e4m3fn), st["ks"], st["vs"], status]
    if op == "attend":
        return list(binding.attention_kv8(st["q"], st["seq_lens"], st["page_table"], st["kc"], st["vc"], st["ks"],
                                          st["vs"], rows=st["rows"]))
    return binding.linear_w4(st["w"], st["s"], st["x"], st["c"]["group"], zeros=st["z"])


def _pages(st):
    S, n, count, table = st["seq_lens"].long(), st["new_lens"].long(), st["page_counts"].long(), st["page_table"]
    free, num_pages, max_pages, n_max = st["free_pages"].long(), st["num_pages"], table.shape[1], st["c"]["n_max"]
    have = st["free_count"].long()
    need = (S + n + PAGE - 1) // PAGE
    bad = (S < 0) | (n < 0) | (n > n_max) | (count < 0) | (count > max_pages) | (count * PAGE < S)
    full = ~bad & (need > max_pages)
    grow = torch.where(bad | full, 0, (need - count).clamp_min(0))
    upto = grow.cumsum(0)
    short = (grow > 0) & (upto > have)
    take = torch.where(short, 0, grow)
    # page i of the table, where it is new: the next one down the stack
    i = torch.arange(max_pages, device=S.device)[None, :]
    nth = (upto - grow)[:, None] + i - count[:, None]
    new = (i >= count[:, None]) & (i < (count + take)[:, None])
    table.copy_(torch.where(new, free[(have - 1 - nth).clamp(0, free.numel() - 1)], table))
    e = S[:, None] + torch.arange(n_max, device=S.device)[None, :]
    page = torch.gather(table.long(), 1, (e // PAGE).clamp(0, max_pages - 1))
    live = torch.arange(n_max, device=S.device)[None, :] < n[:, None]
    ok = ~(bad | full | short)
    lost = (ok[:, None] & live & ((page < 0) | (page >= num_pages))).any(1)
    slots = torch.where((ok & ~lost)[:, None] & live, page * PAGE + e % PAGE, -1)
    status = torch.where(bad, 3, torch.where(full | short, 1, torch.where(lost, 2, 0)))
    i32 = torch.int32
    return [table, slots.to(i32), (count + take).to(i32), (have - take.sum()).to(i32), status.to(i32)]


def _append(st):
    S, rows, table = st["seq_lens"].long(), st["rows"].long(), st["page_table"].long()
    n = st["c"]["n_max"]
    P = (n + PAGE - 2) // PAGE + 1
    # the pages that the new rows fall into, and the row that falls on each of their entries
    pages = (S // PAGE)[:, None] + torch.arange(P, device=S.device)[None, :]
    entry = pages[:, :, None] * PAGE + torch.arange(PAGE, device=S.device)
    row = entry - S[:, None, None]
    fresh = (row >= 0) & (row < rows[:, None, None])
    old = row < 0
    hit = fresh.any(2)
    # the cache's last page belongs to nobody: it stands in for pages without a new row, and keeps what it has
    at = torch.where(hit, torch.gather(table, 1, pages.clamp_max(table.shape[1] - 1)), st["kc"].shape[0] - 1).view(-1)
    b = torch.arange(S.shape[0], device=S.device)[:, None, None]
    old = (old & hit[:, :, None]).view(-1, 1, PAGE, 1)
    pick, hit, fresh = (b, row.clamp(0, n - 1)), hit.view(-1, 1), fresh.view(-1, 1, PAGE, 1)
    for x, codes, scale in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
        new = torch.where(fresh, x[pick].flatten(0, 1).transpose(1, 2).float(), 0)
        had = codes[at].view(torch.float8_e4m3fn).float()
        s = _pow2_scale(new.abs().amax(dim=(2, 3)))
        s = torch.where(old.any(2)[:, :, 0], torch.maximum(s, scale[at]), torch.where(hit, s, scale[at]))
        s4 = s[:, :, None, None]
        kept = torch.where(old, had * scale[at][:, :, None, None], new) / s4
        put = torch.where(fresh | old, kept.clamp(-E4M3_MAX, E4M3_MAX), had)
        codes[at] = put.to(torch.float8_e4m3fn).view(torch.uint8)
        scale[at] = s
    status = torch.zeros(S.shape[0], dtype=torch.int32, device=S.device)
    return [st["kc"].view(torch.float8_e4m3fn), st["vc"].view(torch.float8_e4m3fn), st["ks"], st["vs"], status]


def _attend(st):
    c, q, table = st["c"], st["q"], st["page_table"].long().clamp_min(0)
    B, K, nq, nkv, hd = c["B"], c["K"], c["nq"], c["nkv"], c["hd"]
    S = st["seq_lens"].long()
    L, G = table.shape[1] * PAGE, nq // nkv
    last = S[:, None] + torch.arange(K, device=S.device)
    sees = torch.arange(L, device=S.device)[None, None, :] <= last[:, :, None]
    if st["rows"] is not None:
        sees = sees & (torch.arange(K, device=S.device)[None, :] < st["rows"][:, None])[:, :, None]

    def values(codes, scale):
        x = codes[table].view(torch.float8_e4m3fn).float() * scale[table][..., None, None]
        return x.transpose(1, 2).reshape(B, nkv, L, hd)

    k = values(st["kc"], st["ks"])
    rows = q.float().view(B, K, nkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, nkv, K * G, hd)
    s = torch.matmul(rows, k.transpose(2, 3)) / math.sqrt(hd)
    del k
    m = sees[:, None, :, None, :].expand(B, nkv, K, G, L).reshape(B, nkv, K * G, L)
    s = torch.where(m, s, -math.inf)
    top = s.amax(dim=3, keepdim=True)
    w = torch.exp(s - torch.where(top > -math.inf, top, 0))
    total = w.sum(dim=3, keepdim=True)
    v = values(st["vc"], st["vs"])
    # entries behind a request's last are not its own
    v = torch.where((torch.arange(L, device=S.device)[None, :] < (S + K)[:, None])[:, None, :, None], v, 0)
    o = torch.matmul(w, v) / torch.where(total > 0, total, 1)
    o = o.view(B, nkv, K, G, hd).permute(0, 2, 1, 3, 4).reshape(B, K, nq, hd)
    return [o.to(torch.bfloat16), torch.zeros(B, dtype=torch.int32, device=S.device)]


def _linear(st):
    c, w = st["c"], st["w"]
    M, Kd, group = c["M"], c["Kd"], c["group"]
    code = torch.stack([w & 15, w >> 4], dim=2).view(M, Kd).float()
    scale = st["s"].float().repeat_interleave(group, dim=1)[:, :Kd]
    zero = 8.0 if st["z"] is None else st["z"].float().repeat_interleave(group, dim=1)[:, :Kd]
    return torch.matmul(st["x"].float(), ((code - zero) * scale).t())


# ---------------------------------------------------------------- bytes and operations

def work(case):
    c, op = case, case["op"]
    if op == "pages":
        B, S = c["B"], _lens(c)
        n = (max(1, c["n_max"] // 2) + c["n_max"]) / 2
        grown = sum(max(0.0, (s % PAGE + n) / PAGE - (1 if s % PAGE else 0)) for s in S)
        # lengths, counts and status; each taken page read and put into the table; the slots
        return dict(bytes=4.0 * (5 * B + 2 * grown + B * c["n_max"]), flops=0.0)
    if op == "append":
        S, rows = _lens(c), _rows(c, c["n_max"])
        row = c["nkv"] * c["hd"]
        pages = sum(-(-(s + r) // PAGE) - s // PAGE for s, r in zip(S, rows) if r)
        old = sum(s % PAGE for s, r in zip(S, rows) if r)
        return dict(bytes=2.0 * (sum(rows) * row * 3 + old * row + pages * c["nkv"] * 4) + 4.0 * (3 * c["B"] + pages),
                    flops=4.0 * sum(rows) * row)
    if op == "attend":
        S, rows = _lens(c), _rows(c, c["K"])
        live = [s + r for s, r in zip(S, rows) if r]
        entries = sum(live)
        pages = sum(-(-n // PAGE) for n in live)
        q = 2 * 2 * sum(rows) * c["nq"] * c["hd"]
        seen = sum(r * s + r * (r + 1) // 2 for s, r in zip(S, rows))
        return dict(bytes=2.0 * entries * c["nkv"] * c["hd"] + 8.0 * pages * c["nkv"] + 4.0 * pages + q + 12.0 * c["B"],
                    flops=4.0 * seen * c["nq"] * c["hd"])
    M, N, Kd = c["M"], c["N"], c["Kd"]
    ng = -(-Kd // c["group"])
    return dict(bytes=M * Kd / 2 + M * ng * ((2 if c["scale"] == "bf16" else 4) + (1 if c["zeros"] else 0)) +
                2.0 * N * Kd + 4.0 * N * M, flops=2.0 * M * N * Kd)


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    if case["op"] == "pages":
        return None   # whole numbers
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "linear": _exact_linear}[case["op"]](st)


def _e4m3_grid():
    """The 127 finite E4M3 values from 0 up."""
    return torch.tensor([m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10) for e in range(16) for m in range(8)
                         if (e, m) != (15, 7)], dtype=torch.float64, device="cuda")


def _nearest_e4m3(x):
    """x (float64) rounded to the nearest E4M3 value, ties to the even code."""
    grid = _e4m3_grid()
    a = x.abs().clamp_max(E4M3_MAX)
    hi = torch.searchsorted(grid, a).clamp(0, 126)
    lo = (hi - 1).clamp_min(0)
    up, down = grid[hi] - a, a - grid[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    return grid[code].copysign(x)


def _exact_append(st):
    out = []
    S, rows, table = st["seq_lens"].tolist(), st["rows"].tolist(), st["page_table"].tolist()
    for x, codes, scale in ((st["k"], st["kc"], st["ks"]), (st["v"], st["vc"], st["vs"])):
        vals, scales = codes.view(torch.float8_e4m3fn).double(), scale.double()
        # a request at a time: its old entries of the first page, then whole pages of the new rows
        for b, (s, r) in enumerate(zip(S, rows)):
            if not r:
                continue
            p0, p1, off = s // PAGE, -(-(s + r) // PAGE), s % PAGE
            ids = torch.tensor(table[b][p0:p1], device="cuda")
            real = vals[ids] * scales[ids][:, :, None, None]
            line = torch.zeros((p1 - p0) * PAGE, x.shape[2], x.shape[3], dtype=torch.float64, device="cuda")
            line[off:off + r] = x[b, :r].double()
            new = line.view(p1 - p0, PAGE, x.shape[2], x.shape[3]).transpose(1, 2)
            amax = new.abs().amax(dim=(2, 3))
            want = torch.exp2(torch.ceil(torch.log2((amax / E4M3_MAX).clamp_min(2.0 ** -126))))
            if off:
                want[0] = torch.maximum(want[0], scales[ids[0]])
            put = torch.zeros_like(new) + vals[ids]
            flat = torch.arange((p1 - p0) * PAGE, device="cuda").view(p1 - p0, 1, PAGE, 1)
            rounded = _nearest_e4m3(torch.where(flat < off, real, new) / want[:, :, None, None])
            put = torch.where(flat < off + r, rounded, put)
            vals[ids], scales[ids] = put, want
        out.append((vals, scales))
    return [out[0][0], out[1][0], out[0][1], out[1][1], None]


def _exact_attend(st):
    c, q = st["c"], st["q"]
    K, nq, nkv, hd = c["K"], c["nq"], c["nkv"], c["hd"]
    G = nq // nkv
    out = torch.zeros(c["B"], K, nq, hd, dtype=torch.float64, device="cuda")
    S = st["seq_lens"].tolist()
    rows = [K] * c["B"] if st["rows"] is None else st["rows"].tolist()
    for b, (s, r) in enumerate(zip(S, rows)):
        if not r:
            continue
        n = s + r
        ids = st["page_table"][b, :-(-n // PAGE)].long()
        k, v = ((codes[ids].view(torch.float8_e4m3fn).double() * sc[ids].double()[:, :, None, None])
                .transpose(0, 1).reshape(nkv, -1, hd)[:, :n] for codes, sc in ((st["kc"], st["ks"]), (st["vc"], st["vs"])))
        x = torch.einsum("rhgd,hld->hrgl", q[b, :r].double().view(r, nkv, G, hd), k) * hd ** -0.5
        hidden = torch.arange(n, device="cuda")[None, :] > s + torch.arange(r, device="cuda")[:, None]
        x.masked_fill_(hidden[None, :, None, :], -math.inf)
        out[b, :r] = torch.einsum("hrgl,hld->rhgd", torch.softmax(x, dim=3), v).reshape(r, nq, hd)
    return [out, None]


def _exact_linear(st):
    c, w, x = st["c"], st["w"], st["x"].double()
    y = torch.empty(c["N"], c["M"], dtype=torch.float64, device="cuda")
    scale, zero = st["s"].double(), 8 if st["z"] is None else st["z"].double()
    step = 1 << 15
    xg = torch.nn.functional.pad(x, (0, -c["Kd"] % c["group"])).view(c["N"], -1, c["group"])
    for m in range(0, c["M"], step):
        part = w[m:m + step]
        code = torch.empty(part.shape[0], c["Kd"], dtype=torch.float64, device="cuda")
        code[:, 0::2], code[:, 1::2] = (part % 16).double(), (part // 16).double()
        code = torch.nn.functional.pad(code, (0, -c["Kd"] % c["group"])).view(part.shape[0], -1, c["group"])
        z = zero if st["z"] is None else zero[m:m + step, :, None]
        y[:, m:m + step] = torch.einsum("ngk,mgk,mg->nm", xg, code - z, scale[m:m + step])
    return y
