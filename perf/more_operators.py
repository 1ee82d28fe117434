"""Cases of the operators around a 4-bit KV cache: its write with the position rotation on the way, the attention over
it, and the log probabilities of a step's tokens.

Three operators, picked by a case's "op":

  append    new query, key and value rows are rotated to their positions; keys and values are stored in a paged cache
            of 4-bit codes with a scale and a base for each entry of a head, queries are returned
  attend    grouped-query attention of K rows per request over that cache
  logprobs  for each row of logits the log probability of a given token, the entropy, and the k likeliest tokens with
            theirs

`run` computes them in their plain form, or, where `own` is true, with the calls of the package.
"""

import math

import torch

own = False

PAGE = 16          # cache entries in a page


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a decoding step of a single user: one row, latency counts
        dict(name="append one row", op="append", B=1, nq=32, nkv=4, hd=128, lo=2048, hi=2048, n_max=1, ragged=False,
             theta=1e4),
        # a draft pass of 32 requests writes its rows behind the committed entries
        dict(name="append drafts", op="append", B=32, nq=32, nkv=4, hd=128, lo=0, hi=511, n_max=8, ragged=False,
             theta=1e4),
        # prompts of up to 2048 tokens, ragged, are stored in one call
        dict(name="append prompts", op="append", B=8, nq=64, nkv=8, hd=64, lo=0, hi=40, n_max=2048, ragged=True,
             theta=1e4),
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
        # the token that a single user's step has sampled, without alternatives
        dict(name="logprobs one row", op="logprobs", R=1, V=151936, pad=0, k=0, T=1.0, dtype="f32"),
        # the drafts of a single user and the bonus token, with the alternatives that an answer shows
        dict(name="logprobs drafts", op="logprobs", R=8, V=151936, pad=0, k=5, T=0.3, dtype="f32"),
        # a full server's verified positions
        dict(name="logprobs batch", op="logprobs", R=1408, V=151936, pad=0, k=5, T=0.3, dtype="f32"),
        # a batch of logits in bf16 (ties among the likeliest), many alternatives
        dict(name="logprobs bf16", op="logprobs", R=704, V=201088, pad=0, k=20, T=1.0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "logprobs", "logprobs"])
    hd = rng.choice([64, 128])
    nkv = rng.choice([1, 2, 4, 8])
    if op == "append":
        G = rng.choice([1, 2, 4, 5, 8])
        if rng.random() < 0.6:
            B, n_max, hi = _log(rng, 1, 128), rng.randint(1, 16), _log(rng, 1, 4096)
        else:
            B, n_max, hi = rng.randint(1, 8), _log(rng, 17, 2048), rng.randint(0, 40)
        # the pool stays in the range of the listed ones
        hi = min(hi, 65536 // (B * nkv))
        return dict(op=op, B=B, nq=nkv * G if rng.random() < 0.7 else 0, nkv=nkv, hd=hd, lo=rng.randint(0, hi), hi=hi,
                    n_max=n_max, ragged=rng.random() < 0.5, theta=rng.choice([0.0, 1e4, 1e4, 1e6]))
    if op == "attend":
        G = rng.choice([1, 2, 4, 5, 8, 16])
        K = rng.randint(1, min(16, 128 // G)) if rng.random() < 0.6 else 1
        B = _log(rng, 1, 128)
        # entries of all requests together stay below those of the largest listed case
        top = max(64, min(131072, 8192 * 40 * 4 // (B * nkv)))
        hi = _log(rng, 8, top)
        lo = hi if rng.random() < 0.3 else _log(rng, 1, hi) - 1
        return dict(op=op, B=B, K=K, nq=nkv * G, nkv=nkv, hd=hd, lo=lo, hi=hi, ragged=rng.random() < 0.4)
    V = _log(rng, 1000, 201088)
    R = _log(rng, 1, 1408)
    while R * V > 1408 * 151936:
        R //= 2
    return dict(op=op, R=R, V=V, pad=rng.choice([0, 0, 1, 64]), k=rng.choice([0, 1, 5, 20]),
                T=rng.choice([0.3, 0.7, 1.0]), dtype=rng.choice(["f32", "bf16"]))


# ---------------------------------------------------------------- inputs

def _lens(c):
    """The requests' lengths: evenly spread from lo to hi, so that their sum depends on the case alone."""
    B = c["B"]
    return [c["lo"] + (c["hi"] - c["lo"]) * b // max(1, B - 1) for b in range(B)] if B > 1 else [c["hi"]]


def _rows(c, n):
    """New rows of each request: n, or from none to n where the case is ragged; the first has them all."""
    return [(7 * b + n) % (n + 1) if c["ragged"] and b else n for b in range(c["B"])]


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(need, max_pages, g):
    """A page table of randomly placed pages, -1 where a request has none, and the number of pages."""
    total = max(1, int(sum(need)))
    n = torch.tensor(need, device="cuda")
    ids = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    at = torch.arange(max_pages, device="cuda")[None, :]
    first = (n.cumsum(0) - n)[:, None]
    table = torch.where(at < n[:, None], ids[(first + at).clamp_max(total - 1)], -1)
    return table.contiguous(), total


def _quantise(x):
    """Codes 0 .. 15 of x [..., hd] (as numbers) and its scale and base in bf16: x is about base + scale * code."""
    x = x.float()
    base = x.amin(dim=-1).to(torch.bfloat16)
    scale = ((x.amax(dim=-1) - base.float()) / 15.0).to(torch.bfloat16)
    s, lo = scale.float()[..., None], base.float()[..., None]
    code = torch.where(s > 0, torch.round((x - lo) / torch.where(s > 0, s, 1.0)).clamp(0, 15), 0)
    return code.to(torch.uint8), torch.stack([scale, base], dim=-1)


def _pack(code):
    """Two codes to a byte, the even one in its low half."""
    return code[..., 0::2] | (code[..., 1::2] << 4)


def _cache(pages, nkv, hd, g):
    """The codes [2, pages, nkv, 16, hd / 2] and parameters [2, pages, nkv, 16, 2] of random keys and values; some
    entries are larger than others."""
    x = torch.randn(2, pages, nkv, PAGE, hd, generator=g, device="cuda")
    x *= 1.0 + 3.0 * (torch.rand(2, pages, nkv, PAGE, 1, generator=g, device="cuda") < 0.05)
    code, params = _quantise(x)
    return _pack(code), params


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c, op = case, case["op"]
    if op == "append":
        B, n, nq, nkv, hd = c["B"], c["n_max"], c["nq"], c["nkv"], c["hd"]
        S, rows = _lens(c), _rows(c, n)
        need = [-(-(s + r) // PAGE) for s, r in zip(S, rows)]
        table, num_pages = _table(need, max(1, max(need)), g)
        codes, params = _cache(num_pages, nkv, hd, g)
        # queries, keys and values are columns of a fused projection's output, as in a decoder layer
        heads = nq + 2 * nkv
        qkv = torch.randn(B, n, heads * hd, generator=g, device="cuda")
        qkv *= 1.0 + 4.0 * (torch.rand(B, n, 1, generator=g, device="cuda") < 0.1)
        qkv = qkv.to(torch.bfloat16).unflatten(-1, (heads, hd))
        # a request's positions run ahead of its cache's entries, as placeholders were dropped from it
        ahead = torch.randint(0, 16, (B,), generator=g, device="cuda").to(torch.int32)
        return dict(c=c, q=qkv[:, :, :nq] if nq else None, k=qkv[:, :, nq:nq + nkv], v=qkv[:, :, nq + nkv:],
                    seq_lens=_i32(S), positions=_i32(S) + ahead, rows=_i32(rows), page_table=table, codes=codes,
                    params=params)
    if op == "attend":
        B, K, nq, nkv, hd = c["B"], c["K"], c["nq"], c["nkv"], c["hd"]
        S, rows = _lens(c), _rows(c, K)
        order = torch.randperm(B, generator=g, device="cuda").tolist()
        S, rows = [S[i] for i in order], [rows[i] for i in order]
        need = [-(-(s + K) // PAGE) for s in S]
        table, num_pages = _table(need, max(need), g)
        codes, params = _cache(num_pages, nkv, hd, g)
        q = (1.5 * torch.randn(B, K, nq, hd, generator=g, device="cuda")).to(torch.bfloat16)
        return dict(c=c, q=q, seq_lens=_i32(S), rows=_i32(rows) if c["ragged"] else None, page_table=table,
                    codes=codes, params=params)
    R, V = c["R"], c["V"]
    # a model's logits: most tokens far below a few that compete, and rows from sure of theirs to undecided
    x = torch.randn(R, V + c["pad"], generator=g, device="cuda")
    x *= 0.5 + 2.5 * torch.rand(R, 1, generator=g, device="cuda")
    hot = torch.randint(0, V, (R, 8), generator=g, device="cuda")
    x.scatter_add_(1, hot, 10.0 * torch.rand(R, 8, generator=g, device="cuda"))
    x = x.to(torch.bfloat16) if c["dtype"] == "bf16" else x
    # the sampled tokens: one of the likely ones, or any
    rare = torch.randint(0, V, (R,), generator=g, device="cuda")
    tokens = torch.where(torch.rand(R, generator=g, device="cuda") < 0.8, hot[:, 0], rare).to(torch.int32)
    return dict(c=c, logits=x[:, :V], tokens=tokens)


# ---------------------------------------------------------------- one pass

def run(state):
    if own:
        return _own(state)
    return {"append": _append, "attend": _attend, "logprobs": _logprobs}[state["c"]["op"]](state)


def _values(codes):
    """What the bytes hold: n * 2^-9 for the codes n of their low and high halves, which E4M3 has as they stand."""
    return [(codes & 15).view(torch.float8_e4m3fn), (codes >> 4).view(torch.float8_e4m3fn)]


def _own(st):
    from speculative_drafting_pe_gb300 import binding
    op = st["c"]["op"]
    if op == "append":
        q, status = binding.kv4_append(st["k"], st["v"], st["seq_lens"], st["page_table"], st["codes"][0],
                                       st["codes"][1], st["params"][0], st["params"][1], rows=st["rows"],
                                       theta=st["c"]["theta"], positions=st["positions"], q=st["q"])
        return [*_values(st["codes"]), st["params"], q, status]
    if op == "attend":
        return list(binding.attention_kv4(st["q"], st["seq_lens"], st["page_table"], st["codes"][0], st["codes"][1],
                                          st["params"][0], st["params"][1], rows=st["rows"]))
    o = binding.token_logprobs(st["logits"], st["tokens"], top=st["c"]["k"], temperature=st["c"]["T"])
    return [o["logprobs"], o["entropy"], o["top_tokens"], o["top_logprobs"]]


def _append(st):
    c, rows = st["c"], st["rows"].long()
    n, nkv, hd, theta = c["n_max"], c["nkv"], c["hd"], c["theta"]
    j = torch.arange(n, device=rows.device)[None, :]
    live = j < rows[:, None]

    def rotated(x):
        x = x.float()
        if theta == 0:
            return x
        half = hd // 2
        i = torch.arange(half, device=x.device, dtype=torch.float64)
        turn = (st["positions"].long()[:, None] + j).double()[:, :, None, None] * theta ** (-2.0 * i / hd)
        cos, sin = torch.cos(turn).float(), torch.sin(turn).float()
        a, b = x[..., :half], x[..., half:]
        return torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)

    # rows that are padded away stand in for the first row of the first request, and write what it writes
    b = torch.arange(c["B"], device=rows.device)[:, None].expand(-1, n)
    b, i = torch.where(live, b, 0).flatten(), torch.where(live, j, 0).flatten()
    e = st["seq_lens"].long()[b] + i
    page, slot = st["page_table"].long()[b, e // PAGE], e % PAGE
    both = torch.stack([rotated(st["k"])[b, i], st["v"].float()[b, i]])
    code, params = _quantise(both)
    st["codes"][:, page, :, slot] = _pack(code).transpose(0, 1)
    st["params"][:, page, :, slot] = params.transpose(0, 1)
    q = None
    if st["q"] is not None:
        q = torch.where(live[:, :, None, None], rotated(st["q"]), 0).to(torch.bfloat16)
    return [*_values(st["codes"]), st["params"], q, torch.zeros_like(st["seq_lens"])]


def _attend(st):
    c, q, table = st["c"], st["q"], st["page_table"].long().clamp_min(0)
    B, K, nq, nkv, hd = c["B"], c["K"], c["nq"], c["nkv"], c["hd"]
    S = st["seq_lens"].long()
    L, G = table.shape[1] * PAGE, nq // nkv
    last = S[:, None] + torch.arange(K, device=S.device)
    sees = torch.arange(L, device=S.device)[None, None, :] <= last[:, :, None]
    if st["rows"] is not None:
        sees = sees & (torch.arange(K, device=S.device)[None, :] < st["rows"][:, None])[:, :, None]

    def values(side):
        w, p = st["codes"][side][table], st["params"][side][table].float()
        x = torch.stack([w & 15, w >> 4], dim=-1).flatten(-2) * p[..., :1] + p[..., 1:]
        return x.transpose(1, 2).reshape(B, nkv, L, hd)

    k = values(0)
    rows = q.float().view(B, K, nkv, G, hd).permute(0, 2, 1, 3, 4).reshape(B, nkv, K * G, hd)
    s = torch.matmul(rows, k.transpose(2, 3)) / math.sqrt(hd)
    del k
    m = sees[:, None, :, None, :].expand(B, nkv, K, G, L).reshape(B, nkv, K * G, L)
    s = torch.where(m, s, -math.inf)
    top = s.amax(dim=3, keepdim=True)
    w = torch.exp(s - torch.where(top > -math.inf, top, 0))
    total = w.sum(dim=3, keepdim=True)
    o = torch.matmul(w, values(1)) / torch.where(total > 0, total, 1)
    o = o.view(B, nkv, K, G, hd).permute(0, 2, 1, 3, 4).reshape(B, K, nq, hd)
    return [o.to(torch.bfloat16), torch.zeros(B, dtype=torch.int32, device=S.device)]


def _logprobs(st):
    c, V = st["c"], st["c"]["V"]
    x = st["logits"].float()
    y = (x - x.amax(dim=1, keepdim=True)) / c["T"]
    e = torch.exp(y)
    total = e.sum(dim=1, dtype=torch.float64)
    log_z = torch.log(total)
    at = torch.gather(y, 1, st["tokens"].long()[:, None])[:, 0].double() - log_z
    entropy = log_z - (e * y).sum(dim=1, dtype=torch.float64) / total
    # order by value, among equal ones by index: one whole number for both
    u = x.view(torch.int32).long()
    rank = torch.where(u < 0, -(u & 0x7FFFFFFF), u) * (1 << 20) + (V - 1 - torch.arange(V, device=x.device))
    ids = torch.topk(rank, c["k"], dim=1).indices
    top = torch.gather(y, 1, ids).double() - log_z[:, None]
    return [at.float(), entropy.float(), ids.to(torch.int32), top.float()]


# ---------------------------------------------------------------- bytes and operations

def work(case):
    c, op = case, case["op"]
    if op == "append":
        S, rows = _lens(c), _rows(c, c["n_max"])
        n = sum(rows)
        pages = sum(-(-(s + r) // PAGE) - s // PAGE for s, r in zip(S, rows) if r)
        # rows in; codes, parameters and rotated queries out; lengths, positions, rows, status and pages
        return dict(bytes=2.0 * n * (c["nq"] + 2 * c["nkv"]) * c["hd"] + 2.0 * n * c["nkv"] * (c["hd"] / 2 + 4) +
                    2.0 * n * c["nq"] * c["hd"] + 4.0 * (4 * c["B"] + pages),
                    flops=3.0 * n * (c["nq"] + c["nkv"]) * c["hd"] + 6.0 * n * 2 * c["nkv"] * c["hd"])
    if op == "attend":
        S, rows = _lens(c), _rows(c, c["K"])
        live = [s + r for s, r in zip(S, rows) if r]
        entries = sum(live)
        pages = sum(-(-n // PAGE) for n in live)
        q = 2 * 2 * sum(rows) * c["nq"] * c["hd"]
        seen = sum(r * s + r * (r + 1) // 2 for s, r in zip(S, rows))
        return dict(bytes=2.0 * entries * c["nkv"] * (c["hd"] / 2 + 4) + 4.0 * pages + q + 12.0 * c["B"],
                    flops=4.0 * seen * c["nq"] * c["hd"])
    R, V = c["R"], c["V"]
    return dict(bytes=R * V * (2.0 if c["dtype"] == "bf16" else 4.0) + R * (12.0 + 8.0 * c["k"]), flops=6.0 * R * V)


# ---------------------------------------------------------------- the definitions, in 64 bits

def exact(case, seed):
    st = prepare(case, seed)
    return {"append": _exact_append, "attend": _exact_attend, "logprobs": _exact_logprobs}[case["op"]](st)


def _exact_rotate(x, at, theta):
    """Rows x [n, heads, hd] at positions at [n]: pairs (i, i + hd/2) as complex numbers, turned."""
    x, hd = x.double(), x.shape[-1]
    if theta == 0:
        return x
    z = torch.complex(x[..., :hd // 2], x[..., hd // 2:])
    angle = at.double()[:, None] / theta ** (torch.arange(0, hd, 2, device=x.device, dtype=torch.float64) / hd)
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    return torch.cat([z.real, z.imag], dim=-1)


def _exact_append(st):
    c, theta = st["c"], st["c"]["theta"]
    codes = torch.stack([st["codes"] % 16, st["codes"] // 16], dim=-1).double()
    params = st["params"].double()
    q = None if st["q"] is None else torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    S, rows, first = st["seq_lens"].tolist(), st["rows"].tolist(), st["positions"].tolist()
    for b, (s, r, p) in enumerate(zip(S, rows, first)):
        if not r:
            continue
        e = torch.arange(s, s + r, device="cuda")
        at = torch.arange(p, p + r, device="cuda")
        page, slot = st["page_table"][b].long()[e // PAGE], e % PAGE
        for side, x in ((0, _exact_rotate(st["k"][b, :r], at, theta)), (1, st["v"][b, :r].double())):
            base = x.amin(dim=2).to(torch.bfloat16).double()
            scale = ((x.amax(dim=2) - base) / 15).to(torch.bfloat16).double()
            n = torch.round((x - base[..., None]) / scale[..., None]).clamp(0, 15)
            codes[side, page, :, slot] = n.unflatten(-1, (-1, 2))
            params[side, page, :, slot] = torch.stack([scale, base], dim=-1)
        if q is not None:
            q[b, :r] = _exact_rotate(st["q"][b, :r], at, theta)
    return [codes[..., 0] / 512, codes[..., 1] / 512, params, q, None]


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
        kv = []
        for side in (0, 1):
            w, p = st["codes"][side][ids], st["params"][side][ids].double()
            x = torch.empty(*w.shape[:-1], hd, dtype=torch.float64, device="cuda")
            x[..., 0::2], x[..., 1::2] = (w % 16).double(), (w // 16).double()
            kv.append((x * p[..., :1] + p[..., 1:]).transpose(0, 1).reshape(nkv, -1, hd)[:, :n])
        x = torch.einsum("rhgd,hld->hrgl", q[b, :r].double().view(r, nkv, G, hd), kv[0]) * hd ** -0.5
        hidden = torch.arange(n, device="cuda")[None, :] > s + torch.arange(r, device="cuda")[:, None]
        x.masked_fill_(hidden[None, :, None, :], -math.inf)
        out[b, :r] = torch.einsum("hrgl,hld->rhgd", torch.softmax(x, dim=3), kv[1]).reshape(r, nq, hd)
    return [out, None]


def _exact_logprobs(st):
    c = st["c"]
    got = []
    # some rows at a time, so that 64 bits of them fit
    for x, t in zip(st["logits"].split(128), st["tokens"].split(128)):
        p = torch.log_softmax(x.double() / c["T"], dim=1)
        h = -(p * torch.exp(p)).sum(dim=1)
        order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices[:, :c["k"]]
        got.append((p.gather(1, t.long()[:, None])[:, 0], h, p.gather(1, order)))
    at, h, top = (torch.cat(v) for v in zip(*got))
    return [at, h, None, top]
