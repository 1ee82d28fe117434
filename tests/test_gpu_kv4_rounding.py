"""The tensor-memory kernel of the attention over the 4-bit cache against float64 with K and V rounded as the header
says: what is left is the weights' rounding and the output's, which a scale or keys that are 1% off do not fit in."""

import numpy as np
import pytest
import torch

from oracle import kv4
from speculative_drafting_pe_gb300 import binding

PAGE, UNIT = 16, 64
SHAPES = [(3, 8, 64), (3, 8, 128), (11, 4, 128), (11, 8, 64), (11, 8, 128), (7, 16, 64), (1, 128, 128), (5, 5, 64)]


def _bits(x):
    """Of float64 values of bf16 the 16 bits."""
    return torch.as_tensor(x).to(torch.bfloat16).view(torch.int16).numpy().astype(np.int64) & 0xFFFF


def _half(x):
    return x.astype(np.float16).astype(np.float64)


def _rounded(codes, params, side, S):
    """Values [heads, entries, hd] of a request's pages as fp16 under a power of two of the page, in units of 64
    entries that every row sees, or of the entry: K as n * scale + base, rounded once (and its base), V as
    (n - 8) * scale + mid, mid and the sum rounded. The power of two follows from the exponents of base and scale."""
    n = kv4.unpack(codes).astype(np.float64).transpose(1, 0, 2, 3)
    par = params.transpose(1, 0, 2, 3)
    bits = _bits(par)
    f = np.maximum((bits[..., 1] >> 7) & 255, ((bits[..., 0] >> 7) & 255) + 4)
    whole = (np.arange(f.shape[1]) // (UNIT // PAGE) + 1) * UNIT - 1 <= S
    f = np.where(whole[None, :, None], f.max(-1, keepdims=True), f).clip(24, 254)
    up, scale, base = np.exp2(140.0 - f), par[..., 0], par[..., 1]
    if side == 0:
        down = np.exp2(-18.0)
        x = _half(n * (_half(scale * up * 64) * 2.0 ** -24)[..., None] + _half(base * up * down)[..., None]) / down
    else:
        x = _half((n - 8) * _half(scale * up)[..., None] + _half((8 * scale + base) * up)[..., None])
    x = x / up[..., None]
    return x.reshape(len(x), -1, x.shape[-1])


def _reference(q, S, k, v, scale):
    """(out, bound) of q [K, heads, hd] over k, v [kv heads, entries, hd]. The bound: half a step of bf16; 2^-11 of each
    weight's product with V and 2^-14 for the fp32 score and the exponential; fp32 sums of a score off by 2^-21 of
    what they add up; products below fp16's normal range off by 2^-26 of the row's largest, which the powers of two
    of K's and V's pages bound within 2^3."""
    K, nq, hd = q.shape
    out, lim = np.zeros(q.shape), np.zeros(q.shape)
    for h in range(nq):
        kh, vh = k[h * len(k) // nq], v[h * len(k) // nq]
        x = scale * (q[:, h] @ kh.T)
        reach = abs(scale) * (np.abs(q[:, h]) @ np.abs(kh).T)
        hidden = np.arange(len(kh))[None] > S + np.arange(K)[:, None]
        x[hidden], reach[hidden] = -np.inf, 0
        w = np.exp(x - x.max(1, keepdims=True))
        w /= w.sum(1, keepdims=True)
        top = (w * np.abs(vh).max(1)[None]).max(1)[:, None]
        out[:, h] = w @ vh
        size = w @ np.abs(vh)
        lim[:, h] = (2.0 ** -8 * np.abs(out[:, h]) + (2.0 ** -11 + 2.0 ** -14 + 2 * 2.0 ** -21 * reach.max(1)[:, None]) * size +
                     (S + K) * 2.0 ** -23 * top)
    return out, lim


def _cache(rng, pages, nkv, hd, spread):
    x = rng.standard_normal((pages, nkv, PAGE, hd)) * np.exp2(rng.integers(-spread, spread + 1, (pages, nkv, PAGE, 1)))
    codes, scale, base, _ = kv4.quantise(x + rng.standard_normal((pages, nkv, PAGE, 1)))
    return kv4.pack(codes), np.stack([scale, base], axis=-1)


def _case(K, G, hd, nkv, lens, spread):
    rng = np.random.default_rng(K * 1000 + G + hd)
    pages = [-(-(s + K) // PAGE) for s in lens]
    table = np.full((len(lens), max(pages) + 1), -1, dtype=np.int32)
    ids = rng.permutation(sum(pages))
    for b, n in enumerate(pages):
        table[b, :n], ids = ids[:n], ids[n:]
    k, v = _cache(rng, sum(pages), nkv, hd, spread), _cache(rng, sum(pages), nkv, hd, spread)
    qt = torch.as_tensor(rng.standard_normal((len(lens), K, nkv * G, hd))).to(torch.bfloat16)
    return qt, table, pages, k, v


def _wants(case, lens, hd, scale=None):
    qt, table, pages, k, v = case
    for b, S in enumerate(lens):
        ids = table[b, :pages[b]]
        kr, vr = (_rounded(c[ids], p[ids], side, S) for side, (c, p) in enumerate((k, v)))
        yield _reference(qt[b].double().numpy(), S, kr, vr, hd ** -0.5 if scale is None else scale)


def _check(case, lens, hd):
    qt, table, _, k, v = case
    dev = [torch.as_tensor(c).cuda() for c in (k[0], v[0])] + [torch.as_tensor(p).to(torch.bfloat16).cuda() for p in (k[1], v[1])]
    S = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, status = binding.attention_kv4(qt.cuda(), S, torch.as_tensor(table).cuda(), *dev)
    assert (status == 0).all()
    for got, (want, lim) in zip(out.double().cpu().numpy(), _wants(case, lens, hd)):
        assert (np.abs(got - want) <= lim).all(), (np.abs(got - want) / lim).max()


@pytest.mark.gpu
@pytest.mark.parametrize("spread", [0, 3])
@pytest.mark.parametrize("K,G,hd", SHAPES)
def test_many_rows(K, G, hd, spread):
    lens = [0, 40, 100, 333, 700]
    _check(_case(K, G, hd, 2, lens, spread), lens, hd)


@pytest.mark.gpu
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("S", [5000, 40000])
def test_one_long_request(S, hd):
    _check(_case(11, 8, hd, 1, [S], 2), [S], hd)


@pytest.mark.parametrize("what", ["keys", "values", "scale"])
@pytest.mark.parametrize("K,G,hd", SHAPES[:4])
def test_the_bound_notices_one_percent(K, G, hd, what):
    """What a softmax scale, or parameters of K or V, 1% too large would give is outside of the bound in many places."""
    lens = [100, 333, 700]
    case = _case(K, G, hd, 2, lens, 2)
    qt, table, pages, k, v = case
    more = lambda x: (x[0], kv4.bf16(x[1] * 1.01))
    wrong = (qt, table, pages, more(k) if what == "keys" else k, more(v) if what == "values" else v)
    scale = hd ** -0.5 * (1.01 if what == "scale" else 1.0)
    for (want, lim), (off, _) in zip(_wants(case, lens, hd), _wants(wrong, lens, hd, scale)):
        off = kv4.bf16(off)
        assert (np.abs(off - want) > lim).mean() > 0.02


@pytest.mark.gpu
@pytest.mark.parametrize("K,G,hd", [(1, 8, 128), (2, 8, 64), (11, 8, 64), (11, 8, 128)])
def test_products_far_below_the_largest(K, G, hd):
    """Two entries have nearly all of the weight and no V in half of the dimensions, where 598 others of 2^-25.4 each
    make the output: small products are off by 2^-26 of the row's largest at most (a register kernel's by 2^-30)."""
    B, S = 1500, 599
    entries = 608
    at = np.arange(entries)
    heavy = (at == 0) | (at == UNIT)                  # one for either softmax group
    # scores in base 2: k is one value throughout, q picks a dimension of it
    kp = np.zeros((entries // PAGE, 1, PAGE, 2))
    kp[..., 1] = np.where(heavy, 0.0, -25.375).reshape(-1, 1, PAGE)
    vp, code = np.zeros_like(kp), np.zeros((entries, hd), dtype=np.uint8)
    vp[..., 0] = kv4.bf16(np.where(heavy, 1 / 15, 0.0)).reshape(-1, 1, PAGE)
    vp[..., 1] = np.where(heavy, 0.0, 1.0).reshape(-1, 1, PAGE)
    code[heavy, :hd // 2] = 15
    codes = kv4.pack(code).reshape(entries // PAGE, 1, PAGE, hd // 2)
    q = torch.zeros(B, K, G, hd, dtype=torch.bfloat16, device="cuda")
    q[..., 3] = 1.0
    dev = [torch.as_tensor(np.zeros_like(codes)).cuda(), torch.as_tensor(codes).cuda()]
    dev += [torch.as_tensor(p).to(torch.bfloat16).cuda() for p in (kp, vp)]
    table = torch.arange(entries // PAGE, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    # the last row sees all: entries 0 .. S + j
    lens = torch.full((B,), S - K + 1, dtype=torch.int32, device="cuda")
    out, status = binding.attention_kv4(q, lens, table, *dev, scale=float(np.log(2.0)))
    assert (status == 0).all()
    got = out.double().cpu().numpy()
    for j in range(K):
        small = S - K + 1 + j + 1 - 2
        want = small * 2.0 ** -25.375 / (2 + small * 2.0 ** -25.375)
        part = 2.0 ** -26 if K * G > 16 else 2.0 ** -30
        lim = 2.0 ** -8 * want + 2.0 ** -11 * want + small * part / 2 + 2.0 ** -40
        assert (np.abs(got[:, j, :, hd // 2:] - want) <= lim).all(), (got[:, j, :, hd // 2:].min(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("K,G,hd", [(1, 8, 128), (2, 8, 128), (1, 8, 64), (11, 8, 64), (11, 8, 128)])
def test_outputs_do_not_change_from_call_to_call(K, G, hd):
    """Nor with what scratch held before: whatever part of a head a block has, its sums are joined in one order."""
    lens = [2000, 3, 900, 15, 4100]
    qt, table, _, k, v = _case(K, G, hd, 2, lens, 2)
    dev = [torch.as_tensor(c).cuda() for c in (k[0], v[0])] + [torch.as_tensor(p).to(torch.bfloat16).cuda() for p in (k[1], v[1])]
    args = (qt.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), torch.as_tensor(table).cuda(), *dev)
    first, _ = binding.attention_kv4(*args)
    for fill in (float("nan"), 0.0, -1.0, 1e30):
        junk = [torch.full((n,), fill, device="cuda") for n in (1 << 10, 1 << 16, 1 << 21, 6000000)]
        del junk
        again, _ = binding.attention_kv4(*args)
        assert torch.equal(first, again)
