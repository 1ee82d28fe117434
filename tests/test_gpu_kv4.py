"""The 4-bit paged KV cache on the GPU against float64: the write side code for code, the attention within the bounds
that its roundings give."""

import numpy as np
import pytest
import torch

from oracle import kv4
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu

PAGE = 16


def _dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda", dtype=dtype)


def _i(a):
    return None if a is None else _dev(np.asarray(a), torch.int32)


def _bf16(a):
    """float64 values of a bf16 copy of a, and that copy on the device."""
    t = torch.as_tensor(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


def _table(rng, need, max_pages, spare=3):
    total = int(sum(need)) + spare
    ids = rng.permutation(total)
    table = np.full((len(need), max_pages), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = ids[at:at + n]
        at += n
    return table, total


def _cache(rng, pages, nkv, hd, spread=3):
    """Codes and parameters of random rows, their magnitudes spread over powers of two."""
    x = rng.standard_normal((pages, nkv, PAGE, hd)) * np.exp2(rng.integers(-spread, spread + 1, (pages, nkv, PAGE, 1)))
    codes, scale, base, _ = kv4.quantise(x + rng.standard_normal((pages, nkv, PAGE, 1)))
    return kv4.pack(codes), np.stack([scale, base], axis=-1)


# ---------------------------------------------------------------- write side

def _append(q, k, v, S, rows, positions, theta, table, pages, wide=None, in_place=False):
    """Append to a cache of junk; every byte against float64. A turned key is off by a few fp32 steps of its head's
    largest value, so a code may be the other one where the quotient is within 2^-16 of half a step, and base and
    scale the next bf16 value where theirs is as near to a border. Queries: half a bf16 step and the same."""
    rng = np.random.default_rng(1)
    nkv, hd = k.shape[2:]
    (kx, kt), (vx, vt) = _bf16(k), _bf16(v)
    qx, qt = (None, None) if q is None else _bf16(q)
    wrote, turned, status = kv4.append(qx, kx, vx, S, rows, positions, theta, table, pages)
    codes = [rng.integers(0, 256, (pages, nkv, PAGE, hd // 2), dtype=np.uint8) for _ in range(2)]
    params = [torch.as_tensor(rng.standard_normal((pages, nkv, PAGE, 2))).to(torch.bfloat16) for _ in range(2)]
    dc, dp = [_dev(c) for c in codes], [p.cuda() for p in params]
    if wide is not None:
        qt, kt, vt = wide(qt, kt, vt)
    got, st = binding.kv4_append(kt, vt, _i(S), _dev(table), dc[0], dc[1], dp[0], dp[1], rows=_i(rows), theta=theta,
                                 positions=_i(positions), q=qt, q_out=qt if in_place else None)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(st.cpu().numpy(), status)
    have = [kv4.unpack(c.cpu().numpy()) for c in dc]
    par = [p.double().cpu().numpy() for p in dp]
    want = [kv4.unpack(c) for c in codes]
    old = [p.double().numpy() for p in params]
    for side, at, h, slot, n, scale, base, part in wrote:
        old[side][at, h, slot] = par[side][at, h, slot]
        want[side][at, h, slot] = have[side][at, h, slot]
        s, b = par[side][at, h, slot]
        if not np.isfinite(scale):
            assert np.isnan(s) and np.isnan(b)
            continue
        exact = side == 1 or theta == 0
        if exact:
            assert (s, b) == (scale, base)
        else:
            assert abs(s - scale) <= 2.0 ** -7 * abs(scale) and abs(b - base) <= 2.0 ** -7 * abs(base) + 2.0 ** -120
        if (s, b) == (scale, base):
            near = np.abs(part - np.floor(part) - 0.5) < 2.0 ** -16
            assert (have[side][at, h, slot] == n)[~near].all()
            assert (np.abs(have[side][at, h, slot].astype(int) - n.astype(int)) <= 1).all()
    for side in range(2):   # and nothing else
        np.testing.assert_array_equal(have[side], want[side])
        np.testing.assert_array_equal(par[side], old[side])
    if q is not None:
        g = got.double().cpu().numpy()
        top = np.abs(np.where(np.isfinite(qx), qx, 0)).max(-1, keepdims=True)
        fine = np.isfinite(turned)
        np.testing.assert_array_equal(np.isfinite(g), fine)
        lim = 2.0 ** -8 * np.abs(turned) + 2.0 ** -20 * top
        assert (np.abs(g - turned)[fine] <= np.broadcast_to(lim, g.shape)[fine]).all()
    return have, par


def _case(rng, B, n, hi, ragged):
    S = rng.integers(0, hi + 1, B).astype(np.int32)
    rows = rng.integers(0, n + 1, B).astype(np.int32) if ragged else None
    need = -(-(S + (rows if ragged else n)) // PAGE)
    table, pages = _table(rng, need, int(need.max()) + 1)
    return S, rows, table, pages


@pytest.mark.parametrize("theta", [0.0, 1e4])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("B,nq,nkv,n,hi,ragged", [(1, 1, 1, 1, 0, False), (3, 4, 2, 5, 40, False), (9, 5, 1, 11, 90, True),
                                                  (2, 3, 3, 70, 17, True), (4, 16, 8, 16, 16, False),
                                                  (2, 0, 3, 9, 30, False), (200, 2, 1, 9, 20, True)])
def test_append(B, nq, nkv, n, hi, ragged, hd, theta):
    rng = np.random.default_rng(hd + B + n)
    S, rows, table, pages = _case(rng, B, n, hi, ragged)
    mag = np.exp2(rng.integers(-6, 7, (B, n, 1, 1)))
    x = lambda heads: rng.standard_normal((B, n, heads, hd)) * mag
    _append(x(nq) if nq else None, x(nkv), x(nkv) + 3.0, S, rows, S + rng.integers(0, 20, B), theta, table, pages)


@pytest.mark.parametrize("hd", [64, 128])
def test_append_of_strided_rows_in_place(hd):
    """Columns of a fused projection, the queries turned where they stand."""
    rng = np.random.default_rng(hd)
    B, nq, nkv, n = 3, 4, 2, 7
    S, rows, table, pages = _case(rng, B, n, 30, True)

    def wide(q, k, v):
        both = torch.full((B, n, nq + 2 * nkv + 1, hd), float("nan"), dtype=torch.bfloat16, device="cuda")
        both[:, :, :nq], both[:, :, nq:nq + nkv], both[:, :, nq + nkv:-1] = q, k, v
        return both[:, :, :nq], both[:, :, nq:nq + nkv], both[:, :, nq + nkv:-1]
    x = lambda heads: rng.standard_normal((B, n, heads, hd))
    _append(x(nq), x(nkv), x(nkv), S, rows, None, 1e4, table, pages, wide=wide, in_place=True)


@pytest.mark.parametrize("theta", [1.0, 1e4, 1e6, 5e5])
@pytest.mark.parametrize("first", [0, 1, 131071, 10 ** 6, 2 ** 24 + 1, 2 ** 31 - 9])
def test_far_positions(first, theta):
    rng = np.random.default_rng(first % 97)
    S = np.array([3, 0], dtype=np.int32)
    table, pages = _table(rng, [1, 1], 2)
    x = lambda: rng.standard_normal((2, 8, 2, 128))
    _append(x(), x(), x(), S, None, np.array([first, max(0, first - 5)]), theta, table, pages)


@pytest.mark.parametrize("hd", [64, 128])
def test_values_at_the_ends_of_their_range(hd):
    rng = np.random.default_rng(5)
    n = 16
    k, v = rng.standard_normal((1, n, 2, hd)), rng.standard_normal((1, n, 2, hd))
    v[0, 0] = 0.0                       # one value throughout
    v[0, 1] = -7.25
    v[0, 2, 0, 5] = np.inf
    v[0, 3, 1, hd - 1] = -np.inf
    v[0, 4, 1, 0] = np.nan
    v[0, 5] *= 2.0 ** 120
    v[0, 6] *= 2.0 ** -120
    v[0, 7] = 1000.0 + v[0, 7]          # a narrow band far from zero
    v[0, 8, :, :] = np.where(np.arange(hd) == 7, 1e30, 1e-30)
    v[0, 9] *= 2.0 ** -128              # below the smallest normal number
    k[0, 2, 1, 3] = np.nan
    k[0, 3, 0, hd // 2] = np.inf
    q = rng.standard_normal((1, n, 2, hd))
    q[0, 1, 0, 3] = np.inf
    q[0, 2, 1, hd - 1] = np.nan
    table, pages = _table(rng, [1], 1)
    _append(None, k, v, np.array([0]), None, None, 0.0, table, pages)
    _append(None, k, v, np.array([0]), None, None, 1e4, table, pages)
    # a pair with an infinity or a NaN turns into NaN or infinities, and no other
    qt = torch.as_tensor(q).to(torch.bfloat16).cuda()
    kt = torch.zeros((1, n, 1, hd), dtype=torch.bfloat16, device="cuda")
    c = [torch.zeros((pages, 1, PAGE, hd // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    p = [torch.zeros((pages, 1, PAGE, 2), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out, _ = binding.kv4_append(kt, kt, _i([0]), _dev(table), *c, *p, q=qt, theta=1e4)
    odd = ~torch.isfinite(out)[0].cpu()
    at = [tuple(x) for x in odd.nonzero().tolist()]
    assert at == [(1, 0, 3), (1, 0, 3 + hd // 2), (2, 1, hd // 2 - 1), (2, 1, hd - 1)]


def test_refused_requests_write_nothing_and_leave_the_others():
    rng = np.random.default_rng(11)
    n, hd = 5, 64
    S = np.array([4, -1, 30, 8, 12, 14, 2, 2 ** 31 - 1], dtype=np.int32)
    rows = np.array([5, 2, 5, 6, -1, 5, 0, 5], dtype=np.int32)
    table = np.array([[0, 1], [2, 3], [4, 5], [6, 7], [8, 9], [10, 99], [-1, -1], [12, 13]], dtype=np.int32)
    x = lambda: rng.standard_normal((8, n, 2, hd))
    for theta, positions in ((1e4, None), (0.0, None), (1e4, np.array([0, 0, 0, 0, 0, 0, 0, 0])),
                             (1e4, np.array([-1, 0, 0, 0, 0, 0, 2 ** 31 - 1, 0])), (0.0, np.full(8, -5))):
        _append(x(), x(), x(), S, rows, positions, theta, table, 14)


# ---------------------------------------------------------------- attention

def _lim(ref, size, reach, top, L, rows):
    """Half a step of bf16; weights times V's scale in fp16, products below fp16's normal range, L of them; fp32
    scores, whose products and sums are off by some 2^-21 of what they add up. With more than 16 rows K and V
    themselves go to fp16, each value by two roundings."""
    scores = 2.0 ** -21 * reach[..., None]
    value = 0.0
    if rows > 16:
        scores, value = scores + 2.0 ** -10 * reach[..., None], 2.0 ** -10
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -14 + value + 2.0 * np.minimum(scores, 1.0)) * size + L * 2.0 ** -24 * top


def _attend(rng, B, K, nq, nkv, hd, S, rows=None, scale=None, codes=None, params=None, table=None, pages=None, q=None,
            spread=2):
    if table is None:
        table, pages = _table(rng, [-(-(int(s) + K) // PAGE) for s in S], int(-(-(S.max() + K) // PAGE)) + 2)
    if codes is None:
        (kc, kp), (vc, vp) = _cache(rng, pages, nkv, hd, spread), _cache(rng, pages, nkv, hd, spread)
        codes, params = [kc, vc], [kp, vp]
    q = rng.standard_normal((B, K, nq, hd)) if q is None else q
    qx, qt = _bf16(q)
    scale = hd ** -0.5 if scale is None else scale
    ref, status, size, reach = kv4.attention(qx, S, rows, table, codes, params, scale)
    dp = [torch.as_tensor(x).to(torch.bfloat16).cuda() for x in params]
    out, st = binding.attention_kv4(qt, _i(S), _dev(table), _dev(codes[0]), _dev(codes[1]), *dp, scale=scale, rows=_i(rows))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(st.cpu().numpy(), status)
    got = out.double().cpu().numpy()
    _, va = kv4.values(codes[1], params[1])
    top = va[np.isfinite(va)].max()
    lim = _lim(ref, size, reach, top, int(S.max()) + K, K * nq // nkv)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
    fine = np.isfinite(ref)
    assert (np.abs(got - ref)[fine] <= lim[fine]).all(), (np.abs(got - ref) / lim)[fine].max()
    return got


SHAPES = [(1, 1), (1, 5), (3, 2), (4, 2), (2, 8), (8, 2), (3, 5), (5, 5), (11, 4), (8, 8), (11, 8), (16, 8), (7, 16), (1, 128)]


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", SHAPES)
def test_attention(K, G, hd):
    rng = np.random.default_rng(K * 131 + G + hd)
    B, nkv = 5, 2
    S = np.array([0, 1, 15, 100, 333], dtype=np.int32)
    _attend(rng, B, K, nkv * G, nkv, hd, S)
    _attend(rng, B, K, nkv * G, nkv, hd, S, rows=rng.integers(0, K + 1, B), scale=0.3)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", [(1, 8), (2, 8), (11, 8)])
def test_every_length_around_pages_and_units(K, G, hd):
    rng = np.random.default_rng(hd + K)
    S = np.arange(0, 131, dtype=np.int32)
    _attend(rng, len(S), K, G, 1, hd, S)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", [(1, 8), (2, 8), (11, 8)])
@pytest.mark.parametrize("S", [5000, 40000])
def test_one_long_request(K, G, hd, S):
    rng = np.random.default_rng(S)
    _attend(rng, 1, K, G, 1, hd, np.array([S], dtype=np.int32))


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", [(1, 8), (2, 8), (11, 8)])
def test_negative_and_zero_softmax_scales(K, G, hd):
    rng = np.random.default_rng(hd)
    for scale in (-0.2, 0.0, 3.0):
        _attend(rng, 2, K, 2 * G, 2, hd, np.array([40, 100]), scale=scale, spread=0)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", [(1, 8), (2, 8), (11, 8)])
def test_entries_that_no_row_sees_may_hold_anything(K, G, hd):
    rng = np.random.default_rng(K + hd)
    S = np.array([0, 3, 17, 40], dtype=np.int32)
    table, pages = _table(rng, -(-(S + K) // PAGE), 6)
    codes, params = zip(*(_cache(rng, pages, 1, hd) for _ in range(2)))
    live = np.zeros((pages, PAGE), dtype=bool)
    for b, s in enumerate(S):
        for e in range(s + K):
            live[table[b, e // PAGE], e % PAGE] = True
    clean = _attend(rng, 4, K, G, 1, hd, S, codes=codes, params=params, table=table, pages=pages,
                    q=np.random.default_rng(2).standard_normal((4, K, G, hd)))
    for x in params:
        x[:, 0][~live] = np.array([np.nan, np.inf])
    for x in codes:
        x[:, 0][~live] = 0xFF
    dirty = _attend(rng, 4, K, G, 1, hd, S, codes=codes, params=params, table=table, pages=pages,
                    q=np.random.default_rng(2).standard_normal((4, K, G, hd)))
    np.testing.assert_array_equal(clean, dirty)


@pytest.mark.parametrize("side", [0, 1])
@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", [(3, 2), (2, 8), (11, 8)])
def test_a_parameter_that_is_not_finite_reaches_the_rows_that_see_it(K, G, hd, side):
    rng = np.random.default_rng(hd + side)
    for S, e in ((100, 3), (100, 95), (100, 101), (20, 21), (64, 64), (64, 65)):
        if e > S + K - 1:
            continue
        for bad in ((np.nan, 0.5), (0.5, np.nan), (np.inf, 0.0), (0.25, -np.inf)):
            table, pages = _table(rng, [-(-(S + K) // PAGE)], 9)
            codes, params = zip(*(_cache(rng, pages, 1, hd) for _ in range(2)))
            params[side][table[0, e // PAGE], 0, e % PAGE] = bad
            qt = torch.as_tensor(rng.standard_normal((1, K, G, hd))).to(torch.bfloat16)
            dp = [torch.as_tensor(x).to(torch.bfloat16).cuda() for x in params]
            out, st = binding.attention_kv4(qt.cuda(), _i([S]), _dev(table), _dev(codes[0]), _dev(codes[1]), *dp)
            got = out.double().cpu().numpy()[0]
            assert int(st[0]) == 0
            sees = S + np.arange(K) >= e
            assert np.isfinite(got[~sees]).all() and not np.isfinite(got[sees]).any(axis=(1, 2)).all()
            assert np.isnan(got[sees]).any(axis=2).all()
            # and the rows that do not see it are what they are without it
            params[side][table[0, e // PAGE], 0, e % PAGE] = 0.5
            ref, _, size, reach = kv4.attention(qt.double().numpy(), [S], None, table, codes, params, hd ** -0.5)
            lim = _lim(ref, size, reach, 64.0, S + K, K * G)[0]
            assert (np.abs(got - ref[0])[~sees] <= lim[~sees]).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", [(1, 8), (2, 8), (11, 8)])
def test_queries_that_are_not_finite_and_far_apart(K, G, hd):
    rng = np.random.default_rng(hd * K)
    q = rng.standard_normal((2, K, G, hd))
    q[0, 0, 0] *= 2.0 ** 40
    q[0, 0, 1] *= 2.0 ** -90
    q[0, 0, 2] = 0.0
    q[1, 0, 3, 5] = np.inf
    q[1, 0, 4, 6] = -np.inf
    q[1, 0, 5, 7] = np.nan
    S = np.array([50, 70])
    table, pages = _table(rng, -(-(S + K) // PAGE), 6)
    codes, params = zip(*(_cache(rng, pages, 1, hd, 0) for _ in range(2)))
    qt = torch.as_tensor(q).to(torch.bfloat16)
    dp = [torch.as_tensor(x).to(torch.bfloat16).cuda() for x in params]
    out, _ = binding.attention_kv4(qt.cuda(), _i(S), _dev(table), _dev(codes[0]), _dev(codes[1]), *dp)
    got = out.double().cpu().numpy()
    odd = np.zeros((2, K, G), dtype=bool)
    odd[1, 0, 3:6] = True
    assert np.isnan(got[odd]).all() and np.isfinite(got[~odd]).all()
    ref, _, size, reach = kv4.attention(qt.double().numpy(), S, None, table, codes, params, hd ** -0.5)
    even = ~odd
    even[0, 0, 0] = False    # its scores lie 2^40 apart: the largest alone counts
    lim = _lim(ref, size, reach, 64.0, 100, K * G)
    assert (np.abs(got - ref)[even] <= lim[even]).all()
    kk, _ = kv4.values(codes[0][table[0, :5]], params[0][table[0, :5]])
    vv, _ = kv4.values(codes[1][table[0, :5]], params[1][table[0, :5]])
    best = (kk[:, 0].reshape(-1, hd)[:51] @ qt.double().numpy()[0, 0, 0]).argmax()
    np.testing.assert_allclose(got[0, 0, 0], vv[:, 0].reshape(-1, hd)[best], rtol=2.0 ** -7, atol=2.0 ** -8)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", [(1, 8), (2, 8), (11, 8)])
@pytest.mark.parametrize("small", [-20, -60, -100])
def test_values_of_scales_far_apart(K, G, hd, small):
    """An entry of small values that has all the weight keeps its bits beside one of large ones."""
    rng = np.random.default_rng(hd - small)
    S = 70
    table, pages = _table(rng, [-(-(S + K) // PAGE)], 6)
    codes, params = zip(*(_cache(rng, pages, 1, hd, 0) for _ in range(2)))
    # keys: entry 5 wins for every query by far
    k = rng.standard_normal((S + K, hd))
    q = np.abs(rng.standard_normal((1, K, G, hd))) + 1.0
    k -= 60.0
    k[5] = 60.0 + rng.random(hd)
    v = rng.standard_normal((S + K, hd))
    v[5] *= 2.0 ** small
    for side, x in ((0, k), (1, v)):
        c, s, b, _ = kv4.quantise(x)
        for e in range(S + K):
            codes[side][table[0, e // PAGE], 0, e % PAGE] = kv4.pack(c[e])
            params[side][table[0, e // PAGE], 0, e % PAGE] = s[e], b[e]
    qx, qt = _bf16(q)
    dp = [torch.as_tensor(x).to(torch.bfloat16).cuda() for x in params]
    out, _ = binding.attention_kv4(qt, _i([S]), _dev(table), _dev(codes[0]), _dev(codes[1]), *dp)
    ref, _, size, _ = kv4.attention(qx, [S], None, table, codes, params, hd ** -0.5)
    assert (np.abs(ref) < 2.0 ** (small + 4)).all()
    got = out.double().cpu().numpy()
    # With more than 16 rows V goes to fp16 under a power of two of its page: the page's largest value, which the
    # exponents of base and scale bound within a factor of 8, stands below 2^15, and half of fp16's smallest step is
    # 2^-25: 2^-37 of the page's largest value, below which entry 5's bits are lost.
    rounds, floor = (2.0 ** -10, 2.0 ** -37 * np.abs(v[:16]).max()) if K * G > 16 else (0.0, 0.0)
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -10 + rounds) * size + floor).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", [(1, 8), (2, 8), (11, 8)])
def test_requests_that_are_refused(K, G, hd):
    rng = np.random.default_rng(K)
    S = np.array([40, -1, 96 - K + 1, 40, 40, 40, 30], dtype=np.int32)
    rows = np.array([K, K, K, K + 1, -1, K, 0], dtype=np.int32)
    table = rng.permutation(60)[:42].reshape(7, 6).astype(np.int32)
    table[5, 1] = 60
    table[0, 4:] = -7
    codes, params = zip(*(_cache(rng, 60, 2, hd) for _ in range(2)))
    got = _attend(rng, 7, K, 2 * G, 2, hd, S, rows=rows, codes=codes, params=params, table=table, pages=60)
    assert not got[1:].any()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", [(1, 8), (2, 8), (11, 8)])
def test_strided_queries_and_outputs(K, G, hd):
    rng = np.random.default_rng(hd + K)
    B, nkv = 3, 2
    S = np.array([20, 50, 90])
    table, pages = _table(rng, -(-(S + K) // PAGE), 8)
    codes, params = zip(*(_cache(rng, pages, nkv, hd) for _ in range(2)))
    dev = [_dev(codes[0]), _dev(codes[1])] + [torch.as_tensor(x).to(torch.bfloat16).cuda() for x in params]
    wide = torch.as_tensor(rng.standard_normal((B, K, nkv * G + 3, hd))).to(torch.bfloat16).cuda()
    q = wide[:, :, 2:-1]
    want, _ = binding.attention_kv4(q.contiguous(), _i(S), _dev(table), *dev)
    room = torch.full((B, K, nkv * G + 1, hd), 7.0, dtype=torch.bfloat16, device="cuda")
    binding.attention_kv4(q, _i(S), _dev(table), *dev, out=room[:, :, 1:])
    assert torch.equal(room[:, :, 1:], want) and bool((room[:, :, 0] == 7.0).all())
