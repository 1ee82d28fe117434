"""The 8-bit paged KV cache on the GPU against float64: the write side bit for bit, the attention within the bounds
that its roundings give."""

import numpy as np
import pytest
import torch

from oracle import lowbit
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu

PAGE = 16


def _dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda", dtype=dtype)


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


def _cache(rng, pages, nkv, hd, junk=True):
    """Codes and scales of random rows; with `junk`, any bytes at all where nobody has written."""
    x = rng.standard_normal((pages, nkv, PAGE, hd)) * np.exp2(rng.integers(-3, 4, (pages, nkv, 1, 1)))
    s = np.empty((pages, nkv), dtype=np.float32)
    for p in range(pages):
        for h in range(nkv):
            s[p, h] = lowbit.kv8_scale(x[p, h])
    return lowbit.e4m3_encode(x / s[:, :, None, None]), s


# ---------------------------------------------------------------- write side

def _append(k, v, S, rows, table, kc, vc, ks, vs, kd=None, vd=None):
    kx, kt = _bf16(k)
    vx, vt = _bf16(v)
    want = lowbit.kv8_append(kx, vx, S, rows, table, kc, vc, ks, vs)
    dev = [_dev(a) for a in (kc, vc, ks, vs)]
    status = binding.kv8_append(kt if kd is None else kd(kt), vt if vd is None else vd(vt), _dev(S, torch.int32),
                                _dev(table), *dev, rows=None if rows is None else _dev(rows, torch.int32))
    torch.cuda.synchronize()
    np.testing.assert_array_equal(status.cpu().numpy(), want[4])
    for name, got, ref in zip(("k_codes", "v_codes", "k_scale", "v_scale"), dev, want):
        np.testing.assert_array_equal(got.cpu().numpy(), ref, err_msg=name)
    return dev, want


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("B,nkv,n,hi,ragged", [(1, 1, 1, 0, False), (3, 2, 5, 40, False), (9, 4, 11, 90, True),
                                               (2, 3, 70, 17, True), (4, 8, 16, 16, False)])
def test_append_bit_for_bit(B, nkv, n, hi, ragged, hd):
    rng = np.random.default_rng(hd + B + n)
    S = rng.integers(0, hi + 1, B).astype(np.int32)
    rows = rng.integers(0, n + 1, B).astype(np.int32) if ragged else None
    full = rows if ragged else np.full(B, n)
    need = -(-(S + full) // PAGE)
    table, pages = _table(rng, need, int(need.max()) + 1)
    kc, ks = _cache(rng, pages, nkv, hd)
    vc, vs = _cache(rng, pages, nkv, hd)
    mag = np.exp2(rng.integers(-6, 7, (B, n, nkv, 1)))    # old codes move, or the old scale stays
    _append(rng.standard_normal((B, n, nkv, hd)) * mag, rng.standard_normal((B, n, nkv, hd)) / mag, S, rows, table,
            kc, vc, ks, vs)


def test_append_of_strided_rows():
    rng = np.random.default_rng(5)
    B, n, nkv, hd = 3, 4, 2, 64
    S = np.array([0, 15, 30], dtype=np.int32)
    table, pages = _table(rng, [1, 2, 3], 3)
    kc, ks = _cache(rng, pages, nkv, hd)

    def columns(at):
        def put(t):
            wide = torch.full((B, n, 5 * nkv * hd), float("nan"), dtype=torch.bfloat16, device="cuda")
            wide[..., at * nkv * hd:(at + 1) * nkv * hd] = t.flatten(2)
            return wide[..., at * nkv * hd:(at + 1) * nkv * hd].unflatten(-1, (nkv, hd))
        return put

    _append(rng.standard_normal((B, n, nkv, hd)), rng.standard_normal((B, n, nkv, hd)), S, None, table, kc, kc, ks, ks,
            columns(3), columns(4))


def test_append_extremes():
    # zeros, the smallest and largest bf16 values, the border between two scales, infinities and NaN
    hd = 64
    row = np.zeros((1, 6, 1, hd))
    row[0, 0, 0, :4] = [448.0, -448.0, 2.0 ** -126, 1.0]
    row[0, 1, 0, :3] = [np.inf, -np.inf, np.nan]
    row[0, 2, 0, :2] = [3.3e38, -1e30]
    vals = np.zeros((1, 6, 1, hd))
    vals[0, 3, 0, :3] = [2.0 ** -133, -2.0 ** -130, 0.0]
    S, table = np.array([13], np.int32), np.array([[1, 0]], np.int32)
    kc, ks = _cache(np.random.default_rng(1), 2, 1, hd)
    zero = np.zeros_like(kc)
    _append(row, vals, S, None, table, kc, zero, ks, np.full((2, 1), 2.0 ** -126, np.float32))
    _append(row * 0, np.full((1, 6, 1, hd), 449.0), S, None, table, zero, kc, np.zeros((2, 1), np.float32), ks)


def test_append_twice_is_append_once():
    # the same rows again change nothing; rows in two calls give the codes of one where the scale is the same
    rng = np.random.default_rng(8)
    S, table = np.array([3, 20], np.int32), np.array([[2, 0], [1, 3]], np.int32)
    kc, ks = _cache(rng, 5, 2, 128)
    x = rng.standard_normal((2, 9, 2, 128))
    dev, want = _append(x, x, S, None, table, kc, kc, ks, ks)
    _append(x, x, S, None, table, *[want[i] for i in (0, 1, 2, 3)])


def test_append_refuses_requests_alone():
    rng = np.random.default_rng(2)
    S = np.array([-1, 0, 30, 5, 16, 3], np.int32)
    rows = np.array([1, 4, 3, -1, 2, 2], np.int32)
    table = np.array([[0, 1], [2, 3], [4, 5], [6, 7], [8, -1], [12, 9]], np.int32)   # [4]: no page, [5]: beyond the pool
    kc, ks = _cache(rng, 12, 2, 64)
    _, want = _append(rng.standard_normal((6, 3, 2, 64)), rng.standard_normal((6, 3, 2, 64)), S, rows, table, kc, kc,
                      ks, ks)
    assert want[4].tolist() == [3, 3, 1, 3, 2, 2]


# ---------------------------------------------------------------- attention

def _bound(out, size, cache_top, L):
    """Half a step of the bf16 output, 2^-8 |o|; the weights rounded to fp16 (2^-11 of each, with 2^-13 for the fp32
    score and the exponential), and where a weight falls below fp16's normal range half its smallest step, 2^-25, of
    the largest value, L times at most."""
    return 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2.0 ** -13) * size + L * 2.0 ** -25 * cache_top


def _attend(q, S, rows, table, kc, vc, ks, vs, scale=None, place=None, **kw):
    qx, qt = _bf16(q)
    hd = q.shape[-1]
    ref, status, size = lowbit.attention_kv8(qx, S, rows, table, kc, vc, ks, vs, hd ** -0.5 if scale is None else scale)
    qt = qt if place is None else place(qt)
    got, st = binding.attention_kv8(qt, _dev(S, torch.int32), _dev(table), _dev(kc), _dev(vc), _dev(ks), _dev(vs),
                                    scale=scale, rows=None if rows is None else _dev(rows, torch.int32), **kw)
    torch.cuda.synchronize()
    np.testing.assert_array_equal(st.cpu().numpy(), status)
    got = got.double().cpu().numpy()
    top = np.nanmax(np.abs(lowbit.e4m3_decode(vc) * vs[:, :, None, None].astype(np.float64)), initial=0.0)
    lim = _bound(ref, size, top, int(np.max(S, initial=0)) + q.shape[1])
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref))
    err = np.where(np.isnan(ref), 0, np.abs(got - ref))
    assert (err <= np.where(np.isnan(lim), 0, lim)).all(), (err.max(), (err / np.maximum(lim, 1e-30)).max())
    return got, ref


def _case(seed, S, K, nq, nkv, hd, rows=None, junk=True):
    rng = np.random.default_rng(seed)
    S = np.asarray(S, dtype=np.int32)
    full = np.full(len(S), K) if rows is None else np.asarray(rows)
    need = -(-(S + full) // PAGE)
    table, pages = _table(rng, need, max(1, int(need.max())) + 1)
    kc, ks = _cache(rng, pages, nkv, hd)
    vc, vs = _cache(rng, pages, nkv, hd)
    if junk:   # entries behind a request's last one hold NaN codes, pages of nobody NaN scales
        used = np.zeros((pages, PAGE), bool)
        for b, n in enumerate(S + full):
            for e in range(n):
                used[table[b, e // PAGE], e % PAGE] = True
        for c in (kc, vc):
            c[np.broadcast_to(~used[:, None, :, None], c.shape)] = 0x7F
        for s in (ks, vs):
            s[~used.any(1)] = np.nan
    q = 2.0 * rng.standard_normal((len(S), K, nq, hd))
    return q, S, None if rows is None else np.asarray(rows, np.int32), table, kc, vc, ks, vs


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("S,K,nq,nkv", [
    ([0], 1, 1, 1), ([0], 3, 4, 2), ([15], 1, 8, 1), ([16], 2, 8, 2), ([130, 0, 7, 64], 1, 8, 2),
    ([50, 500, 31], 7, 16, 2), ([333], 16, 8, 1), ([90, 17], 5, 5, 1), ([1000, 3], 11, 16, 2), ([40], 1, 128, 1),
    ([12] * 40, 2, 4, 4)])
def test_attention_matches_float64(S, K, nq, nkv, hd):
    _attend(*_case(len(S) + K + hd, S, K, nq, nkv, hd))


@pytest.mark.parametrize("S,K,nq,nkv,hd", [([3000], 1, 8, 2, 128), ([5000, 100], 4, 8, 1, 64), ([2500], 9, 32, 4, 128)])
def test_attention_split_over_many_blocks(S, K, nq, nkv, hd):
    _attend(*_case(K, S, K, nq, nkv, hd))


@pytest.mark.parametrize("hd", [64, 128])
def test_attention_of_padded_rows(hd):
    got, _ = _attend(*_case(4, [60, 10, 0, 33, 200], 6, 8, 2, hd, rows=[6, 0, 1, 3, 5]))
    assert (got[1] == 0).all() and (got[3, 3:] == 0).all()


def test_attention_of_strided_queries_into_a_wider_output():
    q, S, rows, table, kc, vc, ks, vs = _case(6, [70, 20], 3, 8, 2, 64)

    def place(t):
        wide = torch.full((2, 3, 12 * 64), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[..., :8 * 64] = t.flatten(2)
        return wide[..., :8 * 64].unflatten(-1, (8, 64))

    wide = torch.full((2, 3, 1000), 5.0, dtype=torch.bfloat16, device="cuda")
    _attend(q, S, rows, table, kc, vc, ks, vs, place=place, out=wide[..., 8:520].unflatten(-1, (8, 64)), scale=0.3)
    assert (wide[..., :8] == 5).all() and (wide[..., 520:] == 5).all()


def test_attention_scales_of_any_size():
    # scales that are no powers of two, tiny, zero and negative ones, and values far apart from page to page
    q, S, rows, table, kc, vc, ks, vs = _case(7, [400, 100], 4, 8, 2, 128, junk=False)
    rng = np.random.default_rng(9)
    vs *= rng.uniform(0.5, 2.0, vs.shape).astype(np.float32) * np.exp2(rng.integers(-6, 7, vs.shape)).astype(np.float32)
    ks *= rng.uniform(0.2, 1.0, ks.shape).astype(np.float32)
    vs[table[0, 3]], vs[table[0, 5]], ks[table[0, 7]], ks[table[0, 0]] = 0.0, 2.0 ** -126, 0.0, -ks[table[0, 0]]
    _attend(q, S, rows, table, kc, vc, ks, vs)


def test_attention_with_far_scores():
    # one entry outweighs all others by e^80 and more, early or late
    for at in (0, 77, 300):
        q, S, rows, table, kc, vc, ks, vs = _case(at, [301], 1, 4, 1, 64, junk=False)
        ks[:] = 2.0 ** -9
        q[:] = 8.0
        kc[table[0, at // PAGE], 0, at % PAGE] = 0x7E
        ks[table[0, at // PAGE], 0] = 2.0 ** -6
        _attend(q, S, rows, table, kc, vc, ks, vs)


def test_attention_nan_stays_with_the_rows_that_see_it():
    # entry S + 2 belongs to row 2: rows 0 and 1 do not see it
    for which in (0, 1):
        q, S, rows, table, kc, vc, ks, vs = _case(11, [45], 4, 8, 2, 128)
        clean, _ = _attend(q, S, rows, table, kc, vc, ks, vs)
        (kc, vc)[which][table[0, 47 // PAGE], 0, 47 % PAGE, 5] = 0xFF
        got, _ = binding.attention_kv8(_bf16(q)[1], _dev(S), _dev(table), _dev(kc), _dev(vc), _dev(ks), _dev(vs))
        got = got.double().cpu().numpy()
        np.testing.assert_array_equal(got[0, :2], clean[0, :2])
        np.testing.assert_array_equal(got[0, :, 4:], clean[0, :, 4:])     # the other kv head
        assert np.isnan(got[0, 2:, :4]).all()


def test_attention_refuses_requests_alone():
    q, S, rows, table, kc, vc, ks, vs = _case(12, [20, 20, 20, 20, 20, 400], 2, 8, 2, 64, rows=[2] * 6)
    S[0], rows[1], rows[2] = -1, 3, -1
    table[3, 1], table[4, 0] = len(kc), -1
    table[5, 20] = -7
    ok = _case(12, [20, 20, 20, 20, 20, 400], 2, 8, 2, 64, rows=[2] * 6)
    got, ref = _attend(q, S, rows, table, kc, vc, ks, vs)
    assert (got == 0).all()
    S = np.array([20, 16 * table.shape[1] - 1, 20, 20, 20, 20], np.int32)
    _attend(ok[0], S, ok[2], ok[3], *ok[4:])


def test_attention_repeats_bit_for_bit_and_under_capture():
    q, S, rows, table, kc, vc, ks, vs = _case(13, [700, 40, 1500], 3, 16, 2, 128)
    args = [_bf16(q)[1], _dev(S), _dev(table), _dev(kc), _dev(vc), _dev(ks), _dev(vs)]
    first = binding.attention_kv8(*args)[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = binding.attention_kv8(*args, stream=side)[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        third, status = binding.attention_kv8(*args)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, second) and torch.equal(first, third) and (status == 0).all()
    # two captured calls, replayed at once on two streams
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(binding.attention_kv8(*args)[0])
        graphs.append(g)
    torch.cuda.synchronize()
    for g, s in zip(graphs, (side, torch.cuda.Stream())):
        with torch.cuda.stream(s):
            for _ in range(20):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)
