"""The attention over the 8-bit cache where its roundings, its shares of the work and its rules for what is not finite
show: every kernel behind the entry point (few and many query rows, 64- and 128-wide heads) against float64."""

import numpy as np
import pytest
import torch

from oracle import lowbit
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu

PAGE = 16
# K, query heads, kv heads, width: the kernel of few rows and the tensor-memory one, of either width
KERNELS = [(4, 4, 2, 128), (4, 8, 2, 64), (4, 16, 2, 128), (4, 16, 2, 64)]
NAMES = ["few rows, 128 wide", "few rows, 64 wide", "many rows, 128 wide", "many rows, 64 wide"]


def _dev(a):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda")


def _bf16(a):
    t = torch.as_tensor(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


def _cache(rng, pages, nkv, hd, top=4):
    """Random codes of full range and power-of-two scales."""
    x = rng.standard_normal((pages, nkv, PAGE, hd))
    s = np.exp2(rng.integers(-2, top, (pages, nkv))).astype(np.float32) * np.float32(2.0 ** -7)
    return lowbit.e4m3_encode(x * 2.0 ** 7), s


def _exact(q, S, table, kc, vc, ks, vs, scale):
    """Outputs, how far they may be off, and sum_e w_e |v_e|.

    Half a step of the bf16 output, 2^-8 |o|. Every weight rounded to fp16 (2^-11) after fp32 steps and an exponential
    (2^-13). A weight below fp16's normal range is off by 2^-25 at most where the row's largest w |scale of v| stands
    at 2^5 or above, so by 2^-30 of that, times a code of 448, for each of L entries. Scores: sums in fp32 of eight
    products of 32 dimensions (few rows: 16), each off by 2^-22 of what is summed in size; and the queries as they
    enter. Few rows: an fp16 copy whose largest value lies in [1, 2), off by 2^-25 at most. Many rows: two E4M3 terms,
    the largest value in [128, 256), together off by 2^-10 at most, where a value is below 1/4. A score off by d
    changes a weight by a factor of exp(+-2 d) at most."""
    B, K, nq, hd = q.shape
    nkv = kc.shape[1]
    many = K * nq // nkv > (8 if hd == 128 else 16)
    out, lim, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape)
    top = np.exp2(np.floor(np.log2(np.maximum(np.abs(q).max(-1, keepdims=True), 1e-300))))
    dq = np.where(np.abs(q) < top * 2.0 ** -9, top * 2.0 ** -17, 0) if many else top * 2.0 ** -25
    dq = dq + 2.0 ** -19 * np.abs(q)
    for b in range(B):
        ids = table[b, :-(-(S[b] + K) // PAGE)]
        kk = lowbit.e4m3_decode(kc[ids]) * ks[ids].astype(np.float64)[:, :, None, None]
        sv = vs[ids].astype(np.float64)
        vv = lowbit.e4m3_decode(vc[ids]) * sv[:, :, None, None]
        for g in range(nkv):
            ke, ve, se = kk[:, g].reshape(-1, hd), vv[:, g].reshape(-1, hd), np.repeat(np.abs(sv[:, g]), PAGE)
            ka = np.abs(ke)
            for h in range(g * nq // nkv, (g + 1) * nq // nkv):
                for j in range(K):
                    n = S[b] + j + 1
                    x = scale * (ke[:n] @ q[b, j, h])
                    w = np.exp(x - x.max())
                    w /= w.sum()
                    o = w @ ve[:n]
                    d = w * np.expm1(2 * scale * (ka[:n] @ dq[b, j, h]))
                    out[b, j, h], size[b, j, h] = o, w @ np.abs(ve[:n])
                    lim[b, j, h] = (2.0 ** -8 * np.abs(o) + (2.0 ** -11 + 2.0 ** -13) * size[b, j, h] +
                                    n * 2.0 ** -30 * 448 * (w * se[:n]).max() + d @ np.abs(ve[:n] - o))
    return out, lim, size


def _call(q, S, table, kc, vc, ks, vs):
    lens, cache = _dev(np.asarray(S, np.int32)), map(_dev, (kc, vc, ks, vs))
    got, status = binding.attention_kv8(q, lens, _dev(table), *cache)
    torch.cuda.synchronize()
    assert (status == 0).all()
    return got.double().cpu().numpy()


def _check(got, ref, lim):
    err = np.abs(got - ref)
    assert np.isfinite(got).all() and (err <= lim).all(), (err / np.maximum(lim, 1e-300)).max()


def _check_copies(q, S, table, kc, vc, ks, vs, copies, ref, lim):
    """The batch `copies` times over: a warp has several pages of a request, or one."""
    got = _call(q.repeat(copies, 1, 1, 1), np.tile(S, copies), np.tile(table, (copies, 1)), kc, vc, ks, vs)
    for c in range(copies):
        _check(got[c * len(S):(c + 1) * len(S)], ref, lim)


# ---------------------------------------------------------------- scales of V far apart

@pytest.mark.parametrize("K,nq,nkv,hd", KERNELS, ids=NAMES)
@pytest.mark.parametrize("low", [-12, -24, -60])
def test_small_values_that_have_the_weight(K, nq, nkv, hd, low):
    # pages of large values that hardly any weight falls on, among pages of values 2^low as large that have it: the
    # output is theirs, to the precision of any other
    rng = np.random.default_rng(K + hd)
    S = [300, 75]
    table = rng.permutation(60)[:40].reshape(2, 20).astype(np.int32)
    kc, ks = _cache(rng, 60, nkv, hd)
    vc, vs = _cache(rng, 60, nkv, hd)
    loud = np.zeros(60, dtype=bool)
    loud[table[0, [0, 3, 4, 9, 18]]] = loud[table[1, [1, 4]]] = True
    kc = np.where(loud[:, None, None, None], kc | 0x80, kc & 0x7F)   # queries are positive
    ks[:] = 2.0 ** -7
    vs[~loud] *= np.float32(2.0 ** low)
    qx, qt = _bf16(5 * (np.abs(rng.standard_normal((2, K, nq, hd))) + 0.5))
    ref, lim, size = _exact(qx, S, table, kc, vc, ks, vs, hd ** -0.5)
    assert size.max() < 2.0 ** (low + 5)      # the large values have no say
    for copies in (1, 60):
        _check_copies(qt, S, table, kc, vc, ks, vs, copies, ref, lim)


@pytest.mark.parametrize("K,nq,nkv,hd", KERNELS, ids=NAMES)
def test_scales_of_every_kind(K, nq, nkv, hd):
    # scales that are no powers of two, negative, zero, subnormal and near the ends of their range, from page to page
    rng = np.random.default_rng(nq + hd)
    S = [333, 100, 4]
    table = rng.permutation(66).reshape(3, 22).astype(np.int32)
    kc, ks = _cache(rng, 66, nkv, hd)
    vc, vs = _cache(rng, 66, nkv, hd)
    ks *= rng.uniform(0.2, 1.0, ks.shape).astype(np.float32) * rng.choice([-1, 1], ks.shape).astype(np.float32)
    vs *= rng.uniform(0.2, 1.0, vs.shape).astype(np.float32) * rng.choice([-1, 1], vs.shape).astype(np.float32)
    ks[table[0, [2, 11]]], vs[table[0, [5, 13]]], vs[table[0, 7]] = 0.0, 0.0, 2.0 ** -126
    vs[table[1, [0, 3]]], ks[table[1, 2]] = 2.0 ** -140, 2.0 ** -130
    vs[table[1, 5]] = 2.0 ** 100
    vs[table[2]] = 2.0 ** -90
    qx, qt = _bf16(2.0 * rng.standard_normal((3, K, nq, hd)))
    ref, lim, size = _exact(qx, S, table, kc, vc, ks, vs, hd ** -0.5)
    for copies in (1, 60):
        _check_copies(qt, S, table, kc, vc, ks, vs, copies, ref, lim)


def test_pages_of_zeros_beside_others():
    # rows of zeros are stored with the smallest scale there is; whichever has the weight, the sum is right
    hd, nkv = 64, 1
    rng = np.random.default_rng(3)
    kc, ks = _cache(rng, 8, nkv, hd)
    vc, vs = _cache(rng, 8, nkv, hd)
    vc[[1, 4]], vs[[1, 4]] = 0, 2.0 ** -126
    ks[[1, 4]] *= 16
    table = np.array([[1, 0, 4, 5, 2, 3, 7, 6]], dtype=np.int32)
    for K, nq in ((1, 4), (4, 8)):
        qx, qt = _bf16(4.0 * rng.standard_normal((1, K, nq, hd)))
        ref, lim, size = _exact(qx, [120], table, kc, vc, ks, vs, hd ** -0.5)
        _check(_call(qt, [120], table, kc, vc, ks, vs), ref, lim)


# ---------------------------------------------------------------- what is not finite

@pytest.mark.parametrize("K,nq,nkv,hd", KERNELS, ids=NAMES)
@pytest.mark.parametrize("S", [45, 700])
def test_nan_in_the_cache_stays_with_the_rows_that_see_it(K, nq, nkv, hd, S):
    # entry S + 2 belongs to row 2; rows 0 and 1 do not see it
    rng = np.random.default_rng(S + hd)
    kc, ks = _cache(rng, 50, nkv, hd)
    vc, vs = _cache(rng, 50, nkv, hd)
    table = rng.permutation(50)[:48].reshape(1, 48).astype(np.int32)
    G, at = nq // nkv, (table[0, (S + 2) // PAGE], nkv - 1, (S + 2) % PAGE)
    _, qt = _bf16(rng.standard_normal((1, K, nq, hd)))
    clean = _call(qt, [S], table, kc, vc, ks, vs)
    assert np.isfinite(clean).all()
    for codes in (kc, vc):
        for nan in (0x7F, 0xFF):
            for d in (0, 5, hd // 2 + 3, hd - 1):
                had = codes[at + (d,)]
                codes[at + (d,)] = nan
                got = _call(qt, [S], table, kc, vc, ks, vs)
                codes[at + (d,)] = had
                np.testing.assert_array_equal(got[0, :2], clean[0, :2])
                np.testing.assert_array_equal(got[0, :, :-G], clean[0, :, :-G])   # the other kv head
                assert np.isnan(got[0, 2:, -G:, d]).all()


@pytest.mark.parametrize("K,nq,nkv,hd", KERNELS, ids=NAMES)
def test_queries_that_are_not_finite_spoil_their_row_alone(K, nq, nkv, hd):
    rng = np.random.default_rng(hd + nq)
    S = [200, 31]
    kc, ks = _cache(rng, 40, nkv, hd)
    vc, vs = _cache(rng, 40, nkv, hd)
    table = rng.permutation(40)[:32].reshape(2, 16).astype(np.int32)
    q = rng.standard_normal((2, K, nq, hd))
    clean = _call(_bf16(q)[1], S, table, kc, vc, ks, vs)
    spoilt = np.zeros((2, K, nq), dtype=bool)
    for i, x in enumerate((np.inf, -np.inf, np.nan)):
        b, j, h = i % 2, (2 * i + 1) % K, (3 * i + 1) % nq
        q[b, j, h, (7 * i + hd - 3) % hd] = x
        spoilt[b, j, h] = True
    got = _call(_bf16(q)[1], S, table, kc, vc, ks, vs)
    assert np.isnan(got[spoilt]).all()
    np.testing.assert_array_equal(got[~spoilt], clean[~spoilt])


# ---------------------------------------------------------------- queries of uneven size

@pytest.mark.parametrize("K,nq,nkv,hd", KERNELS, ids=NAMES)
def test_queries_with_one_dimension_far_above_the_others(K, nq, nkv, hd):
    # the first dimension of a query is 2^12 times the others, and nearly nothing in the keys
    rng = np.random.default_rng(hd + nq)
    S = [150, 40]
    kc, ks = _cache(rng, 40, nkv, hd)
    vc, vs = _cache(rng, 40, nkv, hd)
    ks[:] = 2.0 ** -7
    kc[..., 0] &= 0x87        # no larger than 7/8 of E4M3's smallest normal value
    table = rng.permutation(40)[:30].reshape(2, 15).astype(np.int32)
    q = rng.standard_normal((2, K, nq, hd)) * 2.0 ** -2
    q[..., 0] = rng.choice([-1, 1], q.shape[:3]) * rng.uniform(0.6, 1.9, q.shape[:3]) * 2.0 ** 10
    qx, qt = _bf16(q)
    ref, lim, size = _exact(qx, S, table, kc, vc, ks, vs, hd ** -0.5)
    _check(_call(qt, S, table, kc, vc, ks, vs), ref, lim)


# ---------------------------------------------------------------- rows that end anywhere in a warp

@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [1, 7, 9, 15, 17, 31, 33, 40, 63, 65, 88, 97, 127, 128])
def test_any_number_of_rows(rows, hd):
    # heads that one CTA has whole, and heads that several share
    rng = np.random.default_rng(rows)
    S = [130, 3]
    kc, ks = _cache(rng, 40, 1, hd)
    vc, vs = _cache(rng, 40, 1, hd)
    table = rng.permutation(40)[:34].reshape(2, 17).astype(np.int32)
    for K, nq in {(rows, 1), (1, rows)}:
        qx, qt = _bf16(rng.standard_normal((2, K, nq, hd)))
        ref, lim, _ = _exact(qx, S, table, kc, vc, ks, vs, hd ** -0.5)
        for copies in (1, 40):
            _check_copies(qt, S, table, kc, vc, ks, vs, copies, ref, lim)


# ---------------------------------------------------------------- no page is lost, none counts twice

def _marked(rng, pages, nkv, hd, share):
    """Values 1 in one dimension of each page (by its place in the table, `share` pages to a dimension in turn), and
    keys of any kind."""
    kc, ks = _cache(rng, 64, nkv, hd)
    at = torch.as_tensor(rng.integers(0, 64, pages)).cuda()
    kc, ks = _dev(kc)[at].contiguous(), _dev(ks)[at].contiguous()
    vc = torch.zeros(pages, nkv, PAGE, hd, dtype=torch.uint8, device="cuda")
    place = torch.arange(pages, device="cuda")
    vc[place, :, :, place // share % hd] = 0x38
    return kc, ks, vc, torch.ones(pages, nkv, device="cuda")


MANY = [
    # B, K, query heads, kv heads, width, entries
    (1, 1, 8, 1, 128, [70000]), (2, 2, 8, 1, 64, [30000, 12345]), (1, 7, 8, 1, 128, [65000]),
    (3, 5, 16, 2, 64, [9000, 40000, 77]), (300, 1, 1, 1, 64, [5000, 3, 12000, 640]),
    # shares longer than a CTA's tables, heads cut by them once and several times
    (8, 1, 8, 8, 128, [40000]), (8, 2, 8, 8, 64, [40000]), (16, 3, 64, 8, 64, [36000]), (16, 5, 16, 8, 128, [36000]),
    (50, 1, 8, 8, 64, [9600]), (64, 5, 16, 8, 64, [9600]), (64, 9, 8, 8, 128, [9600]),
    (120, 1, 8, 8, 128, [50000, 100]), (60, 2, 64, 8, 64, [60000, 31000, 9]), (40, 9, 8, 8, 128, [100000, 5]),
    (40, 5, 32, 8, 64, [90000, 120000])]


@pytest.mark.parametrize("B,K,nq,nkv,hd,lens", MANY)
def test_every_page_counts_once(B, K, nq, nkv, hd, lens):
    # queries of zero see every entry alike: dimension d of the output is the share of the entries whose page marks it
    S = np.resize(lens, B).astype(np.int64)
    pages = -(-(int(S.max()) + K) // PAGE)
    rng = np.random.default_rng(B + K)
    for share in (1, -(-pages // hd)):       # neighbours in dimensions of their own, or in runs
        kc, ks, vc, vs = _marked(rng, pages, nkv, hd, share)
        table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, pages).contiguous()
        q = torch.zeros(B, K, nq, hd, dtype=torch.bfloat16, device="cuda")
        got, status = binding.attention_kv8(q, _dev(S.astype(np.int32)), table, kc, vc, ks, vs)
        assert (status == 0).all()
        got = got.double().cpu().numpy()
        dim = np.arange(pages * PAGE) // PAGE // share % hd
        for s in set(lens):
            want = np.stack([np.bincount(dim[:s + j + 1], minlength=hd) / (s + j + 1) for j in range(K)])
            # the bf16 output, the sums' fp32 steps; every weight is a power of two
            err = np.abs(got[S == s] - want[None, :, None, :])
            assert (err <= (2.0 ** -8 + 2.0 ** -14) * want[None, :, None, :]).all(), (s, err.max())


@pytest.mark.parametrize("B,K,nq,nkv,hd,S", [(8, 1, 8, 8, 128, 40000), (16, 3, 64, 8, 64, 36000),
                                             (64, 9, 8, 8, 128, 9600), (1, 2, 8, 1, 64, 50000)])
def test_long_requests_with_scores_of_every_size(B, K, nq, nkv, hd, S):
    # the same request B times over: shares and their joins lie elsewhere in each
    rng = np.random.default_rng(B)
    kc, ks = _cache(rng, 200, nkv, hd)
    vc, vs = _cache(rng, 200, nkv, hd)
    ks *= 4
    table = rng.integers(0, 200, (1, -(-(S + K) // PAGE))).astype(np.int32)
    qx, qt = _bf16(rng.standard_normal((1, K, nq, hd)))
    ref, lim, size = _exact(qx, [S], table, kc, vc, ks, vs, hd ** -0.5)
    got = _call(qt.expand(B, K, nq, hd).contiguous(), [S] * B, np.repeat(table, B, 0), kc, vc, ks, vs)
    _check(got, ref, lim)


@pytest.mark.parametrize("K", [1, 9])
def test_scratch_does_not_follow_the_page_table(K):
    # two partial tiles for each multiprocessor and a table of cuts, however many pages a request could have
    need = [binding._kv8_scratch(0, 256, K, 64, 8, 128, pages) for pages in (64, 512, 8192, 100000)]
    tile = (128 if K > 1 else 8) * (128 + 2)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert len(set(need)) == 1 and need[0] <= sms * (2 * tile + 4) + 16


@pytest.mark.parametrize("K,nq,nkv,hd", KERNELS, ids=NAMES)
def test_thousands_of_short_requests(K, nq, nkv, hd):
    # segments of one unit, dozens of them to a CTA
    rng = np.random.default_rng(nq)
    S = rng.integers(0, 70, 40)
    kc, ks = _cache(rng, 60, nkv, hd)
    vc, vs = _cache(rng, 60, nkv, hd)
    table = rng.integers(0, 60, (40, 5)).astype(np.int32)
    qx, qt = _bf16(rng.standard_normal((40, K, nq, hd)))
    ref, lim, _ = _exact(qx, S, table, kc, vc, ks, vs, hd ** -0.5)
    _check_copies(qt, S, table, kc, vc, ks, vs, 100, ref, lim)


@pytest.mark.parametrize("B,K,nq,nkv,hd,S,width", [(3, 1, 8, 8, 128, 900, 30000), (8, 1, 8, 8, 128, 40000, 2600),
                                                   (8, 5, 16, 8, 64, 300, 30000), (16, 5, 16, 8, 128, 36000, 2300)])
def test_windows_replayed_from_a_graph(B, K, nq, nkv, hd, S, width):
    # tables with room for more than a CTA's, with and without that many entries
    rng = np.random.default_rng(B)
    kc, ks = _cache(rng, 100, nkv, hd)
    vc, vs = _cache(rng, 100, nkv, hd)
    table = _dev(rng.integers(0, 100, (B, width)).astype(np.int32))
    lens = _dev(np.full(B, S, np.int32))
    q = _bf16(rng.standard_normal((B, K, nq, hd)))[1]
    cache = [_dev(a) for a in (kc, vc, ks, vs)]
    want, status = binding.attention_kv8(q, lens, table, *cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = binding.attention_kv8(q, lens, table, *cache)
    for _ in range(5):
        got.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and (status == 0).all()
    narrow, _ = binding.attention_kv8(q, lens, table[:, :-(-(S + K) // PAGE)].contiguous(), *cache)
    assert torch.equal(narrow, want)


# ---------------------------------------------------------------- a wait that gives up

@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("barrier,width", [(1, 60), (2, 60), (3, 60), (2, 60000)])
def test_waits_that_give_up_refuse_the_call_and_leave_the_next_alone(barrier, width, hd):
    # Host-side injection: a barrier of the tensor-memory kernel waits for one arrival more than there are. Its waits
    # end after their limit; every request with rows reports it, and all outputs are zero.
    import time

    rng = np.random.default_rng(barrier + hd)
    B, K, nq, nkv = 5, 6, 16, 2
    S, rows = [900, 30, 7, -1, 300], [6, 3, 0, 6, 6]
    kc, ks = _cache(rng, 80, nkv, hd)
    vc, vs = _cache(rng, 80, nkv, hd)
    table = rng.integers(0, 80, (B, width)).astype(np.int32)
    _, qt = _bf16(rng.standard_normal((B, K, nq, hd)))
    args = [qt] + [_dev(a) for a in (np.asarray(S, np.int32), table, kc, vc, ks, vs)]
    rows = _dev(np.asarray(rows, np.int32))
    clean, status = binding.attention_kv8(*args, rows=rows)
    assert status.tolist() == [0, 0, 0, binding.PE_REQ_BAD_INPUT, 0] and (clean[0] != 0).any()
    torch.cuda.synchronize()
    binding.test_stall_attention_kv8(barrier)
    few, status = binding.attention_kv8(qt[:, :1, :nkv].contiguous(), *args[1:])   # few rows: another kernel
    assert (status[[0, 1, 2, 4]] == 0).all()
    t0 = time.time()
    out = torch.full_like(qt, 3.0)
    out, status = binding.attention_kv8(*args, rows=rows, out=out)
    torch.cuda.synchronize()
    assert 0.5 < time.time() - t0 < 20.0
    late = binding.PE_REQ_TIMEOUT
    assert status.tolist() == [late, late, 0, binding.PE_REQ_BAD_INPUT, late] and (out == 0).all()
    out, status = binding.attention_kv8(*args, rows=rows)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0, 0, binding.PE_REQ_BAD_INPUT, 0] and torch.equal(out, clean)
