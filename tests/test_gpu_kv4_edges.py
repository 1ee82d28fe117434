"""The 4-bit cache's operators where their shares of the work, their ranges and their rules show: long and many
requests, captured calls, entries that a row does not see, other streams, and a serving step of all of them."""

import time

import numpy as np
import pytest
import torch

from oracle import kv4
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu

PAGE = 16
# K, query heads, kv heads, width: the kernel of few rows (one and two tiles of them) and the tensor-memory one
KERNELS = [(4, 4, 2, 128), (4, 8, 2, 64), (5, 16, 2, 128), (4, 16, 2, 64)]
NAMES = ["few rows, 128 wide", "few rows, 64 wide", "many rows, 128 wide", "many rows, 64 wide"]


def _dev(a, dtype=None):
    return torch.as_tensor(np.ascontiguousarray(a), device="cuda", dtype=dtype)


def _i(a):
    return _dev(np.asarray(a), torch.int32)


def _bf16(a):
    t = torch.as_tensor(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


def _cache(rng, pages, nkv, hd, spread=2):
    x = rng.standard_normal((pages, nkv, PAGE, hd)) * np.exp2(rng.integers(-spread, spread + 1, (pages, nkv, PAGE, 1)))
    codes, scale, base, _ = kv4.quantise(x + rng.standard_normal((pages, nkv, PAGE, 1)))
    return kv4.pack(codes), np.stack([scale, base], axis=-1)


def _on_device(k, v):
    return [_dev(k[0]), _dev(v[0])] + [torch.as_tensor(p).to(torch.bfloat16).cuda() for p in (k[1], v[1])]


def _lim(ref, size, reach, top, L, rows):
    """Half a step of bf16; weights times V's scale in fp16, and L products below fp16's normal range, off by 2^-25
    where the row's largest stands at 1 or above; scores in fp32, off by some 2^-21 of what they add up. With more
    than 16 rows K and V go to fp16, a value by two roundings at most."""
    scores, value = 2.0 ** -21 * reach[..., None], 0.0
    if rows > 16:
        scores, value = scores + 2.0 ** -10 * reach[..., None], 2.0 ** -10
    return 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -14 + value + 2.0 * np.minimum(scores, 1.0)) * size + L * 2.0 ** -24 * top


def _check(got, ref, size, reach, v, L, rows):
    _, va = kv4.values(*v)
    err, lim = np.abs(got - ref), _lim(ref, size, reach, va.max(), L, rows)
    assert np.isfinite(got).all() and (err <= lim).all(), (err / np.maximum(lim, 1e-300)).max()


# ---------------------------------------------------------------- no page is lost, none counts twice

MANY = [
    # B, K, query heads, kv heads, width, entries
    (1, 1, 8, 1, 128, [70000]), (2, 2, 8, 1, 64, [30000, 12345]), (1, 7, 8, 1, 128, [65000]),
    (3, 5, 16, 2, 64, [9000, 40000, 77]), (300, 1, 1, 1, 64, [5000, 3, 12000, 640]),
    # shares longer than a CTA's tables, heads cut by them once and several times
    (8, 1, 8, 8, 128, [80000]), (8, 2, 8, 8, 64, [80000]), (16, 3, 64, 8, 64, [72000]), (16, 9, 16, 8, 128, [72000]),
    (50, 1, 8, 8, 64, [19200]), (64, 9, 16, 8, 64, [19200]), (64, 17, 8, 8, 128, [9600]),
    (120, 1, 8, 8, 128, [50000, 100]), (60, 3, 64, 8, 64, [60000, 31000, 9]), (40, 17, 8, 8, 128, [100000, 5])]


@pytest.mark.parametrize("B,K,nq,nkv,hd,lens", MANY)
def test_every_page_counts_once(B, K, nq, nkv, hd, lens):
    # queries of zero see every entry alike: dimension d of the output is the share of the entries whose page marks it
    S = np.resize(lens, B).astype(np.int64)
    pages = -(-(int(S.max()) + K) // PAGE)
    rng = np.random.default_rng(B + K)
    keys = _cache(rng, 64, nkv, hd)
    at = torch.as_tensor(rng.integers(0, 64, pages)).cuda()
    kc, kp = _dev(keys[0])[at].contiguous(), torch.as_tensor(keys[1]).to(torch.bfloat16).cuda()[at].contiguous()
    place = torch.arange(pages, device="cuda")
    vp = torch.zeros(pages, nkv, PAGE, 2, dtype=torch.bfloat16, device="cuda")
    vp[..., 0] = 1.0
    for share in (1, -(-pages // hd)):       # neighbours in dimensions of their own, or in runs
        dim = place // share % hd
        vc = torch.zeros(pages, nkv, PAGE, hd // 2, dtype=torch.uint8, device="cuda")
        vc[place, :, :, dim // 2] = (1 << (4 * (dim % 2))).to(torch.uint8)[:, None, None]
        table = place.to(torch.int32).expand(B, pages).contiguous()
        q = torch.zeros(B, K, nq, hd, dtype=torch.bfloat16, device="cuda")
        got, status = binding.attention_kv4(q, _i(S), table, kc, vc, kp, vp)
        assert (status == 0).all()
        got = got.double().cpu().numpy()
        dim = np.arange(pages * PAGE) // PAGE // share % hd
        for s in set(lens):
            want = np.stack([np.bincount(dim[:s + j + 1], minlength=hd) / (s + j + 1) for j in range(K)])[None, :, None, :]
            # The bf16 output. A code n is held as n - 8, and the 8 of all entries added again: every product and sum
            # of them is a whole number below 2^24 times a power of two, up to their joins by quotients and factors
            # (some 2^-22 each of the sums of 8).
            err = np.abs(got[S == s] - want)
            assert (err <= (2.0 ** -8 + 2.0 ** -14) * want + 2.0 ** -18).all(), (s, err.max())


@pytest.mark.parametrize("B,K,nq,nkv,hd,S", [(8, 1, 8, 8, 128, 80000), (16, 3, 64, 8, 64, 72000),
                                             (64, 17, 8, 8, 128, 9600), (1, 2, 8, 1, 64, 50000)])
def test_long_requests_with_scores_of_every_size(B, K, nq, nkv, hd, S):
    # the same request B times over: shares and their joins lie elsewhere in each
    rng = np.random.default_rng(B)
    k, v = _cache(rng, 200, nkv, hd, 3), _cache(rng, 200, nkv, hd)
    table = rng.integers(0, 200, (1, -(-(S + K) // PAGE))).astype(np.int32)
    qx, qt = _bf16(rng.standard_normal((1, K, nq, hd)))
    ref, _, size, reach = kv4.attention(qx, [S], None, table, [k[0], v[0]], [k[1], v[1]], hd ** -0.5)
    got, status = binding.attention_kv4(qt.expand(B, K, nq, hd).contiguous(), _i([S] * B), _i(np.repeat(table, B, 0)),
                                        *_on_device(k, v))
    assert (status == 0).all()
    got = got.double().cpu().numpy()
    for b in range(B):
        _check(got[b:b + 1], ref, size, reach, v, S + K, K * nq // nkv)


@pytest.mark.parametrize("K,nq,nkv,hd", KERNELS, ids=NAMES)
def test_thousands_of_short_requests(K, nq, nkv, hd):
    # segments of one unit, dozens of them to a CTA; some requests with no row, some refused
    rng = np.random.default_rng(nq)
    S, rows = rng.integers(0, 130, 40).astype(np.int32), rng.integers(0, K + 1, 40).astype(np.int32)
    S[7] = -1
    k, v = _cache(rng, 60, nkv, hd), _cache(rng, 60, nkv, hd)
    table = rng.integers(0, 60, (40, 9)).astype(np.int32)
    qx, qt = _bf16(rng.standard_normal((40, K, nq, hd)))
    ref, want, size, reach = kv4.attention(qx, S, rows, table, [k[0], v[0]], [k[1], v[1]], hd ** -0.5)
    got, status = binding.attention_kv4(qt.repeat(100, 1, 1, 1), _i(np.tile(S, 100)), _i(np.tile(table, (100, 1))),
                                        *_on_device(k, v), rows=_i(np.tile(rows, 100)))
    np.testing.assert_array_equal(status.cpu().numpy(), np.tile(want, 100))
    got = got.double().cpu().numpy().reshape(100, *qx.shape)
    for c in range(100):
        _check(got[c], ref, size, reach, v, 130 + K, K * nq // nkv)


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("rows", [1, 7, 9, 15, 17, 31, 33, 40, 63, 65, 88, 97, 127, 128])
def test_any_number_of_rows(rows, hd):
    # heads that one CTA has whole, and heads that several share
    rng = np.random.default_rng(rows)
    S = np.array([130, 3], dtype=np.int32)
    k, v = _cache(rng, 40, 1, hd), _cache(rng, 40, 1, hd)
    table = rng.permutation(40)[:34].reshape(2, 17).astype(np.int32)
    for K, nq in {(rows, 1), (1, rows)}:
        wide = np.concatenate([table, np.zeros((2, 4), np.int32)], axis=1)
        qx, qt = _bf16(rng.standard_normal((2, K, nq, hd)))
        ref, _, size, reach = kv4.attention(qx, S, None, wide, [k[0], v[0]], [k[1], v[1]], hd ** -0.5)
        for copies in (1, 40):
            got, status = binding.attention_kv4(qt.repeat(copies, 1, 1, 1), _i(np.tile(S, copies)),
                                                _i(np.tile(wide, (copies, 1))), *_on_device(k, v))
            assert (status == 0).all()
            for c in range(copies):
                _check(got[2 * c:2 * c + 2].double().cpu().numpy(), ref, size, reach, v, 131 + K, rows)


@pytest.mark.parametrize("K,nq,nkv,hd", KERNELS, ids=NAMES)
def test_batches_with_next_to_nothing(K, nq, nkv, hd):
    # no live row at all, then one row of one request whose cache is its own entry
    rng = np.random.default_rng(hd)
    k, v = _cache(rng, 4, nkv, hd), _cache(rng, 4, nkv, hd)
    _, qt = _bf16(rng.standard_normal((3, K, nq, hd)))
    args = [qt, _i([5, 0, 40]), _i([[0, 1, 2], [3, -1, -1], [0, 1, -1]]), *_on_device(k, v)]
    out, status = binding.attention_kv4(*args, rows=_i([0, 0, 0]), out=torch.full_like(qt, 2.0))
    assert (status == 0).all() and (out == 0).all()
    out, status = binding.attention_kv4(*args, rows=_i([0, 1, 0]), out=torch.full_like(qt, 2.0))
    assert (status == 0).all() and (out[0] == 0).all() and (out[2] == 0).all() and (out[1, 1:] == 0).all()
    own, _ = kv4.values(v[0][3, :, 0], v[1][3, :, 0])       # its only entry has all the weight
    got = out[1, 0].double().cpu().numpy().reshape(nkv, nq // nkv, hd)
    size = np.abs(own).max(-1, keepdims=True) * 2
    assert (np.abs(got - own[:, None]) <= 2.0 ** -8 * np.abs(own)[:, None] + 2.0 ** -9 * size[:, None]).all()


# ---------------------------------------------------------------- what a row does not see

@pytest.mark.parametrize("K,nq,nkv,hd", KERNELS, ids=NAMES)
@pytest.mark.parametrize("S", [45, 700])
@pytest.mark.parametrize("huge", [2.0 ** 20, 2.0 ** 100])
def test_later_entries_of_any_size_move_no_earlier_row(K, nq, nkv, hd, S, huge):
    # entry S + 2 belongs to row 2; its keys and values are far larger than the others', rows 0 and 1 do not see it
    rng = np.random.default_rng(S + hd)
    k, v = _cache(rng, 50, nkv, hd), _cache(rng, 50, nkv, hd)
    table = rng.permutation(50)[:48].reshape(1, 48).astype(np.int32)
    at = (table[0, (S + 2) // PAGE], slice(None), (S + 2) % PAGE)
    _, qt = _bf16(rng.standard_normal((1, K, nq, hd)))
    clean, _ = binding.attention_kv4(qt, _i([S]), _i(table), *_on_device(k, v))
    for side in (k, v):
        had = side[1][at].copy()
        side[1][at] = np.array([huge / 16, -huge / 2])
        got, status = binding.attention_kv4(qt, _i([S]), _i(table), *_on_device(k, v))
        side[1][at] = had
        assert (status == 0).all() and torch.equal(got[0, :2], clean[0, :2])
        assert not torch.equal(got[0, 2:], clean[0, 2:]) and torch.isfinite(got).all()


# ---------------------------------------------------------------- captured calls, streams, scratch

@pytest.mark.parametrize("B,K,nq,nkv,hd,S,width", [(3, 1, 8, 8, 128, 900, 30000), (8, 1, 8, 8, 128, 80000, 5100),
                                                   (8, 5, 32, 8, 64, 300, 30000), (16, 9, 16, 8, 128, 72000, 4600)])
def test_windows_replayed_from_a_graph(B, K, nq, nkv, hd, S, width):
    # tables with room for more than a CTA's, with and without that many entries
    rng = np.random.default_rng(B)
    cache = _on_device(_cache(rng, 100, nkv, hd), _cache(rng, 100, nkv, hd))
    table = _i(rng.integers(0, 100, (B, width)))
    lens = _i(np.full(B, S))
    q = _bf16(rng.standard_normal((B, K, nq, hd)))[1]
    want, status = binding.attention_kv4(q, lens, table, *cache)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got, _ = binding.attention_kv4(q, lens, table, *cache)
    for _ in range(5):
        got.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and (status == 0).all()
    narrow, _ = binding.attention_kv4(q, lens, table[:, :-(-(S + K) // PAGE)].contiguous(), *cache)
    assert torch.equal(narrow, want)


@pytest.mark.parametrize("K", [1, 9])
def test_scratch_does_not_follow_the_page_table(K):
    need = [binding._kv4_scratch(0, 256, K, 64, 8, 128, pages) for pages in (64, 512, 8192, 100000)]
    tile = (128 if K > 1 else 8) * (128 + 2)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert len(set(need)) == 1 and need[0] <= sms * (2 * tile + 4) + 16


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K", [1, 6])
def test_rows_and_scratch_at_sixteen_bytes(K, hd):
    # neither the output's rows nor the scratch begin on 32 bytes; the result is that of aligned ones
    B, nq, nkv, S = 4, 16, 2, 900
    rng = np.random.default_rng(hd)
    dev = _on_device(_cache(rng, 30, nkv, hd), _cache(rng, 30, nkv, hd))
    table, lens = _i(rng.integers(0, 30, (B, 60))), _i([S, 3, 200, S - 7])
    q = _bf16(rng.standard_normal((B, K, nq, hd)))[1]
    want, _ = binding.attention_kv4(q, lens, table, *dev)
    lib, width = binding.load(), nq * hd
    need = binding._kv4_scratch(0, B, K, nq, nkv, hd, 60)
    ws = torch.empty(need + 4, device="cuda")
    wide = torch.full((B * K, width + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    status = _i([9] * B)
    rc = lib.pe_attention_kv4(B, K, nq, nkv, hd, q.data_ptr(), width, lens.data_ptr(), None, table.data_ptr(), 60, 30,
                              dev[0].data_ptr(), dev[1].data_ptr(), dev[2].data_ptr(), dev[3].data_ptr(), hd ** -0.5,
                              wide.data_ptr() + 16, width + 24, ws.data_ptr() + 16, need, status.data_ptr(),
                              torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and (status == 0).all()
    assert torch.equal(wide[:, 8:8 + width].reshape(want.shape), want)
    assert (wide[:, :8] == 3).all() and (wide[:, 8 + width:] == 3).all()


@pytest.mark.parametrize("K,nq", [(1, 4), (9, 4)])
def test_cache_past_four_gigabytes(K, nq):
    # the same rows written and read through pages at the end of a cache of 4.7 GB a half, and through low ones
    nkv, hd, pages = 1, 128, 4_600_000
    rng = np.random.default_rng(K)
    S, n = np.array([37, 5]), 90
    k, v = (torch.as_tensor(rng.standard_normal((2, n, nkv, hd))).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.as_tensor(rng.standard_normal((2, K, nq, hd))).to(torch.bfloat16).cuda()
    low = rng.permutation(20)[:16].reshape(2, 8).astype(np.int32)
    results = []
    for count, table in ((20, low), (pages, pages - 1 - low)):
        cache = [torch.empty((count, nkv, PAGE, hd // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
        cache += [torch.empty((count, nkv, PAGE, 2), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        _, status = binding.kv4_append(k, v, _i([0, 0]), _i(table), *cache, theta=1e4)
        assert (status == 0).all()
        out, status = binding.attention_kv4(q, _i(S), _i(table), *cache)
        assert (status == 0).all()
        at = torch.as_tensor(table.ravel().astype(np.int64)).cuda()
        results.append([out] + [c[at].view(2, 8, -1)[:, :5].clone() for c in cache])
        del cache
    for a, b in zip(*results):
        assert torch.equal(a, b)


# ---------------------------------------------------------------- a wait that gives up

@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("barrier,width", [(1, 60), (2, 60), (3, 60), (2, 60000)])
def test_waits_that_give_up_refuse_the_call_and_leave_the_next_alone(barrier, width, hd):
    # Host-side injection: a barrier of the tensor-memory kernel waits for one arrival more than there are. Its waits
    # end after their limit; every request with rows reports it, and all outputs are zero.
    rng = np.random.default_rng(barrier + hd)
    B, K, nq, nkv = 5, 6, 16, 2
    S, rows = [900, 30, 7, -1, 300], _i([6, 3, 0, 6, 6])
    _, qt = _bf16(rng.standard_normal((B, K, nq, hd)))
    args = [qt, _i(S), _i(rng.integers(0, 80, (B, width))), *_on_device(_cache(rng, 80, nkv, hd), _cache(rng, 80, nkv, hd))]
    clean, status = binding.attention_kv4(*args, rows=rows)
    assert status.tolist() == [0, 0, 0, binding.PE_REQ_BAD_INPUT, 0] and (clean[0] != 0).any()
    torch.cuda.synchronize()
    binding.test_stall_attention_kv4(barrier)
    few, status = binding.attention_kv4(qt[:, :1, :nkv].contiguous(), *args[1:])   # few rows: another kernel
    assert (status[[0, 1, 2, 4]] == 0).all()
    t0 = time.time()
    out = torch.full_like(qt, 3.0)
    out, status = binding.attention_kv4(*args, rows=rows, out=out)
    torch.cuda.synchronize()
    assert 0.5 < time.time() - t0 < 20.0
    late = binding.PE_REQ_TIMEOUT
    assert status.tolist() == [late, late, 0, binding.PE_REQ_BAD_INPUT, late] and (out == 0).all()
    out, status = binding.attention_kv4(*args, rows=rows)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 0, 0, binding.PE_REQ_BAD_INPUT, 0] and torch.equal(out, clean)


# ---------------------------------------------------------------- a server's step

class _Server:
    """Steps of one layer and a vocabulary on the device: pages, cache write with the rotation, attention, log
    probabilities; lengths stay on the device."""

    def __init__(self, rng, B, n, nq, nkv, hd, V, pages):
        self.B, self.n, self.V = B, n, V
        self.qkv = torch.as_tensor(rng.standard_normal((B, n, (nq + 2 * nkv) * hd))).to(torch.bfloat16).cuda()
        heads = self.qkv.unflatten(-1, (nq + 2 * nkv, hd))
        self.q, self.k, self.v = heads[:, :, :nq], heads[:, :, nq:nq + nkv], heads[:, :, nq + nkv:]
        self.head = torch.as_tensor(rng.standard_normal((V, nq * hd)) / hd).to(torch.bfloat16).cuda()
        self.lens, self.rows, self.counts = _i([0] * B), _i([n] * B), _i([0] * B)
        self.table, self.free, self.left = _i(np.full((B, 8), -1)), _i(rng.permutation(pages)), _i([pages])
        self.cache = [torch.zeros(pages, nkv, PAGE, hd // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
        self.cache += [torch.zeros(pages, nkv, PAGE, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        self.tokens = _i(rng.integers(0, V, (B, n)))
        self.pages = pages

    def step(self, stream=None):
        o = binding.assign_pages(self.lens, self.rows, self.counts, self.table, self.free, self.left, self.pages, self.n,
                                 stream=stream)
        q, wrote = binding.kv4_append(self.k, self.v, self.lens, self.table, *self.cache, rows=self.rows, theta=1e4, q=self.q,
                                      stream=stream)
        out, seen = binding.attention_kv4(q, self.lens, self.table, *self.cache, rows=self.rows, stream=stream)
        with torch.cuda.stream(stream):      # (its output comes from the current stream's memory)
            logits = binding.linear(self.head, out.view(self.B * self.n, -1), stream=stream)
        said = binding.token_logprobs(logits.view(self.B, self.n, self.V), self.tokens, top=4, stream=stream)
        return [o["page_counts"], o["free_count"], wrote, q, seen, out, *said.values()]


def test_steps_of_a_server():
    # three steps of uneven growth: each equals float64 on what the step before has left
    rng = np.random.default_rng(11)
    B, n, nq, nkv, hd, V = 5, 6, 8, 2, 64, 640
    s = _Server(rng, B, n, nq, nkv, hd, V, 40)
    S = np.zeros(B, dtype=np.int64)
    for rows in ([6, 1, 0, 6, 3], [1, 6, 6, 2, 0], [6, 6, 6, 6, 6]):
        s.lens, s.rows = _i(S), _i(rows)
        counts, left, wrote, q, seen, out, at, h, ids, best = s.step()
        torch.cuda.synchronize()
        s.counts, s.left = counts, left
        assert (wrote == 0).all() and (seen == 0).all()
        codes, params = [c.cpu().numpy() for c in s.cache[:2]], [c.float().cpu().numpy() for c in s.cache[2:]]
        table = s.table.cpu().numpy()
        for b in range(B):      # the queries as they were turned
            x = kv4.rotate(s.q[b, 0].double().cpu().numpy(), int(S[b]), 1e4) if rows[b] else np.zeros((nq, hd))
            assert np.abs(q[b, 0].double().cpu().numpy() - x).max() <= 2.0 ** -8 * np.abs(x).max() + 2.0 ** -20
        ref, _, size, reach = kv4.attention(q.double().cpu().numpy(), S, rows, table, codes, params, hd ** -0.5)
        _check(out.double().cpu().numpy(), ref, size, reach, (codes[1], params[1]), int(S.max()) + n, n * nq // nkv)
        logits = binding.linear(s.head, out.view(B * n, -1)).double().cpu().numpy()
        want = kv4.token_logprobs(logits, s.tokens.cpu().numpy().ravel(), 4, 1.0)
        for got, ref in zip((at, h, ids, best), want):
            np.testing.assert_allclose(got.double().cpu().numpy().reshape(ref.shape), ref, rtol=2.0 ** -19, atol=2.0 ** -19)
        S = S + rows


def test_steps_on_a_given_stream_and_from_a_graph(monkeypatch):
    make = lambda: _Server(np.random.default_rng(2), 3, 9, 16, 2, 64, 700, 30)
    plain = make()
    want = plain.step()
    torch.cuda.synchronize()
    other, side, seen = make(), torch.cuda.Stream(), []
    torch.cuda.synchronize()
    real = torch.empty
    with monkeypatch.context() as m:
        m.setattr(torch, "empty", lambda *a, **k: seen.append(torch.cuda.current_stream()) or real(*a, **k))
        got = other.step(side)
    torch.cuda.synchronize()
    assert len(seen) >= 10 and all(t == side for t in seen)
    caught = make()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = caught.step()
    fresh = [t.clone() for t in (caught.table, caught.free, *caught.cache)]
    for _ in range(3):
        for t, f in zip((caught.table, caught.free, *caught.cache), fresh):
            t.copy_(f)
        graph.replay()
        torch.cuda.synchronize()
        for a, b, c in zip(want, got, kept):
            assert torch.equal(a, b) and torch.equal(a, c)
        for a, b, c in zip(plain.cache, other.cache, caught.cache):
            assert torch.equal(a, b) and torch.equal(a, c)


def test_two_graphs_and_eager_calls_share_nothing():
    # captured calls of one operator run beside each other on two streams
    rng = np.random.default_rng(5)
    nkv, hd, B, K = 2, 128, 4, 9
    cache = _on_device(_cache(rng, 60, nkv, hd), _cache(rng, 60, nkv, hd))
    table = _i(rng.integers(0, 60, (B, 130)))
    logits = torch.as_tensor(rng.standard_normal((9, 30000))).to(torch.bfloat16).cuda()
    tokens = _i(rng.integers(0, 30000, 9))
    jobs = []
    for S in (2000, 77):
        q = _bf16(rng.standard_normal((B, K, 8, hd)))[1]
        lens = _i([S, 3, S // 2, 60])
        run = lambda q=q, lens=lens: [*binding.attention_kv4(q, lens, table, *cache),
                                      *binding.token_logprobs(logits, tokens, top=7).values()]
        want = [t.clone() for t in run()]
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            got = run()
        jobs.append((stream, graph, got, want, run))
    for _ in range(10):
        for stream, graph, *_ in jobs:
            with torch.cuda.stream(stream):
                graph.replay()
        eager = jobs[0][4]()
        torch.cuda.synchronize()
        for _, _, got, want, _ in jobs:
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(eager, jobs[0][3]))
