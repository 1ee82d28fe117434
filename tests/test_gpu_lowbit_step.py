"""The low-bit serving operators as a server runs them: a projection with 4-bit weights, pages, the 8-bit cache
written and attended over, the output projection and the rejected tokens' pages given back, step after step, each
stage against float64 on what the stage before it gave. And the attention's shares of work at its limits."""

import numpy as np
import pytest
import torch

from oracle import lowbit
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu

PAGE = 16


def _i(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32), device="cuda")


def _cpu(t):
    return t.double().cpu().numpy()


def _weights(rng, M, Kd, group):
    w = rng.integers(0, 256, (M, Kd // 2), dtype=np.uint8)
    s = torch.as_tensor(rng.uniform(0.5, 1.5, (M, -(-Kd // group))) / (4.0 * Kd ** 0.5)).to(torch.bfloat16)
    return w, s


def _check_linear(y, x, w, s, group):
    """The bound of a 4-bit product: fp32 sums of the groups' steps, and x below 2^-28 of its row's largest value."""
    W, size = lowbit.unpack_w4(w, s.double().numpy(), None, group)
    X = _cpu(x)
    steps = group // 16 + -(-X.shape[1] // group) + 16
    lim = steps * 2.0 ** -23 * (np.abs(X) @ size.T) + 2.0 ** -35 * np.abs(X).max(1, keepdims=True) * size.sum(1)
    assert (np.abs(_cpu(y) - X @ W.T) <= lim).all()


def _check_attention(got, ref, size, top, L):
    """Half a step of bf16; fp16 weights and fp32 scores; weights below fp16's normal range, L of them at most."""
    lim = 2.0 ** -8 * np.abs(ref) + (2.0 ** -11 + 2.0 ** -13) * size + L * 2.0 ** -25 * top
    assert (np.abs(got - ref) <= lim).all()


class Server:
    """One layer's state and weights; `step` is what a captured graph holds."""

    def __init__(self, seed, B, n, nq, nkv, hd, max_pages, pool):
        rng = np.random.default_rng(seed)
        self.n, self.nq, self.nkv, self.hd, self.pool = n, nq, nkv, hd, pool
        H = self.H = nq * hd
        self.group = 64
        self.w_qkv, self.s_qkv = _weights(rng, (nq + 2 * nkv) * hd, H, self.group)
        self.w_o, self.s_o = _weights(rng, H, H, self.group)
        self.dev_w = [torch.as_tensor(self.w_qkv).cuda(), self.s_qkv.cuda(), torch.as_tensor(self.w_o).cuda(),
                      self.s_o.cuda()]
        self.x = torch.zeros((B * n, H), dtype=torch.bfloat16, device="cuda")
        self.S, self.new, self.keep = _i(np.zeros(B)), _i(np.zeros(B)), _i(np.zeros(B))
        self.counts, self.table = _i(np.zeros(B)), _i(np.full((B, max_pages), -1))
        self.free, self.left = _i(rng.permutation(pool)), _i([pool])
        self.kc = torch.full((pool, nkv, PAGE, hd), 0x7F, dtype=torch.uint8, device="cuda")
        self.vc = self.kc.clone()
        self.ks = torch.full((pool, nkv), float("nan"), device="cuda")
        self.vs = self.ks.clone()

    def step(self):
        B, n, nq, nkv, hd = self.S.shape[0], self.n, self.nq, self.nkv, self.hd
        w_qkv, s_qkv, w_o, s_o = self.dev_w
        y = binding.linear_w4(w_qkv, s_qkv, self.x, self.group)
        qkv = y.to(torch.bfloat16).view(B, n, nq + 2 * nkv, hd)
        q, k, v = qkv.split([nq, nkv, nkv], dim=2)
        o = binding.assign_pages(self.S, self.new, self.counts, self.table, self.free, self.left, self.pool, n)
        self.counts.copy_(o["page_counts"])
        self.left.copy_(o["free_count"])
        # a request that got no pages runs no rows
        rows = torch.where(o["status"] == 0, self.new, 0)
        written = binding.kv8_append(k, v, self.S, self.table, self.kc, self.vc, self.ks, self.vs, rows=rows)
        a, seen = binding.attention_kv8(q, self.S, self.table, self.kc, self.vc, self.ks, self.vs, rows=rows)
        out = binding.linear_w4(w_o, s_o, a.view(B * n, nq * hd), self.group)
        kept = torch.where(o["status"] == 0, torch.minimum(self.keep, self.S + rows), self.S)
        back = binding.release_pages(kept, self.counts, self.table, self.free, self.left, self.pool)
        return dict(y=y, qkv=qkv, slots=o["slot_mapping"], status=o["status"], written=written, a=a, seen=seen,
                    out=out, back=back, kept=kept, rows=rows)


def _plan(rng, B, n, S):
    """New rows of each request, and the entries it keeps of them (0: it ends)."""
    new = rng.integers(0, n + 1, B)
    keep = S + rng.integers(0, new + 1)
    keep[rng.random(B) < 0.08] = 0
    return new, keep


SHAPES = [(5, 4, 4, 2, 64, 12, 26), (3, 11, 16, 2, 128, 9, 60), (7, 1, 8, 1, 64, 6, 40), (40, 3, 4, 4, 64, 4, 100)]


@pytest.mark.parametrize("B,n,nq,nkv,hd,max_pages,pool", SHAPES)
def test_steps_of_a_server(B, n, nq, nkv, hd, max_pages, pool):
    sv = Server(B + hd, B, n, nq, nkv, hd, max_pages, pool)
    rng = np.random.default_rng(n)
    S = np.zeros(B, dtype=np.int32)
    for _ in range(14):
        new, keep = _plan(rng, B, n, S)
        x = torch.as_tensor(rng.standard_normal((B * n, nq * hd))).to(torch.bfloat16)
        sv.x.copy_(x)
        sv.S.copy_(_i(S)), sv.new.copy_(_i(new)), sv.keep.copy_(_i(keep))
        had = [a.cpu().numpy().copy() for a in (sv.counts, sv.table, sv.free, sv.left, sv.kc, sv.vc, sv.ks, sv.vs)]
        o = sv.step()
        torch.cuda.synchronize()
        counts, table, free, left, kc, vc, ks, vs = had
        _check_linear(o["y"], sv.x, sv.w_qkv, sv.s_qkv, sv.group)
        slots, counts, table, left, status = lowbit.assign_pages(S, new, counts, table, free, left[0], pool, n)
        np.testing.assert_array_equal(o["slots"].cpu().numpy(), slots)
        np.testing.assert_array_equal(o["status"].cpu().numpy(), status)
        rows = np.where(status == 0, new, 0)
        qkv = _cpu(o["qkv"])
        q, k, v = np.split(qkv, [nq, nq + nkv], axis=2)
        kc, vc, ks, vs, written = lowbit.kv8_append(k, v, S, rows, table, kc, vc, ks, vs)
        np.testing.assert_array_equal(o["written"].cpu().numpy(), written)
        for got, ref in ((sv.kc, kc), (sv.vc, vc), (sv.ks, ks), (sv.vs, vs)):
            np.testing.assert_array_equal(got.cpu().numpy(), ref)
        ref, seen, size = lowbit.attention_kv8(q, S, rows, table, kc, vc, ks, vs, hd ** -0.5)
        np.testing.assert_array_equal(o["seen"].cpu().numpy(), seen)
        top = np.nanmax(np.abs(lowbit.e4m3_decode(vc) * vs.astype(np.float64)[:, :, None, None]), initial=0.0)
        _check_attention(_cpu(o["a"]), ref, size, top, int(S.max()) + n)
        _check_linear(o["out"], o["a"].view(B * n, nq * hd), sv.w_o, sv.s_o, sv.group)
        kept = np.where(status == 0, np.minimum(keep, S + rows), S)
        counts, table, free, left, back = lowbit.release_pages(kept, counts, table, free, left, pool)
        np.testing.assert_array_equal(o["back"].cpu().numpy(), back)
        np.testing.assert_array_equal(sv.counts.cpu().numpy(), counts)
        np.testing.assert_array_equal(sv.table.cpu().numpy(), table)
        np.testing.assert_array_equal(sv.free.cpu().numpy()[:left], free[:left])
        assert int(sv.left.item()) == left
        # every page is on the stack or with one request
        held = np.concatenate([table[b, :counts[b]] for b in range(B)] + [free[:left]])
        assert sorted(held) == list(range(pool))
        S = kept.astype(np.int32)


def test_steps_replayed_from_a_graph_equal_the_calls():
    B, n, nq, nkv, hd, max_pages, pool = SHAPES[0]
    eager, graphed = (Server(1, B, n, nq, nkv, hd, max_pages, pool) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graphed.step()      # lengths of zero: nothing is taken
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = graphed.step()
    rng = np.random.default_rng(3)
    S = np.zeros(B, dtype=np.int32)
    for _ in range(12):
        new, keep = _plan(rng, B, n, S)
        x = torch.as_tensor(rng.standard_normal((B * n, nq * hd))).to(torch.bfloat16)
        for sv in (eager, graphed):
            sv.x.copy_(x)
            sv.S.copy_(_i(S)), sv.new.copy_(_i(new)), sv.keep.copy_(_i(keep))
        graph.replay()
        want = eager.step()
        torch.cuda.synchronize()
        for name in want:
            assert torch.equal(got[name], want[name]), name
        assert torch.equal(eager.table, graphed.table) and torch.equal(eager.kc, graphed.kc)
        S = want["kept"].cpu().numpy()


# ---------------------------------------------------------------- the attention's shares of work

def _pool(rng, pages, nkv, hd):
    x = rng.standard_normal((pages, nkv, PAGE, hd))
    s = np.array([[lowbit.kv8_scale(x[p, h]) for h in range(nkv)] for p in range(pages)], dtype=np.float32)
    return lowbit.e4m3_encode(x / s[:, :, None, None]), s


def _attend(q, S, table, kc, vc, ks, vs, **kw):
    dev = [torch.as_tensor(a).cuda() for a in (kc, vc, ks, vs)]
    got, status = binding.attention_kv8(q, _i(S), _i(table), *dev, **kw)
    torch.cuda.synchronize()
    assert (status == 0).all()
    return got


@pytest.mark.parametrize("K,nq,nkv,hd", [(1, 8, 2, 128), (5, 8, 2, 64), (3, 32, 2, 128)])
def test_attention_with_a_page_table_far_wider_than_the_requests(K, nq, nkv, hd):
    rng = np.random.default_rng(K)
    S = rng.integers(0, 400, 30).astype(np.int32)
    kc, ks = _pool(rng, 40, nkv, hd)
    vc, vs = _pool(rng, 40, nkv, hd)
    narrow = rng.integers(0, 40, (30, 27)).astype(np.int32)      # pages shared between requests, some twice in one
    wide = np.full((30, 60000), -1, dtype=np.int32)
    wide[:, :27] = narrow
    q = torch.as_tensor(rng.standard_normal((30, K, nq, hd))).to(torch.bfloat16)
    got = _cpu(_attend(q.cuda(), S, wide, kc, vc, ks, vs))
    ref, _, size = lowbit.attention_kv8(q.double().numpy(), S, None, narrow, kc, vc, ks, vs, hd ** -0.5)
    top = np.abs(lowbit.e4m3_decode(vc) * vs.astype(np.float64)[:, :, None, None]).max()
    _check_attention(got, ref, size, top, 400 + K)


@pytest.mark.parametrize("B,K,nq,S", [(8, 1, 8, 40000), (16, 3, 64, 36000)])
def test_attention_of_more_entries_than_one_share_per_multiprocessor_holds(B, K, nq, S):
    # the same long request B times over
    nkv, hd = 8, 64
    rng = np.random.default_rng(B)
    kc, ks = _pool(rng, 50, nkv, hd)
    vc, vs = _pool(rng, 50, nkv, hd)
    table = rng.integers(0, 50, (1, S // PAGE + 1)).astype(np.int32)
    q = torch.as_tensor(rng.standard_normal((1, K, nq, hd))).to(torch.bfloat16)
    got = _attend(q.cuda().expand(B, K, nq, hd).contiguous(), [S] * B, np.repeat(table, B, 0), kc, vc, ks, vs)
    ref, _, size = lowbit.attention_kv8(q.double().numpy(), [S], None, table, kc, vc, ks, vs, hd ** -0.5)
    top = np.abs(lowbit.e4m3_decode(vc) * vs.astype(np.float64)[:, :, None, None]).max()
    for b in range(B):
        _check_attention(_cpu(got[b:b + 1]), ref, size, top, S + K)


@pytest.mark.parametrize("hd", [64, 128])
def test_attention_into_rows_and_scratch_at_sixteen_bytes(hd):
    # neither the output's rows nor the scratch begin on 32 bytes; the result is that of aligned ones
    B, K, nq, nkv, S = 4, 6, 16, 2, 900
    rng = np.random.default_rng(hd)
    kc, ks = _pool(rng, 30, nkv, hd)
    vc, vs = _pool(rng, 30, nkv, hd)
    dev = [torch.as_tensor(a).cuda() for a in (kc, vc, ks, vs)]
    table, lens = _i(rng.integers(0, 30, (B, 60))), _i([S, 3, 200, S - 7])
    q = torch.as_tensor(rng.standard_normal((B, K, nq, hd))).to(torch.bfloat16).cuda()
    want, _ = binding.attention_kv8(q, lens, table, *dev)
    lib, width = binding.load(), nq * hd
    need = binding._kv8_scratch(0, B, K, nq, nkv, hd, 60)
    ws = torch.empty(need + 4, device="cuda")
    wide = torch.full((B * K, width + 24), 3.0, dtype=torch.bfloat16, device="cuda")
    status = _i([9] * B)
    rc = lib.pe_attention_kv8(B, K, nq, nkv, hd, q.data_ptr(), width, lens.data_ptr(), None, table.data_ptr(), 60, 30,
                              dev[0].data_ptr(), dev[1].data_ptr(), dev[2].data_ptr(), dev[3].data_ptr(), hd ** -0.5,
                              wide.data_ptr() + 16, width + 24, ws.data_ptr() + 16, need, status.data_ptr(),
                              torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc == 0 and (status == 0).all()
    assert torch.equal(wide[:, 8:8 + width].reshape(want.shape), want)
    assert (wide[:, :8] == 3).all() and (wide[:, 8 + width:] == 3).all()


def test_calls_on_a_given_stream_allocate_for_it(monkeypatch):
    rng = np.random.default_rng(4)
    nkv, hd, B, K = 2, 64, 3, 6
    kc, ks = _pool(rng, 30, nkv, hd)
    vc, vs = _pool(rng, 30, nkv, hd)
    q = torch.as_tensor(rng.standard_normal((B, K, 16, hd))).to(torch.bfloat16).cuda()
    kv = torch.as_tensor(rng.standard_normal((B, K, nkv, hd))).to(torch.bfloat16).cuda()
    w = torch.as_tensor(rng.integers(0, 256, (80, 128), dtype=np.uint8)).cuda()
    s = torch.ones(80, 4, device="cuda")
    x = torch.ones(2, 256, dtype=torch.bfloat16, device="cuda")

    def run(stream):
        cache = [torch.as_tensor(a).cuda() for a in (kc, vc, ks, vs)]
        table, free, left = _i(np.full((B, 8), -1)), _i(np.arange(30)), _i([30])
        lens, new, counts = _i([0, 0, 0]), _i([100, 3, 60]), _i([0, 0, 0])
        S = _i([94, 0, 54])
        torch.cuda.synchronize()
        seen = []
        with monkeypatch.context() as m:
            real = torch.empty
            m.setattr(torch, "empty", lambda *a, **k: seen.append(torch.cuda.current_stream()) or real(*a, **k))
            o = binding.assign_pages(lens, new, counts, table, free, left, 30, 100, stream=stream)
            written = binding.kv8_append(kv, kv, S, table, *cache, rows=_i([6, 3, 6]), stream=stream)
            out, seen_ok = binding.attention_kv8(q, S, table, *cache, rows=_i([6, 3, 6]), stream=stream)
            y = binding.linear_w4(w, s, x, 64, stream=stream)
            back = binding.release_pages(lens, o["page_counts"], table, free, o["free_count"], 30, stream=stream)
        torch.cuda.synchronize()
        return [o["slot_mapping"], o["status"], written, out, seen_ok, y, back, free, table, *cache], seen

    side = torch.cuda.Stream()
    want, _ = run(None)
    got, seen = run(side)
    assert len(seen) >= 10 and all(t == side for t in seen)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("K,nq", [(1, 4), (6, 4)])
def test_cache_past_four_gigabytes(K, nq):
    # the same rows written and read through pages at the end of a cache of 4.7 GB a half, and through low ones
    nkv, hd, pages = 1, 128, 2_300_000
    rng = np.random.default_rng(K)
    S, n = np.array([37, 5]), 90
    k, v = (torch.as_tensor(rng.standard_normal((2, n, nkv, hd))).to(torch.bfloat16).cuda() for _ in range(2))
    q = torch.as_tensor(rng.standard_normal((2, K, nq, hd))).to(torch.bfloat16).cuda()
    low = rng.permutation(20)[:16].reshape(2, 8).astype(np.int32)
    results = []
    for count, table in ((20, low), (pages, pages - 1 - low)):
        cache = [torch.empty((count, nkv, PAGE, hd), dtype=torch.uint8, device="cuda") for _ in range(2)]
        cache += [torch.empty((count, nkv), device="cuda") for _ in range(2)]
        zero = _i([0, 0])
        assert (binding.kv8_append(k, v, zero, _i(table), *cache) == 0).all()
        out, status = binding.attention_kv8(q, _i(S), _i(table), *cache)
        assert (status == 0).all()
        at = torch.as_tensor(table.ravel().astype(np.int64)).cuda()
        results.append([out] + [c[at].view(2, 8, -1)[:, :5].clone() for c in cache])
        del cache
    for a, b in zip(*results):
        assert torch.equal(a, b)


def test_attention_of_thousands_of_requests():
    rng = np.random.default_rng(6)
    B, K, nq, nkv, hd = 2500, 2, 2, 1, 64
    kc, ks = _pool(rng, 40, nkv, hd)
    vc, vs = _pool(rng, 40, nkv, hd)
    S, rows = rng.integers(0, 40, B).astype(np.int32), rng.integers(0, K + 1, B).astype(np.int32)
    S[rng.random(B) < 0.05] = -1
    table = rng.integers(0, 40, (B, 3)).astype(np.int32)
    q = torch.as_tensor(rng.standard_normal((B, K, nq, hd))).to(torch.bfloat16)
    dev = [torch.as_tensor(a).cuda() for a in (kc, vc, ks, vs)]
    got, status = binding.attention_kv8(q.cuda(), _i(S), _i(table), *dev, rows=_i(rows))
    torch.cuda.synchronize()
    ref, want, size = lowbit.attention_kv8(q.double().numpy(), S, rows, table, kc, vc, ks, vs, hd ** -0.5)
    np.testing.assert_array_equal(status.cpu().numpy(), want)
    top = np.abs(lowbit.e4m3_decode(vc) * vs.astype(np.float64)[:, :, None, None]).max()
    _check_attention(_cpu(got), ref, size, top, 42)
