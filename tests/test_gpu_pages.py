"""Pages on the device: assignment from a free stack, slot maps and release, against a request-at-a-time restatement."""

import numpy as np
import pytest
import torch

from oracle import lowbit
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu


def _i(a):
    return torch.as_tensor(np.asarray(a, dtype=np.int32), device="cuda")


def _batch(B, hi, n_max, max_pages, extra, seed):
    rng = np.random.default_rng(seed)
    S = rng.integers(0, hi + 1, B)
    counts = -(-S // 16)
    counts = np.minimum(counts + rng.integers(0, 2, B), max_pages)   # some hold a page ahead
    ids = rng.permutation(int(counts.sum()) + extra)
    table = np.full((B, max_pages), -1, dtype=np.int32)
    at = 0
    for b in range(B):
        table[b, :counts[b]] = ids[at:at + counts[b]]
        at += counts[b]
    return S.astype(np.int32), rng.integers(0, n_max + 1, B).astype(np.int32), counts.astype(np.int32), table, \
        ids[at:].astype(np.int32), len(ids)


def _check(S, n, counts, table, free, F, num_pages, n_max):
    want = lowbit.assign_pages(S, n, counts, table, free, F, num_pages, n_max)
    t = _i(table)
    o = binding.assign_pages(_i(S), _i(n), _i(counts), t, _i(free), _i([F]), num_pages, n_max)
    torch.cuda.synchronize()
    for name, got, ref in (("slots", o["slot_mapping"], want[0]), ("counts", o["page_counts"], want[1]),
                           ("table", t, want[2]), ("status", o["status"], want[4])):
        np.testing.assert_array_equal(got.cpu().numpy(), ref, err_msg=name)
    assert int(o["free_count"].item()) == want[3]
    return want


@pytest.mark.parametrize("B,hi,n_max,max_pages,extra", [
    (1, 0, 1, 1, 4), (1, 40, 5000, 400, 600), (5, 100, 7, 8, 40), (64, 4096, 8, 300, 300), (300, 60, 33, 9, 1200),
    (1500, 30, 3, 4, 3000), (7, 15, 2049, 140, 2000)])
def test_assign_matches_the_sequential_rule(B, hi, n_max, max_pages, extra):
    S, n, counts, table, free, total = _batch(B, hi, n_max, max_pages, extra, B + n_max)
    _check(S, n, counts, table, free, len(free), total, n_max)


@pytest.mark.parametrize("left", [0, 1, 5, 19])
def test_assign_with_a_stack_that_runs_dry(left):
    S, n, counts, table, free, total = _batch(40, 50, 20, 6, 60, left)
    want = _check(S, n, counts, table, free, left, total, 20)
    whole = lowbit.assign_pages(S, n, counts, table, free, len(free), total, 20)
    assert (want[4] == lowbit.CAPACITY).any() == (len(free) - whole[3] > left)


def test_assign_refuses_requests_alone():
    S, n, counts, table, free, total = _batch(12, 90, 9, 8, 60, 3)
    S[1], n[2], n[3], counts[4], counts[5] = -1, -3, 10, -1, 9      # lengths and counts out of range
    S[6], counts[6] = 100, 2                                        # committed entries without a page
    S[7], counts[7], n[7] = 128, 8, 4                               # past the table
    table[8, 0] = -1
    S[8], counts[8], n[8] = 3, 1, 2                                 # a page of the new entries is missing
    free[-1] = total + 7                                            # a stack entry outside the pool
    want = _check(S, n, counts, table, free, len(free), total, 9)
    assert set(want[4]) == {0, 1, 2, 3}


def test_assign_leaves_rows_behind_the_request_alone():
    t = _i(np.full((2, 6), 77))
    o = binding.assign_pages(_i([0, 0]), _i([17, 0]), _i([0, 0]), t, _i([4, 5, 6]), _i([3]), 8, 20)
    assert t.cpu().tolist() == [[6, 5, 77, 77, 77, 77], [77] * 6]
    assert o["free_count"].item() == 1 and o["page_counts"].tolist() == [2, 0]


@pytest.mark.parametrize("B,seed", [(1, 0), (33, 1), (1024, 2), (2100, 3)])
def test_release_matches_the_sequential_rule(B, seed):
    rng = np.random.default_rng(seed)
    S, _, counts, table, free, total = _batch(B, 200, 4, 14, 50, seed)
    keep = np.where(rng.random(B) < 0.3, 0, np.minimum(S, rng.integers(0, 220, B))).astype(np.int32)
    if B > 30:
        keep[3], counts[4], table[5, 0], keep[5], counts[5] = -1, 15, total, 0, max(1, counts[5])
    stack = np.concatenate([free, np.full(total - len(free), -5, np.int32)]).astype(np.int32)
    for cap in (len(stack), len(free) + 20):
        want = lowbit.release_pages(keep, counts, table, stack[:cap], len(free), total)
        c, t, s, f = _i(counts), _i(table), _i(stack[:cap]), _i([len(free)])
        status = binding.release_pages(_i(keep), c, t, s, f, total)
        torch.cuda.synchronize()
        for name, got, ref in (("counts", c, want[0]), ("table", t, want[1]), ("stack", s, want[2]),
                               ("status", status, want[4])):
            np.testing.assert_array_equal(got.cpu().numpy(), ref, err_msg=name)
        assert f.item() == want[3]


def test_assign_and_release_in_a_captured_step():
    # a graph whose replays walk the counts forward, as a server's step does
    S, counts, f = _i([0, 0, 0]), _i([0, 0, 0]), _i([30])
    n, t, stack = _i([5, 16, 1]), _i(np.full((3, 10), -1)), _i(np.arange(30))

    def step():
        o = binding.assign_pages(S, n, counts, t, stack, f, 30, 16)
        counts.copy_(o["page_counts"])
        f.copy_(o["free_count"])
        S.add_(n)
        return o

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    S.zero_(), counts.zero_(), f.fill_(30), t.fill_(-1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step()
    left, cnt, table = 30, np.zeros(3, np.int32), np.full((3, 10), -1, np.int32)
    for i in range(6):
        graph.replay()
        slots, cnt, table, left, status = lowbit.assign_pages(np.array([5, 16, 1]) * i, [5, 16, 1], cnt, table,
                                                              np.arange(30), left, 30, 16)
        np.testing.assert_array_equal(o["slot_mapping"].cpu().numpy(), slots)
        np.testing.assert_array_equal(t.cpu().numpy(), table)
        assert f.item() == left
    binding.release_pages(_i([0, 0, 0]), counts, t, stack, f, 30)
    assert f.item() == 30 and sorted(stack.tolist()) == list(range(30)) and (t == -1).all()
