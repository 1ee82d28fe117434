"""Attention over the 4-bit cache where one entry has all of a row's weight and others' values are far larger."""

import numpy as np
import pytest
import torch

from oracle import kv4
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu

PAGE = 16
# K and query heads of a kv head: one and two tiles of the register kernels' rows, the tensor-memory kernels
ROWS = [(1, 8), (2, 8), (11, 8)]


def _i(a):
    return torch.as_tensor(np.asarray(a), dtype=torch.int32).cuda()


def _bf16(a):
    t = torch.as_tensor(np.asarray(a, dtype=np.float32)).to(torch.bfloat16)
    return t.double().numpy(), t.cuda()


def _store(x):
    """Codes and parameters (float64 values of bf16) of rows x [entries, hd], in pages of one head; random rows
    behind the last."""
    pages = -(-len(x) // PAGE)
    x = np.concatenate([x, np.random.default_rng(0).standard_normal((pages * PAGE - len(x), x.shape[1]))])
    codes, scale, base, _ = kv4.quantise(x.reshape(pages, 1, PAGE, -1))
    return kv4.pack(codes), np.stack([scale, base], axis=-1)


def _flat(codes, params):
    x, size = kv4.values(codes, params)
    return x.reshape(-1, x.shape[-1]), size.reshape(-1, x.shape[-1])


def _attend4(q, S, k, v):
    table = np.arange(len(k[0]), dtype=np.int32)[None]
    dev = [torch.as_tensor(c).cuda() for c in (k[0], v[0])] + [_bf16(c)[1] for c in (k[1], v[1])]
    out, status = binding.attention_kv4(q, _i([S]), _i(table), *dev)
    assert int(status[0]) == 0
    return out.double().cpu().numpy()[0]


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", ROWS)
@pytest.mark.parametrize("S", [70, 900])
@pytest.mark.parametrize("winner", ["constant", "zero", "small"])
@pytest.mark.parametrize("big", [18, 21, 40, 100])
def test_large_values_without_weight_next_to_one_that_has_it_all(K, G, hd, S, winner, big):
    """An entry whose V has a scale of 0 (one value throughout), or a small one, and all of the weight: products
    with it are lifted far up, where large values that have no weight, or are not seen, must stay finite."""
    rng = np.random.default_rng(hd + big)
    q = np.abs(rng.standard_normal((1, K, G, hd))) + 1.0
    k = rng.standard_normal((S + K, hd)) - 60.0
    k[5] = 60.0 + rng.random(hd)      # scores lie some 2000 above the others
    v = rng.standard_normal((S + K, hd))
    v[5] = {"constant": 3.0, "zero": 0.0}.get(winner, v[5] * 2.0 ** -40)
    if K * G <= 16:
        v[6:16] *= 2.0 ** big
    # (with more rows entry 5 has 2^-37 of what its page holds: test_values_of_scales_far_apart)
    v[16:] *= 2.0 ** big
    kk, vv = _store(k), _store(v)
    want, size = (x[5] for x in _flat(*vv))
    got = _attend4(_bf16(q)[1], S, kk, vv)
    floor = 2.0 ** -37 * np.abs(v[:16]).max() if K * G > 16 else 0.0
    lim = 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * size + floor
    assert np.isfinite(got).all() and (np.abs(got - want) <= lim).all()
