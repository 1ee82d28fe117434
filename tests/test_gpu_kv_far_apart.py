"""Attention over the 4-bit and the 8-bit cache where one entry has all of a row's weight: scores that lie far apart,
in requests long enough for pages and units that every row sees whole, and values of V that do."""

import numpy as np
import pytest
import torch

from oracle import e4m3_decode, kv4, lowbit
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


def _clear(k, q, S, reach, part):
    """Of each row of q [K, G, hd] the entry with the largest score, and whether it stands `part` of `reach`, the
    largest sum of |q| |k|, above the next: more than scores, queries and keys are rounded by, and by so much that the
    next has no weight."""
    best, clear = np.zeros(q.shape[:2], dtype=int), np.zeros(q.shape[:2], dtype=bool)
    for j in range(len(q)):
        x = k[:S + j + 1] @ q[j].T
        best[j] = x.argmax(0)
        top = np.sort(x, axis=0)[-2:]
        clear[j] = top[1] - top[0] > part * reach[j]
    assert clear.mean() > 0.3
    return best, clear


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", ROWS)
@pytest.mark.parametrize("S", [130, 900, 6000])
@pytest.mark.parametrize("up", [15, 24, 26, 28, 31, 40, 60])
@pytest.mark.parametrize("spread", [0, 24])
def test_kv4_scores_far_apart(K, G, hd, S, up, spread):
    rng = np.random.default_rng(hd + up + S)
    kk = _store(rng.standard_normal((S + K, hd)))
    far = np.exp2(rng.integers(-spread, spread + 1, (-(-(S + K) // PAGE), 1, 1))).repeat(PAGE, 1).reshape(-1, 1)[:S + K]
    vv = _store(rng.standard_normal((S + K, hd)) * far)
    qx, qt = _bf16(rng.standard_normal((1, K, G, hd)) * 2.0 ** up)
    (k, ka), (v, va) = _flat(*kk), _flat(*vv)
    best, clear = _clear(k, qx[0], S, (np.abs(qx[0]) @ ka.T).max(-1), 2.0 ** (-9 if K * G > 16 else -11))
    got = _attend4(qt, S, kk, vv)
    want = v[best]
    lim = 2.0 ** -8 * np.abs(want) + 2.0 ** -9 * va[best]
    if K * G > 16:
        lim = lim + 2.0 ** -36 * va.reshape(-1, PAGE, hd).max((1, 2))[best // PAGE][..., None]
    assert np.isfinite(got).all()
    assert (np.abs(got - want)[clear] <= lim[clear]).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", ROWS)
@pytest.mark.parametrize("S", [130, 900, 6000])
@pytest.mark.parametrize("up", [15, 24, 26, 28, 31, 40, 60])
@pytest.mark.parametrize("spread", [0, 24])
def test_kv8_scores_far_apart(K, G, hd, S, up, spread):
    rng = np.random.default_rng(hd + up + S)
    pages = -(-(S + K) // PAGE)
    codes = [lowbit.e4m3_encode(rng.standard_normal((pages, 1, PAGE, hd))) for _ in range(2)]
    scale = np.ones((pages, 1), dtype=np.float32)
    v_scale = np.exp2(rng.integers(-spread, spread + 1, (pages, 1))).astype(np.float32)
    qx, qt = _bf16(rng.standard_normal((1, K, G, hd)) * 2.0 ** up)
    k = e4m3_decode(codes[0])[:, 0].reshape(-1, hd)
    v = (e4m3_decode(codes[1]) * v_scale[..., None, None])[:, 0].reshape(-1, hd)
    best, clear = _clear(k, qx[0], S, (np.abs(qx[0]) @ np.abs(k).T).max(-1), 2.0 ** -11)
    dev = [torch.as_tensor(c).cuda() for c in (*codes, scale, v_scale)]
    out, status = binding.attention_kv8(qt, _i([S]), _i(np.arange(pages)[None]), *dev)
    assert int(status[0]) == 0
    got, want = out.double().cpu().numpy()[0], v[best]
    assert np.isfinite(got).all()
    # the output's rounding, and the weight's
    assert (np.abs(got - want)[clear] <= ((2.0 ** -8 + 2.0 ** -10) * np.abs(want))[clear]).all()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", ROWS)
@pytest.mark.parametrize("S", [60, 600, 6000])
@pytest.mark.parametrize("power", [-100, -60, 60, 104])
def test_kv4_values_times_a_power_of_two(K, G, hd, S, power):
    """Outputs follow V's power of two, to the ends of the range that the header gives (6000 values below 2^106)."""
    rng = np.random.default_rng(hd + S)
    kk, vv = _store(rng.standard_normal((S + K, hd))), _store(rng.standard_normal((S + K, hd)))
    qt = _bf16(2.0 * rng.standard_normal((1, K, G, hd)))[1]
    plain = _attend4(qt, S, kk, vv)
    moved = _attend4(qt, S, kk, (vv[0], np.ldexp(vv[1], power)))
    # a step of the output apart at most, where reference points fall on either side of a rounding; fp16 products
    assert (np.abs(np.ldexp(moved, -power) - plain) <= 2.0 ** -7 * np.abs(plain) + 2.0 ** -11).all()
