"""The linear layer with 4-bit weights against a float64 product of the unpacked weights."""

import numpy as np
import pytest
import torch

from oracle import lowbit
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu


def _make(M, N, Kd, group, zeros, kind, seed):
    rng = np.random.default_rng(seed)
    ng = -(-Kd // group)
    w = rng.integers(0, 256, (M, Kd // 2), dtype=np.uint8)
    s = torch.as_tensor(rng.uniform(0.2, 1.5, (M, ng)) * rng.choice([-1.0, 1.0], (M, ng))).to(kind)
    z = rng.integers(0, 16, (M, ng), dtype=np.uint8) if zeros else None
    x = torch.as_tensor(rng.standard_normal((N, Kd)) * np.exp2(rng.integers(-4, 5, (N, 1)))).to(torch.bfloat16)
    return w, s, z, x


def _check(w, s, z, x, group, **kw):
    y = binding.linear_w4(torch.as_tensor(w).cuda(), s.cuda(), kw.pop("xd", None) if "xd" in kw else x.cuda(), group,
                          zeros=None if z is None else torch.as_tensor(z).cuda(), **kw)
    torch.cuda.synchronize()
    W, size = lowbit.unpack_w4(w, s.double().numpy(), z, group)
    X = x.double().numpy()
    ref = X @ W.T
    # fp32 sums: at most a group of the MMA's steps, one step per group and a
    # few products, each off by 2^-23 of what is summed in size (the MMA may
    # cut where fp32 rounds); x below 2^-28 of its row's largest value is off
    # by 2^-35 of that value
    steps = group // 16 + -(-x.shape[1] // group) + 16
    lim = steps * 2.0 ** -23 * (np.abs(X) @ size.T) + 2.0 ** -35 * np.abs(X).max(1, keepdims=True) * size.sum(1)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert (err <= lim).all(), (err / np.maximum(lim, 1e-300)).max()
    return y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,Kd,zeros,kind", [
    (1, 1, 32, False, torch.float32), (16, 8, 256, True, torch.bfloat16), (17, 9, 288, True, torch.float32),
    (100, 3, 1056, False, torch.bfloat16), (2048, 1, 4096, False, torch.bfloat16), (640, 16, 2048, True, torch.float32),
    (333, 33, 544, True, torch.bfloat16), (64, 11, 8640, True, torch.bfloat16), (30000, 2, 96, False, torch.float32),
    (25000, 12, 512, True, torch.bfloat16), (2500, 8, 9216, False, torch.float32)])
def test_linear_w4_matches_float64(M, N, Kd, group, zeros, kind):
    _check(*_make(M, N, Kd, group, zeros, kind, M + N + Kd), group)


def test_linear_w4_every_code_in_every_place():
    # one-hot rows read the weights back exactly
    M, Kd = 48, 320
    w = np.stack([np.resize(np.arange(256, dtype=np.uint8), Kd // 2 + m)[m:] for m in range(M)])
    s = torch.ones(M, Kd // 32)
    z = np.tile(np.arange(Kd // 32, dtype=np.uint8), (M, 1))
    for k0 in range(0, Kd, 64):
        x = torch.zeros(64, Kd, dtype=torch.bfloat16)
        x[torch.arange(64), k0 + torch.arange(64)] = 1.0
        y = binding.linear_w4(torch.as_tensor(w).cuda(), s.cuda(), x.cuda(), 32, zeros=torch.as_tensor(z).cuda())
        W, _ = lowbit.unpack_w4(w, s.numpy(), z, 32)
        np.testing.assert_array_equal(y.cpu().numpy(), W[:, k0:k0 + 64].T)


def test_linear_w4_large_and_small_rows():
    # rows of very different size, one with a single value far above the others, one of zeros
    w, s, z, x = _make(200, 6, 512, 64, True, torch.float32, 5)
    x[0] *= 2.0 ** 100
    x[1] *= 2.0 ** -100
    x[2, 7] = 2.0 ** 20
    x[3] = 0
    x[4] = 2.0 ** -126
    _check(w, s, z, x, 64)


def test_linear_w4_of_strided_rows_and_into_a_wider_output():
    w, s, z, x = _make(130, 5, 256, 32, False, torch.bfloat16, 6)
    wide = torch.full((5, 800), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide[:, 8:264] = x.cuda()
    out = torch.full((5, 333), 7.0, device="cuda")
    _check(w, s, z, x, 32, xd=wide[:, 8:264], y=out[:, 3:133])
    assert (out[:, :3] == 7).all() and (out[:, 133:] == 7).all()


def test_linear_w4_nan_stays_in_its_row():
    w, s, z, x = _make(64, 9, 512, 128, True, torch.float32, 7)
    clean = _check(w, s, z, x, 128)
    x[4, 100] = float("nan")
    x[8, 3] = float("inf")
    y = binding.linear_w4(torch.as_tensor(w).cuda(), s.cuda(), x.cuda(), 128, zeros=torch.as_tensor(z).cuda())
    keep = [n for n in range(9) if n not in (4, 8)]
    assert torch.equal(y[keep], clean[keep]) and torch.isnan(y[4]).all() and not torch.isfinite(y[8]).any()


def test_linear_w4_repeats_bit_for_bit_and_under_capture():
    w, s, z, x = _make(3000, 11, 2048, 32, True, torch.bfloat16, 8)
    args = [torch.as_tensor(w).cuda(), s.cuda(), x.cuda(), 32, torch.as_tensor(z).cuda()]
    first = binding.linear_w4(*args)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        second = binding.linear_w4(*args)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, second)
