"""The linear layer with 4-bit weights at the ends of its arguments' ranges, against float64."""

import numpy as np
import pytest
import torch

from oracle import lowbit
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu


def _check(w, s, z, x, group):
    """fp32 sums: a group's MMA steps, one step for each group and a few products, each off by 2^-23 of what is summed
    in size (the MMA may cut where fp32 rounds); x below 2^-28 of its row's largest value is off by 2^-35 of that."""
    zeros = None if z is None else torch.as_tensor(z).cuda()
    y = binding.linear_w4(torch.as_tensor(w).cuda(), s.cuda(), x.cuda(), group, zeros=zeros)
    torch.cuda.synchronize()
    W, size = lowbit.unpack_w4(w, s.double().numpy(), z, group)
    X = x.double().numpy()
    steps = group // 16 + -(-x.shape[1] // group) + 16
    lim = steps * 2.0 ** -23 * (np.abs(X) @ size.T) + 2.0 ** -35 * np.abs(X).max(1, keepdims=True) * size.sum(1)
    err = np.abs(y.double().cpu().numpy() - X @ W.T)
    assert (err <= lim).all(), (err / np.maximum(lim, 1e-300)).max()
    return y


@pytest.mark.parametrize("kind", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,N,Kd", [(50, 3, 256), (33, 11, 1184)])
def test_zero_points_of_a_whole_byte(M, N, Kd, group, kind):
    rng = np.random.default_rng(M + group)
    ng = -(-Kd // group)
    w = rng.integers(0, 256, (M, Kd // 2), dtype=np.uint8)
    z = rng.integers(0, 256, (M, ng), dtype=np.uint8)
    z[0], z[1], w[2], z[2], w[3], z[3] = 255, 0, 0, 255, 255, 0
    s = torch.as_tensor(rng.uniform(0.2, 1.5, (M, ng)) * rng.choice([-1.0, 1.0], (M, ng))).to(kind)
    x = torch.as_tensor(rng.standard_normal((N, Kd))).to(torch.bfloat16)
    _check(w, s, z, x, group)


@pytest.mark.parametrize("group", [32, 128])
def test_every_code_with_every_zero_point(group):
    # one-hot rows read the weights back exactly
    M, Kd = 256, 256
    w = np.tile(np.arange(256, dtype=np.uint8)[:, None], (1, Kd // 2))
    z = np.stack([(np.arange(Kd // group) * 37 + m * 5) % 256 for m in range(M)]).astype(np.uint8)
    x = torch.zeros(16, Kd, dtype=torch.bfloat16)
    x[torch.arange(16), torch.arange(16) * 16 + 3] = 1.0
    y = binding.linear_w4(torch.as_tensor(w).cuda(), torch.ones(M, Kd // group).cuda(), x.cuda(), group,
                          zeros=torch.as_tensor(z).cuda())
    W, _ = lowbit.unpack_w4(w, np.ones(z.shape), z, group)
    np.testing.assert_array_equal(y.cpu().numpy(), W[:, torch.arange(16) * 16 + 3].T)


def test_scales_near_the_ends_of_their_range():
    # 2^96 is the largest that is promised; the smallest ones are not normal numbers
    rng = np.random.default_rng(4)
    M, N, Kd, group = 40, 5, 512, 64
    w = rng.integers(0, 256, (M, Kd // 2), dtype=np.uint8)
    s = torch.as_tensor(rng.uniform(1.0, 1.9, (M, Kd // group)).astype(np.float32))
    s[::2] *= 2.0 ** 95
    s[1::2] *= 2.0 ** -120
    x = torch.as_tensor(rng.standard_normal((N, Kd)) * 2.0 ** -6).to(torch.bfloat16)
    _check(w, s, None, x, group)


@pytest.mark.parametrize("N", [17, 24, 65, 352])
def test_the_rows_of_a_batch(N):
    rng = np.random.default_rng(N)
    M, Kd, group = 272, 1024, 32
    w = rng.integers(0, 256, (M, Kd // 2), dtype=np.uint8)
    z = rng.integers(0, 16, (M, Kd // group), dtype=np.uint8)
    s = torch.as_tensor(rng.uniform(0.2, 1.5, (M, Kd // group))).to(torch.bfloat16)
    x = torch.as_tensor(rng.standard_normal((N, Kd))).to(torch.bfloat16)
    _check(w, s, z, x, group)
