"""The rotation of pe_kv4_append to the last bits of its angles, and keys whose turned values all but agree."""

from decimal import Decimal, getcontext

import numpy as np
import pytest
import torch

from oracle import kv4
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu

TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459")


def _turn(theta, hd, position):
    """position * theta^(-2i/hd) of each pair in radians, its whole turns taken off in 60 digits."""
    getcontext().prec = 60
    root = Decimal(theta) ** (Decimal(-2) / hd)
    turns = [position * root ** i / TWO_PI for i in range(hd // 2)]
    return np.array([float((t - int(t)) * TWO_PI) for t in turns])


def _pairs(angle):
    """bf16 a, b below 1 for each angle with the smallest |a cos - b sin|: what is left of it shows the angle's error."""
    mantissa = np.arange(128, 256) / 256.0
    out = np.zeros((len(angle), 2))
    for i, t in enumerate(angle):
        c, s = np.cos(t), np.sin(t)
        if abs(c) <= abs(s):
            a, b = mantissa, kv4.bf16(mantissa * c / s)
        else:
            a, b = kv4.bf16(mantissa * s / c), mantissa
        at = np.abs(a * c - b * s).argmin()
        out[i] = a[at], b[at]
    return out


def _append(q, k, theta, position):
    hd = k.shape[-1]
    cache = [torch.zeros(1, k.shape[2], 16, hd // 2, dtype=torch.uint8, device="cuda") for _ in range(2)]
    params = [torch.zeros(1, k.shape[2], 16, 2, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
    dev = lambda x: torch.as_tensor(x, dtype=torch.float32).to(torch.bfloat16).cuda()
    out, status = binding.kv4_append(dev(k), dev(np.zeros_like(k)), i(0), i(0).view(1, 1), *cache, *params, theta=theta,
                                     positions=i(position), q=None if q is None else dev(q))
    assert int(status[0]) == 0
    return out, cache[0].cpu().numpy(), params[0].double().cpu().numpy()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("theta", [1e4, 5e5, 1e6, 150000.0])
@pytest.mark.parametrize("position", [1, 131071, 10 ** 8 + 7, 2 ** 31 - 2, 2 ** 31 - 1025])
def test_angles_of_far_positions(theta, hd, position):
    angle = _turn(theta, hd, position)
    ab = _pairs(angle)
    q = np.concatenate([ab[:, 0], ab[:, 1]])[None, None, None]
    out, _, _ = _append(q, np.zeros((1, 1, 1, hd)), theta, position)
    got = out.double().cpu().numpy()[0, 0, 0]
    c, s = np.cos(angle), np.sin(angle)
    want = np.concatenate([ab[:, 0] * c - ab[:, 1] * s, ab[:, 1] * c + ab[:, 0] * s])
    # Sine and cosine: one step of the function and half a step of the first-order term behind its 24 bits, 2^-24 of
    # values below 1 each. Then a product's rounding, half of 2^-24, and the output's. The angle itself: 2^-32 of a turn.
    size = np.tile(np.abs(ab).sum(1), 2)
    lim = size * (1.5 * 2.0 ** -24 + 2 * np.pi * 2.0 ** -32) + 2.0 ** -25 + 2.0 ** -8 * np.abs(want)
    assert (np.abs(got - want) <= lim).all(), ((np.abs(got - want) / lim).max(), (np.abs(got - want) / lim).argmax())


def _agreeing(theta, hd):
    """A position and bf16 a, b whose turned values, the same for every pair at a base of 1, lie between two bf16
    values, nearer to the upper one."""
    for position in range(1, 4000):
        c, s = np.cos(float(position)), np.sin(float(position))
        a = np.arange(128, 256)[:, None] / 128.0
        b = kv4.bf16(a * (c - s) / (c + s))              # both would be a / (cos + sin)
        x, y = a * c - b * s, b * c + a * s
        lo, hi = np.minimum(x, y), np.maximum(x, y)
        at = np.argwhere((kv4.bf16(lo) > hi + 1e-5 * np.abs(hi)) & (lo > 0.1))
        if len(at):
            i = at[0][0]
            return position, float(a[i, 0]), float(b[i, 0]), float(kv4.bf16(lo[i])[0])
    raise AssertionError("none found")


@pytest.mark.parametrize("hd", [64, 128])
def test_a_scale_is_never_negative(hd):
    """All values of a key below the bf16 value that their smallest rounds to: the scale is 0, not below it."""
    position, a, b, base = _agreeing(1.0, hd)
    k = np.concatenate([np.full(hd // 2, a), np.full(hd // 2, b)])[None, None, None]
    _, codes, params = _append(None, k, 1.0, position)
    np.testing.assert_array_equal(params[0, 0, 0], [0.0, base])
    assert not codes[0, 0, 0].any()


@pytest.mark.parametrize("hd", [64, 128])
def test_the_largest_magnitudes(hd):
    """What lies farther apart than fp32 holds stands as NaN, one value throughout as it is."""
    k = np.full((1, 1, 4, hd), 2.0 ** 127)
    k[0, 0, 1] *= -1
    k[0, 0, 2, ::2] *= -1                              # 2^128 apart
    k[0, 0, 3, ::2] *= -0.5
    _, codes, params = _append(None, k, 0.0, 0)
    got = params[0, :, 0]
    np.testing.assert_array_equal(got[:2], [[0.0, 2.0 ** 127], [0.0, -2.0 ** 127]])
    assert np.isnan(got[2]).all()
    assert got[3, 1] == -2.0 ** 126 and got[3, 0] == kv4.bf16(1.5 * 2.0 ** 127 / 15)
    assert not codes[0, :2, 0].any() and (kv4.unpack(codes[0, 3, 0]) == np.where(np.arange(hd) % 2, 15, 0)).all()
