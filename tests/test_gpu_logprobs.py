"""Log probabilities, entropy and likeliest tokens on the GPU against float64."""

import numpy as np
import pytest
import torch

from oracle import kv4
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu


def _check(logits, tokens, top, temperature):
    """logits on the device, any stride. A weight is off by some 2^-21 (its exponent's argument and the function),
    the sums of V of them by 2^-20 of themselves at most, a result by a few roundings of its own."""
    x = logits.double().cpu().numpy()
    o = binding.token_logprobs(logits, torch.as_tensor(np.asarray(tokens), dtype=torch.int32, device="cuda"), top=top,
                               temperature=temperature)
    torch.cuda.synchronize()
    V = x.shape[-1]
    at, h, ids, best = kv4.token_logprobs(x.reshape(-1, V), np.asarray(tokens).reshape(-1), top, temperature)
    for name, got, ref in (("logprobs", o["logprobs"], at), ("entropy", o["entropy"], h), ("top", o["top_logprobs"], best)):
        got = got.double().cpu().numpy().reshape(ref.shape)
        with np.errstate(over="ignore"):
            ref = np.where(np.isinf(ref.astype(np.float32)), np.copysign(np.inf, ref), ref)   # -FLT_MAX / 0.5 is no fp32 number
        np.testing.assert_array_equal(np.isnan(got), np.isnan(ref), err_msg=name)
        np.testing.assert_array_equal(np.isinf(got), np.isinf(ref), err_msg=name)
        fine = np.isfinite(ref)
        lim = 2.0 ** -20 + 2.0 ** -22 * np.abs(ref) + (2.0 ** -20 * np.abs(ref) if name == "entropy" else 0.0)
        assert (np.abs(got[fine] - ref[fine]) <= lim[fine]).all(), (name, (np.abs(got[fine] - ref[fine]) / lim[fine]).max())
    np.testing.assert_array_equal(o["top_tokens"].cpu().numpy().reshape(ids.shape), ids)


def _logits(rng, R, V, dtype, spread=3.0):
    return torch.as_tensor(rng.standard_normal((R, V)) * spread).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("R,V,top,temperature", [
    (1, 1, 1, 1.0), (3, 2, 2, 0.5), (2, 7, 5, 1.0), (5, 33, 32, 0.3), (4, 1000, 16, 0.7), (2, 4096, 17, 1.0),
    (1, 50257, 5, 1.0), (7, 32001, 20, 0.3), (1, 151936, 32, 1.0), (3, 201088, 1, 2.0), (400, 4099, 3, 1.0),
    (2, 151936, 0, 1.0), (40, 65536, 5, 0.7)])
def test_rows(R, V, top, temperature, dtype):
    rng = np.random.default_rng(V + R)
    _check(_logits(rng, R, V, dtype), rng.integers(0, V, R), top, temperature)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,skip", [(1, 0), (3, 1), (8, 5), (64, 7)])
def test_strides_and_starts_off_the_vector(pad, skip, dtype):
    rng = np.random.default_rng(pad)
    wide = _logits(rng, 5, 9001 + pad + skip, dtype)
    wide[:, :skip] = 1e6
    wide[:, 9001 + skip:] = 1e6
    _check(wide[:, skip:9001 + skip], rng.integers(0, 9001, 5), 7, 1.0)
    three = _logits(rng, 6, 500 + pad, dtype).view(2, 3, 500 + pad)[:, :, :500]
    _check(three, rng.integers(0, 500, (2, 3)), 3, 1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 5000, 70000])
@pytest.mark.parametrize("top", [1, 5, 16, 20, 32])
def test_ties_and_orders(V, top, dtype):
    rng = np.random.default_rng(V + top)
    x = torch.stack([torch.zeros(V), torch.arange(V) * (8.0 / V), -torch.arange(V) * (8.0 / V),
                     torch.as_tensor(rng.integers(0, 3, V)).float(), torch.as_tensor(rng.integers(0, 200, V)).float(),
                     torch.where(torch.arange(V) % 512 == 3, 4.0, 1.0) + torch.arange(V) * 1e-4,
                     torch.where(torch.arange(V) < V - 3, -1.0, 2.0), -torch.zeros(V)])
    x[7, ::2] = 0.0    # 0 and -0 are the same value
    _check(x.to(dtype).cuda(), rng.integers(0, V, len(x)), top, 1.0)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [40, 5000, 70000])
@pytest.mark.parametrize("top", [0, 1, 5, 20, 32])
def test_masks_and_values_that_are_not_finite(V, top, dtype):
    rng = np.random.default_rng(V)
    low = torch.finfo(dtype).min
    x = _logits(rng, 12, V, dtype)
    inf = float("inf")
    keep = torch.as_tensor(rng.permutation(V)[:3])
    for r, mask in ((0, -inf), (1, low)):           # three tokens are left
        had = x[r, keep].clone()
        x[r] = mask
        x[r, keep] = had
    x[2] = -inf                                     # none is
    x[3] = low                                      # all are alike
    x[4, 5] = inf
    x[5, 6] = float("nan")
    x[6] = -inf
    x[6, V - 1] = 2.0                               # one is left
    x[7] = 1e4 * x[7].clamp(-3, 3)                  # sure of one
    x[8] = float("nan")
    x[9, V // 2:] = low
    x[10, :V // 2] = -inf
    x[11] = 2.0 ** 100
    tokens = rng.integers(0, V, 12)
    tokens[0], tokens[6] = int(keep[0]), V - 1
    _check(x, tokens, top, 1.0)
    tokens[:4] = [-1, V, 2 ** 31 - 1, -2 ** 31]
    _check(x, tokens, top, 0.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [4096, 5003, 33001])
@pytest.mark.parametrize("top", [0, 1, 8, 9, 20, 32])
def test_rows_for_every_small_block(V, top, dtype):
    # more rows than large blocks are used for; rows of every kind among them
    rng = np.random.default_rng(V + top)
    R = 4 * torch.cuda.get_device_properties(0).multi_processor_count + 13
    x = _logits(rng, R, V + 3, dtype)[:, :V]
    x[0], x[1], x[2] = 0.0, -float("inf"), torch.finfo(dtype).min
    x[3, 7:] = -float("inf")
    x[4, 5], x[5, 6] = float("inf"), float("nan")
    x[6] = (torch.arange(V) % 256 == 3).float() * 4        # many of the largest with one thread
    x[7] = -torch.arange(V) * 2.0 ** -10
    x[8] = torch.as_tensor(rng.integers(0, 3, V)).float()
    x[9, :V - 20] = -1e4
    x[10] = torch.where(torch.arange(V) % 512 < 3, 9.0, 1.0) + torch.arange(V) % 7 * 0.125
    _check(x, rng.integers(0, V, R), top, 0.7)


@pytest.mark.parametrize("R", [1, 700])
def test_long_rows(R):
    # cells of several batches
    rng = np.random.default_rng(R)
    x = torch.randn(R, 300007, device="cuda", generator=torch.Generator("cuda").manual_seed(R)).to(torch.bfloat16)
    at = rng.choice(R, min(R, 40), replace=False)
    tokens = torch.as_tensor(rng.integers(0, 300007, R), dtype=torch.int32, device="cuda")
    o = binding.token_logprobs(x, tokens, top=20)
    some = torch.as_tensor(at).cuda()
    lp, h, ids, best = kv4.token_logprobs(x[some].double().cpu().numpy(), tokens[some].cpu().numpy(), 20, 1.0)
    np.testing.assert_array_equal(o["top_tokens"][some].cpu().numpy(), ids)
    for got, ref in ((o["logprobs"], lp), (o["entropy"], h), (o["top_logprobs"], best)):
        np.testing.assert_allclose(got[some].double().cpu().numpy(), ref, rtol=2.0 ** -19, atol=2.0 ** -19)


def test_results_do_not_change_from_call_to_call():
    rng = np.random.default_rng(3)
    for R in (1, 9, 400, 700):
        x = _logits(rng, R, 30000, torch.bfloat16)
        t = torch.as_tensor(rng.integers(0, 30000, R), dtype=torch.int32, device="cuda")
        first = binding.token_logprobs(x, t, top=20)
        for _ in range(5):
            again = binding.token_logprobs(x, t, top=20)
            assert all(torch.equal(first[k], again[k]) for k in first)


def test_what_the_sampling_operators_draw_by():
    """The probabilities are those that drafts are sampled by: the frequency of each token over many uniforms."""
    rng = np.random.default_rng(0)
    V, T = 500, 0.7
    x = _logits(rng, 1, V, torch.float32, 1.5)
    o = binding.token_logprobs(x.expand(V, V), torch.arange(V, dtype=torch.int32, device="cuda"), temperature=T)
    p = torch.softmax(x[0].double() / T, 0)
    assert torch.allclose(o["logprobs"].double().exp(), p, rtol=2.0 ** -18)
