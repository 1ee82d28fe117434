"""Attention over the 8-bit cache where scores are so large that their fp32 steps exceed the kernels' own shifts."""

import numpy as np
import pytest
import torch

from oracle import e4m3_decode, lowbit
from speculative_drafting_pe_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("K,G", [(1, 8), (2, 8), (11, 8)])
def test_the_largest_of_scores_that_lie_far_apart_has_all_the_weight(K, G, hd):
    rng = np.random.default_rng(hd + K)
    S = 50
    table = rng.permutation(8)[:5].reshape(1, 5).astype(np.int32)
    codes = [lowbit.e4m3_encode(rng.standard_normal((8, 1, 16, hd))) for _ in range(2)]
    scale = np.ones((8, 1), dtype=np.float32)
    q = torch.as_tensor(rng.standard_normal((1, K, G, hd)) * 2.0 ** 40).to(torch.bfloat16)
    dev = [torch.as_tensor(c).cuda() for c in (*codes, scale, scale)]
    out, _ = binding.attention_kv8(q.cuda(), torch.tensor([S], dtype=torch.int32, device="cuda"),
                                   torch.as_tensor(table).cuda(), *dev)
    k, v = (e4m3_decode(c[table[0]])[:, 0].reshape(-1, hd) for c in codes)
    for j in range(K):
        x = k[:S + j + 1] @ q[0, j].double().numpy().T
        want = v[x.argmax(0)]
        assert (np.abs(out[0, j].double().cpu().numpy() - want) <= 2.0 ** -8 * np.abs(want)).all()
