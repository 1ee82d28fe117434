"""What the 4-bit cache's operators and the log probabilities refuse before anything is launched (no GPU)."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import kv4
from speculative_drafting_pe_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


P = ctypes.c_void_p(64)      # aligned addresses that nothing reads
P2, P3 = ctypes.c_void_p(128), ctypes.c_void_p(192)
ODD = ctypes.c_void_p(68)
INF, NAN = float("inf"), float("nan")


def test_append_refusals(lib):
    def call(B=1, n=1, nq=4, nkv=2, hd=64, q=P, ldq=256, k=P, ldk=128, v=P, ldv=128, theta=1e4, pos=None, s=P, rows=None,
             t=P, mp=1, pages=1, kc=P, vc=P, kp=P, vp=P, qo=P2, ldo=256, st=P3):
        return lib.pe_kv4_append(B, n, nq, nkv, hd, q, ldq, k, ldk, v, ldv, theta, pos, s, rows, t, mp, pages, kc, vc, kp,
                                 vp, qo, ldo, st, None)
    for bad in (dict(B=0), dict(n=0), dict(nkv=0), dict(nq=-1), dict(mp=0), dict(pages=0), dict(ldk=127), dict(ldv=130),
                dict(ldq=252), dict(ldq=258), dict(ldo=255), dict(q=None), dict(qo=None), dict(k=None), dict(v=None),
                dict(s=None), dict(t=None), dict(kc=None), dict(vp=None), dict(st=None), dict(k=ODD), dict(qo=ODD),
                dict(kc=ODD), dict(vp=ODD), dict(mp=1 << 28), dict(n=1 << 28), dict(nq=1 << 21, ldq=1 << 30, ldo=1 << 30),
                dict(theta=-1.0), dict(theta=0.5), dict(theta=INF), dict(theta=NAN),
                dict(qo=P, ldo=512), dict(st=P), dict(rows=P2, st=P2), dict(pos=P2, st=P2)):
        assert call(**bad) == -1, bad
    assert call(hd=96) == -2 and call(hd=32) == -2


def test_attention_refusals(lib):
    def call(B=1, K=1, nq=4, nkv=2, hd=64, q=P, ldq=256, s=P, t=P, mp=1, pages=1, kc=P, vc=P, kp=P, vp=P, scale=1.0, o=P2,
             ldo=256, ws=P, floats=1 << 30, st=P3, rows=None):
        return lib.pe_attention_kv4(B, K, nq, nkv, hd, q, ldq, s, rows, t, mp, pages, kc, vc, kp, vp, scale, o, ldo, ws,
                                    floats, st, None)
    for bad in (dict(B=0), dict(K=0), dict(mp=0), dict(pages=0), dict(ldq=252), dict(ldq=255), dict(ldo=248),
                dict(q=None), dict(o=None), dict(ws=None), dict(st=None), dict(kp=None), dict(q=ODD), dict(o=ODD),
                dict(ws=ODD), dict(vc=ODD), dict(vp=ODD), dict(pages=1 << 26), dict(mp=1 << 28), dict(o=P), dict(st=P),
                dict(rows=P2, st=P2)):
        assert call(**bad) == -1, bad
    for bad in (dict(nq=5), dict(nkv=0), dict(hd=32), dict(K=65), dict(nq=260, ldq=260 * 64, ldo=260 * 64)):
        assert call(**bad) == -2, bad
    assert lib.pe_attention_kv4_scratch(1, 1, 4, 2, 64, 1, None) == -1


def test_logprob_refusals(lib):
    def call(R=1, V=8, dtype=1, x=P, ld=8, t=P, temp=1.0, lp=P, h=P, top=2, ids=P, best=P):
        return lib.pe_token_logprobs(R, V, dtype, x, ld, t, temp, lp, h, top, ids, best, None)
    v = ctypes.c_void_p
    for bad in (dict(R=0), dict(V=0), dict(dtype=7), dict(top=-1), dict(top=33, V=100, ld=100), dict(top=9), dict(ld=7),
                dict(ld=-8), dict(temp=0.0), dict(temp=-1.0), dict(temp=NAN), dict(temp=INF), dict(temp=2.0 ** -64),
                dict(temp=2.0 ** 65), dict(x=None), dict(t=None), dict(lp=None), dict(ids=None), dict(best=None),
                dict(x=v(65)), dict(t=v(66)), dict(h=v(66)), dict(R=(1 << 30) + 1), dict(V=(1 << 30) + 1, ld=1 << 31)):
        assert call(**bad) == -1, bad


def test_binding_refuses_before_the_library(lib):
    z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d)
    b = torch.bfloat16
    cache = [z(3, 2, 16, 32, d=torch.uint8), z(3, 2, 16, 32, d=torch.uint8), z(3, 2, 16, 2, d=b), z(3, 2, 16, 2, d=b)]
    kv = z(1, 2, 2, 64, d=b)
    for args, more in (
            ((kv, z(1, 3, 2, 64, d=b), z(1), z(1, 1), *cache), {}),                      # values of another shape
            ((kv, kv, z(1), z(1, 1), *cache), dict(q_out=z(1, 2, 4, 64, d=b))),          # q_out without q
            ((kv, kv, z(1), z(1, 1), *cache), dict(q=z(1, 3, 4, 64, d=b))),              # other rows of q
            ((kv, kv, z(1), z(1, 1), *cache), dict(positions=z(2))),
            ((kv, kv, z(1), z(1, 1), cache[0], cache[1], cache[2].float(), cache[3]), {}),
            ((z(1, 2, 2, 128, d=b), z(1, 2, 2, 128, d=b), z(1), z(1, 1), *cache), {}),   # heads of another width
            ((kv, kv, z(1), z(1, 1), *cache), {})):                                      # CPU tensors
        with pytest.raises(ValueError):
            binding.kv4_append(*args, **more)
    for args in ((z(1, 1, 4, 128, d=b), z(1), z(1, 1), *cache), (z(1, 1, 4, 64, d=torch.float16), z(1), z(1, 1), *cache),
                 (z(1, 1, 4, 64, d=b), z(2), z(1, 1), *cache), (z(1, 1, 4, 64, d=b), z(1), z(1, 1), *cache)):
        with pytest.raises(ValueError):
            binding.attention_kv4(*args)
    x = z(2, 9, d=torch.float32)
    for args, more in (((x.half(), z(2)), {}), ((x[0], z(1)), {}), ((x, z(3)), {}), ((x, z(2, d=torch.int64)), {}),
                       ((x, z(2)), dict(top=33)), ((x, z(2)), dict(top=-1)), ((x, z(2)), {}),
                       ((z(3, 4, 9, d=b)[:, ::3], z(3, 2)), {})):
        with pytest.raises(ValueError):
            binding.token_logprobs(*args, **more)


def test_stalls_of_no_barrier(lib):
    for barrier in (0, 4, -1):
        assert lib.pe_test_stall_attention_kv4(barrier) == -1


def test_restatement_of_the_codes():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((50, 64)) * np.exp2(rng.integers(-30, 30, (50, 1)))
    codes, scale, base, _ = kv4.quantise(x)
    params = np.stack([scale, base], axis=-1)
    back, _ = kv4.values(kv4.pack(codes), params)
    # half a step, and what base and scale were rounded by over 15 steps
    assert (np.abs(back - x) <= 0.5 * scale[:, None] + 2.0 ** -8 * np.abs(base[:, None]) + 15 * 2.0 ** -8 * scale[:, None]).all()
    np.testing.assert_array_equal(kv4.unpack(kv4.pack(codes)), codes)
    assert codes.min() >= 0 and codes.max() <= 15
    flat = kv4.quantise(np.full((1, 8), 3.0))
    assert (flat[0] == 0).all() and flat[1][0] == 0 and flat[2][0] == 3.0


def test_restatement_of_the_rotation():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 128))
    np.testing.assert_array_equal(kv4.rotate(x, 0, 1e4), x)
    np.testing.assert_allclose(np.linalg.norm(kv4.rotate(x, 12345, 1e4)), np.linalg.norm(x))
    # a product of two rows depends on the difference of their positions
    y = rng.standard_normal((3, 128))
    a = (kv4.rotate(x, 107, 1e4) * kv4.rotate(y, 100, 1e4)).sum(-1)
    np.testing.assert_allclose(a, (kv4.rotate(x, 7, 1e4) * y).sum(-1), rtol=1e-9)
