"""What the low-bit operators refuse before anything is launched (no GPU), and their restatement's own pins."""

import ctypes

import numpy as np
import pytest
import torch

from oracle import e4m3_decode, lowbit
from speculative_drafting_pe_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


P = ctypes.c_void_p(64)      # an aligned address that nothing reads
ODD = ctypes.c_void_p(68)


def test_linear_w4_refusals(lib):
    def call(M=16, N=1, Kd=64, group=32, w=P, kind=0, s=P, z=None, x=P, ldx=64, y=P, ldy=16):
        return lib.pe_linear_w4(M, N, Kd, group, w, kind, s, z, x, ldx, y, ldy, None)
    for bad in (dict(M=0), dict(N=0), dict(Kd=0), dict(Kd=48), dict(w=None), dict(s=None), dict(x=None), dict(y=None),
                dict(kind=2), dict(ldx=60), dict(ldx=68), dict(ldy=15), dict(w=ODD), dict(x=ODD)):
        assert call(**bad) == -1, bad
    assert call(group=16) == -2 and call(group=0) == -2


def test_linear_w4_refuses_scales_and_outputs_off_their_type(lib):
    v = ctypes.c_void_p
    for kind, s, y in ((0, 65, 64), (0, 66, 66), (1, 66, 64), (1, 68, 65)):
        assert lib.pe_linear_w4(16, 1, 64, 32, P, kind, v(s), None, P, 64, v(y), 16, None) == -1, (kind, s, y)


def test_assign_and_release_refusals(lib):
    def assign(B=1, s=P, n=P, c=P, co=ODD, t=P, mp=1, pages=1, f=P, cap=1, fc=P, fo=ODD, n_max=1, sl=P, st=P):
        return lib.pe_assign_pages(B, s, n, c, co, t, mp, pages, f, cap, fc, fo, n_max, sl, st, None)
    for bad in (dict(B=0), dict(mp=0), dict(pages=0), dict(cap=0), dict(n_max=0), dict(s=None), dict(t=None),
                dict(st=None), dict(co=P), dict(fo=P), dict(pages=1 << 28), dict(mp=1 << 28)):
        assert assign(**bad) == -1, bad

    def release(B=1, k=P, c=P, co=P, t=P, mp=1, pages=1, f=P, cap=1, fc=P, fo=P, st=P):
        return lib.pe_release_pages(B, k, c, co, t, mp, pages, f, cap, fc, fo, st, None)
    for bad in (dict(B=0), dict(mp=0), dict(cap=0), dict(k=None), dict(f=None), dict(st=None)):
        assert release(**bad) == -1, bad


def test_append_refusals(lib):
    def call(B=1, n=1, nkv=2, hd=64, k=P, ldk=128, v=P, ldv=128, s=P, t=P, mp=1, pages=1, kc=P, vc=P, ks=P, vs=P, st=P):
        return lib.pe_kv8_append(B, n, nkv, hd, k, ldk, v, ldv, s, None, t, mp, pages, kc, vc, ks, vs, st, None)
    for bad in (dict(B=0), dict(n=0), dict(nkv=0), dict(mp=0), dict(pages=0), dict(ldk=127), dict(ldv=130), dict(k=None),
                dict(t=None), dict(vs=None), dict(k=ODD), dict(kc=ODD), dict(mp=1 << 28)):
        assert call(**bad) == -1, bad
    assert call(hd=96) == -2


def test_attention_refusals(lib):
    def call(B=1, K=1, nq=4, nkv=2, hd=64, q=P, ldq=256, s=P, t=P, mp=1, pages=1, kc=P, vc=P, ks=P, vs=P, o=P, ldo=256,
             ws=P, floats=1 << 30, st=P):
        return lib.pe_attention_kv8(B, K, nq, nkv, hd, q, ldq, s, None, t, mp, pages, kc, vc, ks, vs, 1.0, o, ldo, ws,
                                    floats, st, None)
    for bad in (dict(B=0), dict(K=0), dict(mp=0), dict(pages=0), dict(ldq=252), dict(ldq=255), dict(ldo=248),
                dict(q=None), dict(o=None), dict(ws=None), dict(st=None), dict(q=ODD), dict(o=ODD), dict(ws=ODD),
                dict(vc=ODD), dict(pages=1 << 26), dict(mp=1 << 28)):
        assert call(**bad) == -1, bad
    for bad in (dict(nq=5), dict(nkv=0), dict(hd=32), dict(K=65), dict(nq=260, ldq=260 * 64, ldo=260 * 64)):
        assert call(**bad) == -2, bad


def test_binding_refuses_before_the_library(lib):
    z = lambda *s, d=torch.int32: torch.zeros(*s, dtype=d)
    with pytest.raises(ValueError):      # CPU tensors
        binding.linear_w4(z(16, 32, d=torch.uint8), z(16, 2, d=torch.float32), z(1, 64, d=torch.bfloat16), 32)
    with pytest.raises(ValueError):      # scales of another group
        binding.linear_w4(z(16, 32, d=torch.uint8), z(16, 1, d=torch.float32), z(1, 64, d=torch.bfloat16), 32)
    with pytest.raises(ValueError):      # lengths of another type
        binding.assign_pages(z(2, d=torch.int64), z(2), z(2), z(2, 3), z(4), z(1), 4, 2)
    cache = [z(3, 2, 16, 64, d=torch.uint8), z(3, 2, 16, 64, d=torch.uint8), z(3, 2, d=torch.float32),
             z(3, 2, d=torch.float32)]
    with pytest.raises(ValueError):      # values of another shape than the keys
        binding.kv8_append(z(1, 2, 2, 64, d=torch.bfloat16), z(1, 3, 2, 64, d=torch.bfloat16), z(1), z(1, 1), *cache)
    with pytest.raises(ValueError):      # heads of another width than the cache's
        binding.attention_kv8(z(1, 1, 4, 128, d=torch.bfloat16), z(1), z(1, 1), *cache)
    with pytest.raises(ValueError):      # rows that are not evenly spaced
        binding._row_stride(z(4, 6, 2, 64)[::2, ::2][:, :2], "k")


def test_row_strides():
    t = torch.zeros(4, 6, 2, 64)
    assert binding._row_stride(t, "t") == 128
    assert binding._row_stride(torch.zeros(4, 6, 512)[..., 128:256].unflatten(-1, (2, 64)), "t") == 512
    assert binding._row_stride(t[:1, :1], "t") == 128 and binding._row_stride(t[:, :1], "t") == 6 * 128
    with pytest.raises(ValueError):
        binding._row_stride(t.transpose(2, 3), "t")


def test_restatement_of_the_codes():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    np.testing.assert_array_equal(lowbit.e4m3_encode(e4m3_decode(codes)), codes)
    x = np.random.default_rng(0).standard_normal(4000) * 100
    t = torch.as_tensor(x, dtype=torch.float32).clamp(-448, 448)
    np.testing.assert_array_equal(lowbit.e4m3_encode(t.double().numpy()), t.to(torch.float8_e4m3fn).view(torch.uint8))
    for top, s in ((448.0, 1.0), (449.0, 2.0), (224.0, 0.5), (0.0, 2.0 ** -126), (2.0 ** -130, 2.0 ** -126)):
        assert lowbit.kv8_scale(np.array([0.0, -top, np.inf, np.nan])) == s


def test_restatement_of_pages_keeps_every_page_once():
    rng = np.random.default_rng(1)
    free, table, counts, F = np.arange(64, dtype=np.int32), np.full((6, 20), -1, np.int32), np.zeros(6, np.int32), 64
    S = np.zeros(6, dtype=np.int64)
    for _ in range(30):
        n = rng.integers(0, 9, 6)
        _, counts, table, F, st = lowbit.assign_pages(S, n, counts, table, free, F, 64, 8)
        S = np.where(st == 0, S + n, S)
        S = np.where(rng.random(6) < 0.2, 0, S)
        counts, table, free, F, st = lowbit.release_pages(S, counts, table, free, F, 64)
        held = [p for b in range(6) for p in table[b, :counts[b]]]
        assert sorted(held + free[:F].tolist()) == list(range(64)) and (counts == -(-S // 16)).all()


def test_stalls_of_no_barrier(lib):
    for barrier in (0, 4, -1):
        assert lib.pe_test_stall_attention_kv8(barrier) == -1
