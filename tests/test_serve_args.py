"""Refusals of the few-token operators, before any CUDA call (no GPU).

As in tests/test_abi.py, every call fails a check or has nothing to do: none
may pass its checks with the placeholder pointers used here.
"""
import ctypes

import pytest
import torch

import w4a4_mxfp4_post_b200 as kq

P = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    from w4a4_mxfp4_post_b200 import build

    build.build()
    return kq.lib()


def cache(pages=4, heads=2, page=16, d=64, kc=16, ks=16, vc=16, vs=16):
    return kq._CACHE.pack(kc or 0, ks or 0, vc or 0, vs or 0, pages, heads, page, d)


def batch(table=16, stride=3, pages=3, cu=16, lens=16, B=2):
    return kq._BATCH.pack(table or 0, stride, pages, cu or 0, lens or 0, B)


def err(L):
    return L.kq_last_error().decode()


def test_gemv_refusals(L):
    def call(x=16, ldx=64, c=16, s=16, o=16, M=2, N=8, K=64, ws=None, n=0):
        return L.mxf4_gemv(P(x), ldx, P(c), P(s), P(o), 0, M, N, K, P(ws), n, None)

    assert call(M=33) == -2 and "mxf4_gemm" in err(L)
    assert call(M=-1) == -2 and call(N=-1) == -2 and call(K=48) == -2 and call(K=0) == -2
    assert call(N=1 << 31) == -2 and call(K=1 << 31, ldx=1 << 31) == -2
    assert call(ldx=56) == -2 and "ldx" in err(L)
    assert call(x=None) == -1 and call(c=None) == -1 and call(s=None) == -1 and call(o=None) == -1
    assert call(x=8) == -3 and call(c=8) == -3 and call(s=4) == -3 and call(o=8) == -3 and call(ldx=68) == -3
    assert call(x=None, c=None, s=None, o=None, M=0) == 0 and call(x=None, c=None, s=None, o=None, N=0) == 0
    assert err(L) == ""
    big = dict(M=17, N=1 << 20, K=1 << 12, ldx=1 << 12)
    need = L.mxf4_gemv_workspace(17, 1 << 20, 1 << 12)
    assert need > 0 and L.mxf4_gemv_workspace(2, 8, 64) == 0 and L.mxf4_gemv_workspace(0, 1 << 20, 1 << 12) == 0
    assert call(**big, ws=16, n=need - 1) == -2 and "workspace" in err(L)
    assert call(**big, n=need) == -1 and call(**big, ws=8, n=need) == -3
    for bad in ((33, 8, 64), (-1, 8, 64), (2, -1, 64), (2, 8, 48), (2, 8, 0), (2, 1 << 31, 64)):
        assert L.mxf4_gemv_workspace(*bad) == -1


SHAPES = [dict(d=48), dict(d=160), dict(d=0), dict(heads=0), dict(heads=65536), dict(page=8), dict(page=24), dict(page=0),
          dict(page=1 << 21), dict(pages=-1), dict(pages=1 << 31)]
BATCHES = [dict(B=-1), dict(pages=-1), dict(pages=4), dict(stride=1 << 32, pages=1 << 31), dict(stride=1 << 27, pages=1 << 27), dict(stride=(1 << 27) - (1 << 16) + 1, pages=(1 << 27) - (1 << 16) + 1)]


def write(L, c, b, k=16, v=16, st=128, sh=64, f32=0, T=4):
    return L.mx_cache_write(P(k), st, sh, P(v), st, sh, f32, c, b, T, None)


def read(L, c, b, k=16, v=16, starts=None, T=4):
    return L.mx_cache_read(c, b, P(starts), P(k), P(v), 0, T, None)


def attend(L, c, b, q=16, st=256, sh=64, o=16, T=4, hq=4, max_new=1, scale=1.0, ws=1024, n=1 << 40, causal=1):
    return L.mx_paged_attention(P(q), st, sh, c, b, scale, causal, P(o), T, hq, max_new,
                                P(ws), n, None)


@pytest.mark.parametrize("fn", [write, read, attend])
def test_shared_refusals(L, fn):
    for kw in SHAPES:
        assert fn(L, cache(**kw), batch()) == -2, kw
    for kw in BATCHES:
        assert fn(L, cache(), batch(**kw)) == -2, kw
    assert fn(L, cache(), batch(), T=-1) == -2 and fn(L, cache(), batch(), T=1 << 31) == -2
    for name in ("kc", "ks", "vc", "vs"):
        assert fn(L, cache(**{name: None}), batch()) == -1
        assert fn(L, cache(**{name: 8}), batch()) == -3
    assert fn(L, cache(), batch(table=None)) == -1 and fn(L, cache(), batch(cu=None)) == -1
    assert fn(L, cache(), batch(table=2)) == -3 and fn(L, cache(), batch(cu=2)) == -3
    assert fn(L, cache(), batch(), T=0) == 0 and fn(L, cache(), batch(B=0)) == 0
    assert err(L) == ""


def test_null_structs(L):
    c, b = cache(), batch()
    assert L.mx_cache_write(P(16), 128, 64, P(16), 128, 64, 0, None, b, 4, None) == -1
    assert L.mx_cache_read(c, None, None, P(16), P(16), 0, 4, None) == -1
    assert L.mx_paged_attention(P(16), 256, 64, None, None, 1.0, 1, P(16), 4, 4, 1, None, 0, None) == -1


def test_cache_refusals(L):
    assert write(L, cache(), batch(lens=None)) == -1
    assert write(L, cache(), batch(), k=None) == -1 and write(L, cache(), batch(), v=None) == -1
    assert write(L, cache(), batch(), k=8) == -3 and write(L, cache(), batch(), v=24) == -3
    assert write(L, cache(), batch(), st=132) == -3 and write(L, cache(), batch(), sh=66, f32=1) == -3
    assert write(L, cache(), batch(), st=-128) == -2 and write(L, cache(), batch(), sh=-64) == -2
    # a pool without pages holds nothing to write
    assert write(L, cache(pages=0, kc=None, ks=None, vc=None, vs=None), batch()) == 0
    assert read(L, cache(), batch(), k=None) == -1 and read(L, cache(), batch(), v=8) == -3
    assert read(L, cache(), batch(), starts=2) == -3


def test_attention_refusals(L):
    assert attend(L, cache(), batch(lens=None)) == -1
    assert attend(L, cache(), batch(), hq=3) == -2 and "heads_q" in err(L)
    assert attend(L, cache(), batch(), hq=0) == -2 and attend(L, cache(), batch(), hq=-4) == -2
    assert attend(L, cache(), batch(), max_new=-1) == -2
    assert attend(L, cache(), batch(), T=(1 << 31) - 1, hq=4) == -2 and attend(L, cache(), batch(), scale=3e38) == -2
    assert attend(L, cache(), batch(), scale=float("nan")) == -2 and attend(L, cache(), batch(), scale=float("inf")) == -2
    assert attend(L, cache(), batch(), q=None) == -1 and attend(L, cache(), batch(), o=None) == -1
    assert attend(L, cache(), batch(), q=8) == -3 and attend(L, cache(), batch(), o=8) == -3
    assert attend(L, cache(), batch(), st=252) == -3 and attend(L, cache(), batch(), sh=-64) == -2
    assert L.mx_attention_workspace(4, 4, 2, 64, 1) >= 0
    assert L.mx_attention_workspace(-1, 4, 2, 64, 1) == -1 and L.mx_attention_workspace(4, 0, 2, 64, 1) == -1
    assert L.mx_attention_workspace(4, 4, 2, 48, 1) == -1 and L.mx_attention_workspace(4, 4, 2, 64, -1) == -1
    assert L.mx_attention_workspace(4, 4, 0, 64, 1) == -1 and L.mx_attention_workspace(4, 4, 3, 64, 1) == -1
    assert attend(L, cache(), batch(), n=64) == -2 and "workspace" in err(L)


def test_binding_refuses_cpu_and_wrong_types():
    x, c = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 32, dtype=torch.uint8)
    with pytest.raises(ValueError):
        kq.mxf4_gemv(x, c, torch.zeros(512, dtype=torch.uint8))
    with pytest.raises(TypeError):
        kq.mxf4_gemv(x.float(), c, torch.zeros(512, dtype=torch.uint8))
    kc, ks = torch.zeros(2, 1, 16, 32, dtype=torch.uint8), torch.zeros(2, 1, 16, 2, dtype=torch.uint8)
    i32 = dict(dtype=torch.int32)
    seqs = (torch.zeros(1, 2, **i32), torch.zeros(2, **i32), torch.zeros(1, **i32))
    k = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kq.mx_cache_write(k, k, kc, ks, kc, ks, *seqs)
    with pytest.raises(ValueError):
        kq.mx_cache_read(kc, ks, kc, ks, seqs[0], seqs[1], 1)
    with pytest.raises(ValueError):
        kq.mx_paged_attention(k, kc, ks, kc, ks, *seqs)
    with pytest.raises(TypeError):
        kq.mx_paged_attention(k.numpy() if False else [1], kc.int(), ks, kc, ks, *seqs)
