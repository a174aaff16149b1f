"""The C ABI of the 4-bit cache on a host without a GPU: exports and argument
checks, which return before any CUDA call, and what the binding refuses."""
import ctypes
import os
import re
import subprocess

import pytest

import attention_qk_norm_b200 as qkn
from attention_qk_norm_b200 import _kv4
from attention_qk_norm_b200 import buildlib as qbuild

OK, NULL, SHAPE, ALIGN, UNSUP, EPS = 0, -1, -2, -3, -5, -7
BF16, FP32, FP16, FP8 = 0, 1, 2, 3
P, G1, G2, POOL, S, TAB, LEN, QS, OUT, WS = (i << 20 for i in range(1, 11))  # never read


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return _kv4._lib()


def test_exports_every_declared_symbol(lib):
    text = open(os.path.join(qbuild.INCLUDE, "qknorm_kv4.h")).read()
    names = set(re.findall(r"^int (qknorm_kv4_\w+)\s*\(", text, re.M))
    out = subprocess.run(["nm", "-D", "--defined-only", qbuild.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert names == set(re.findall(r"\bT (qknorm_kv4_\w+)$", out, re.M))
    assert len(names) == 8
    assert lib.qknorm_kv4_version() == 100
    assert lib.qknorm_kv4_last_cuda_error() == 0
    assert lib.qknorm_kv4_bad_pages(None) == NULL


def append(lib, qkv=P, dtype=BF16, T=4, Hq=16, Hk=2, D=128, stride=None, gq=G1, gk=G2, eps=1e-6,
           slots=S, pool=POOL, pages=8, page=64, scores=None):
    stride = (Hq + 2 * Hk) * D if stride is None else stride
    return lib.qknorm_kv4_append(qkv, dtype, T, Hq, Hk, D, stride, gq, gk, eps, slots, pool,
                                 pages, page, scores, None)


def test_append_validation(lib):
    f = append
    assert f(lib, dtype=4) == UNSUP and f(lib, dtype=-1) == UNSUP
    assert f(lib, D=96) == UNSUP and f(lib, D=32) == UNSUP
    for bad in (dict(T=-1), dict(Hq=-1), dict(Hk=0), dict(stride=20 * 128 - 8), dict(pages=0),
                dict(pages=-1), dict(page=0), dict(page=48), dict(page=512), dict(page=8),
                dict(pages=2 ** 62)):
        assert f(lib, **bad) == SHAPE, bad
    assert f(lib, eps=-1.0) == EPS and f(lib, eps=float("nan")) == EPS
    for bad in (dict(qkv=None), dict(slots=None), dict(pool=None), dict(gq=None), dict(gk=None)):
        assert f(lib, **bad) == NULL, bad
    for bad in (dict(qkv=P + 8), dict(slots=S + 4), dict(pool=POOL + 8), dict(gq=G1 + 4),
                dict(gk=G2 + 8), dict(scores=P + 2), dict(stride=20 * 128 + 4),
                dict(dtype=FP8, stride=20 * 128 + 8)):
        assert f(lib, **bad) == ALIGN, bad
    assert f(lib, T=0, qkv=None, slots=None, pool=None) == OK
    assert f(lib, Hq=0, gq=None, qkv=P + 8) == ALIGN  # no query heads need no gamma_q
    assert f(lib, gq=None, gk=None, qkv=P + 8) == ALIGN  # no weights: nothing normalised


def test_read_validation(lib):
    def f(pool=POOL, pages=8, page=64, Hk=2, D=128, slots=S, N=3, k=P, v=G1, dtype=BF16,
          stride=256):
        return lib.qknorm_kv4_read(pool, pages, page, Hk, D, slots, N, k, v, dtype, stride, None)

    assert f(D=96) == UNSUP and f(dtype=9) == UNSUP
    for bad in (dict(N=-1), dict(Hk=0), dict(page=40), dict(stride=255), dict(pages=0)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(pool=None), dict(slots=None), dict(k=None, v=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(k=P + 8), dict(v=G1 + 2), dict(slots=S + 4), dict(stride=260),
                dict(pool=POOL + 4)):
        assert f(**bad) == ALIGN, bad
    assert f(N=0, slots=None) == OK


def attention(lib, q=P, dtype=BF16, T=3, Hq=16, Hk=2, D=128, stride=20 * 128, pool=POOL, pages=8,
              page=64, table=TAB, tstride=4, maxp=4, lens=LEN, B=3, starts=None, max_q=1,
              scale=0.1, out=OUT, ostride=16 * 128, lse=None, scores=None, ws=WS, wsb=1 << 40):
    return lib.qknorm_kv4_attention(q, dtype, T, Hq, Hk, D, stride, pool, pages, page, table,
                                    tstride, maxp, lens, B, starts, max_q, scale, out, ostride,
                                    lse, scores, ws, wsb, None)


def test_attention_validation(lib):
    f = attention
    assert f(lib, dtype=7) == UNSUP and f(lib, D=80, stride=20 * 80, ostride=16 * 80) == UNSUP
    for bad in (dict(T=-1), dict(Hq=15), dict(Hq=0), dict(Hk=0), dict(stride=16 * 128 - 8),
                dict(ostride=16 * 128 - 8), dict(pages=0), dict(page=24), dict(page=512),
                dict(maxp=5), dict(maxp=-1), dict(maxp=1 << 40), dict(B=-1), dict(B=2),
                dict(max_q=0), dict(max_q=2), dict(scale=float("inf")),
                dict(scale=float("nan")), dict(wsb=0), dict(B=1 << 20, T=1 << 20)):
        assert f(lib, **bad) == SHAPE, bad
    for bad in (dict(q=None), dict(pool=None), dict(table=None), dict(lens=None), dict(out=None),
                dict(ws=None)):
        assert f(lib, **bad) == NULL, bad
    for bad in (dict(q=P + 8), dict(pool=POOL + 8), dict(out=OUT + 8), dict(ws=WS + 8),
                dict(table=TAB + 2), dict(lens=LEN + 1), dict(lse=P + 2), dict(scores=P + 1),
                dict(starts=QS + 2, max_q=4), dict(stride=20 * 128 + 4),
                dict(ostride=16 * 128 + 4)):
        assert f(lib, **bad) == ALIGN, bad
    assert f(lib, T=0, B=0, q=None, pool=None, out=None) == OK


def test_attention_workspace(lib):
    n = ctypes.c_int64(7)
    w = lib.qknorm_kv4_attention_workspace
    assert w(3, BF16, 16, 2, 128, 1, 256, 0, None) == NULL
    assert w(3, BF16, 15, 2, 128, 1, 256, 0, n) == SHAPE and n.value == 0
    assert w(3, BF16, 16, 2, 128, 1, 256, 0, n) == OK and n.value > 0
    small = n.value
    assert w(3, BF16, 16, 2, 128, 1, 256, 1, n) == OK and n.value >= small
    # Enough is accepted (the call then meets the next check), one byte less is not.
    assert attention(lib, wsb=small - 1) == SHAPE
    assert w(65535, FP32, 128, 8, 256, 65535, 2 ** 30, 1, n) == OK and n.value > 0
    assert w(1, FP32, 128, 8, 256, 1, 2 ** 30 + 1, 1, n) == SHAPE
    # More rows or units than 32-bit numbers hold: refused before anything is touched.
    assert w(1, BF16, 65535, 1, 64, 65535, 256, 0, n) == SHAPE
    big = dict(B=60000, T=60000, maxp=1 << 20, tstride=1 << 20, wsb=2 ** 62)
    assert attention(lib, **big) == SHAPE


def test_evict_validation(lib):
    def f(pool=POOL, pages=8, page=64, Hk=2, D=128, scores=S, table=TAB, tstride=4, maxp=4,
          lens=LEN, B=2, dst=QS, dstride=2, dpages=2, budget=100, recent=10, new=OUT, kept=WS):
        return lib.qknorm_kv4_evict(pool, pages, page, Hk, D, scores, table, tstride, maxp, lens,
                                    B, dst, dstride, dpages, budget, recent, new, kept, None)

    assert f(D=32) == UNSUP
    for bad in (dict(budget=0), dict(budget=129), dict(recent=-1), dict(recent=101), dict(B=-1),
                dict(tstride=3), dict(dstride=1), dict(dpages=1), dict(page=33), dict(pages=0),
                dict(Hk=0), dict(maxp=-1), dict(dpages=-1), dict(B=1 << 31),
                dict(maxp=(1 << 24) + 1, tstride=1 << 25)):
        assert f(**bad) == SHAPE, bad
    for bad in (dict(pool=None), dict(scores=None), dict(table=None), dict(lens=None),
                dict(dst=None), dict(new=None), dict(kept=None)):
        assert f(**bad) == NULL, bad
    for bad in (dict(pool=POOL + 8), dict(scores=S + 2), dict(table=TAB + 1), dict(lens=LEN + 2),
                dict(dst=QS + 2), dict(new=OUT + 1), dict(kept=WS + 3)):
        assert f(**bad) == ALIGN, bad
    assert f(B=0, pool=None, scores=None) == OK


def test_binding_refuses_host_tensors_and_bad_caches():
    import torch

    pool = torch.zeros(2, 1, 4, 16 * 128 + 128, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        qkn.KV4Cache(pool, 1, 128)
    with pytest.raises(ValueError, match="D must"):
        qkn.KV4Cache(pool, 1, 96)
    with pytest.raises(ValueError, match="page_size"):
        qkn.KV4Cache(pool, 1, 128, page_size=100)
    with pytest.raises(ValueError, match="page_size"):
        qkn.KV4Cache.empty(2, 1, 128, page_size=100, device="cpu")
