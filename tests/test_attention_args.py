"""CPU checks of the paged-cache entry points: argument errors that return
before any CUDA call, workspace sizes, rotation phases.  No kernel runs."""
import ctypes
import math
from fractions import Fraction

import pytest

from tree_verified_speculative_gb300 import build as mfd_build
from tree_verified_speculative_gb300 import mfd

P = 0x100000
INV, UNS, WS = mfd.MFD_ERR_INVALID_ARG, mfd.MFD_ERR_UNSUPPORTED, mfd.MFD_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    mfd_build.build()
    return mfd.load()


def cache(**kw):
    f = dict(k=P, v=P, k_exp=None, v_exp=None, block_table=P, dtype=mfd.MFD_BF16, n_pages=10, page_size=16, max_pages=4,
             Hk=2, D=64, page_stride=2 * 16 * 64, head_stride=16 * 64, token_stride=64)
    f.update(kw)
    return mfd._KvCacheStruct(*[f[n] for n, _ in mfd._KvCacheStruct._fields_])


BAD_CACHE = [
    (dict(k=None), INV), (dict(v=None), INV), (dict(block_table=None), INV), (dict(k=P + 8), INV), (dict(v=P + 2), INV),
    (dict(dtype=3), INV), (dict(dtype=-1), INV), (dict(n_pages=0), INV), (dict(max_pages=0), INV), (dict(Hk=0), INV),
    (dict(D=0), INV), (dict(page_size=0), INV), (dict(page_size=8), UNS), (dict(page_size=24), UNS), (dict(page_size=512), UNS),
    (dict(D=72), UNS), (dict(D=272, token_stride=272, head_stride=16 * 272, page_stride=32 * 272), UNS),
    (dict(token_stride=63), INV), (dict(token_stride=68), INV), (dict(head_stride=-1024), INV), (dict(page_stride=0), INV),
    (dict(page_stride=1 << 40), UNS), (dict(dtype=mfd.MFD_E4M3), INV), (dict(dtype=mfd.MFD_E4M3, k_exp=P), INV),
    (dict(max_pages=(1 << 31) // 16), UNS),
]


def attend(lib, c, q=P, qs=8 * 64, dtype=mfd.MFD_BF16, R=1, N=1, Hq=8, ctx=P, nodes=None, mask=None, scale=0.1, out=P, lse=None,
           status=P, ws=P, wsb=1 << 40):
    return lib.mfd_tree_attention(q, qs, dtype, R, N, Hq, ctypes.byref(c) if c else None, ctx, nodes, mask, scale, out, lse,
                                  status, ws, wsb, None)


def append(lib, c, q=P, qs=8 * 64, k=P, ks=128, v=P, vs=128, dtype=mfd.MFD_BF16, R=1, N=1, Hq=8, qw=None, kw=None, eps=1e-6,
           phase=P, rot=64, pos=P, ctx=P, nodes=None, q_out=P, status=P):
    return lib.mfd_kv_append(q, qs, k, ks, v, vs, dtype, R, N, Hq, qw, kw, eps, phase, rot, 0, pos, ctx, nodes, q_out,
                             ctypes.byref(c) if c else None, status, None)


@pytest.mark.parametrize("i", range(len(BAD_CACHE)))
def test_every_call_refuses_a_bad_cache(lib, i):
    kw, code = BAD_CACHE[i]
    c = cache(**kw)
    assert attend(lib, c) == code
    assert append(lib, c) == code
    assert lib.mfd_kv_read(ctypes.byref(c), 1, 4, P, P, mfd.MFD_BF16, P, P, P, None) == code
    assert lib.mfd_kv_commit(ctypes.byref(c), 1, 15, P, P, P, P, P, P, None) == code


def test_no_cache(lib):
    assert attend(lib, None) == INV and append(lib, None) == INV
    assert lib.mfd_kv_read(None, 1, 4, P, P, mfd.MFD_BF16, P, P, P, None) == INV
    assert lib.mfd_kv_commit(None, 1, 15, P, P, P, P, P, P, None) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INV), (dict(q=P + 4), INV), (dict(qs=8 * 64 - 8), INV), (dict(qs=8 * 64 + 4), INV), (dict(dtype=mfd.MFD_E4M3), INV),
    (dict(dtype=mfd.MFD_FP16), INV), (dict(R=0), INV), (dict(N=0), INV), (dict(Hq=0), INV), (dict(ctx=None), INV),
    (dict(out=None), INV), (dict(out=P + 8), INV), (dict(status=None), INV), (dict(scale=0.0), INV), (dict(scale=-1.0), INV),
    (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(R=1025), UNS), (dict(N=4097), UNS), (dict(Hq=7, qs=7 * 64), UNS),
    (dict(Hq=1026, qs=1026 * 64), UNS), (dict(N=4096, Hq=64, qs=64 * 64), UNS), (dict(ws=None), WS), (dict(ws=P + 16), WS), (dict(wsb=16), WS),
])
def test_attention_refusals(lib, kw, code):
    assert attend(lib, cache(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(k=P + 4), INV), (dict(ks=120), INV), (dict(vs=132), INV),
    (dict(q_out=None), INV), (dict(qw=P + 2), INV), (dict(kw=P + 8), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV),
    (dict(phase=None), INV), (dict(rot=63), INV), (dict(rot=66), INV), (dict(rot=-2), INV), (dict(pos=None), INV), (dict(ctx=None), INV),
    (dict(status=None), INV), (dict(R=0), INV), (dict(N=0), INV), (dict(Hq=-1), INV), (dict(dtype=mfd.MFD_E4M3), INV),
    (dict(dtype=mfd.MFD_FP16), INV), (dict(Hq=1025, qs=1025 * 64), UNS), (dict(R=1 << 16, N=1 << 15), UNS),
])
def test_append_refusals(lib, kw, code):
    assert append(lib, cache(), **kw) == code


def test_norm_read_commit_refusals(lib):
    def norm(q=P, k=P, D=64, T=1, rot=64, phase=P, qo=P, ko=P, Hq=8, Hk=2, status=P, dtype=mfd.MFD_BF16):
        return lib.mfd_qk_norm_rope(q, Hq * max(D, 1), k, Hk * max(D, 1), dtype, T, Hq, Hk, D, None, None, 1e-6, phase, rot, 0, P, qo, ko,
                                    status, None)
    for kw, code in ((dict(q=None), INV), (dict(k=None), INV), (dict(D=0), INV), (dict(D=72), UNS), (dict(D=272), UNS), (dict(T=0), INV),
                     (dict(phase=None), INV), (dict(qo=None), INV), (dict(ko=P + 2), INV), (dict(Hk=0), INV), (dict(status=None), INV),
                     (dict(dtype=2), INV), (dict(Hq=2000), UNS)):
        assert norm(**kw) == code, kw

    def read(c=None, R=1, L=4, start=P, length=P, dtype=mfd.MFD_BF16, ko=P, vo=P, status=P):
        return lib.mfd_kv_read(ctypes.byref(c or cache()), R, L, start, length, dtype, ko, vo, status, None)
    for kw, code in ((dict(R=0), INV), (dict(L=0), INV), (dict(start=None), INV), (dict(length=None), INV), (dict(dtype=2), INV),
                     (dict(dtype=mfd.MFD_FP16), INV), (dict(ko=None), INV), (dict(vo=P + 4), INV), (dict(status=None), INV), (dict(R=65536), UNS)):
        assert read(**kw) == code, kw

    def commit(R=1, L=15, ptrs=(P,) * 6):
        return lib.mfd_kv_commit(ctypes.byref(cache()), R, L, *ptrs, None)
    assert commit(R=0) == INV and commit(L=0) == INV and commit(L=17) == UNS
    for i in range(6):
        assert commit(ptrs=tuple(None if j == i else P for j in range(6))) == INV


def test_workspace_bytes_limits(lib):
    size = mfd.mfd_tree_attention_workspace_bytes
    for args in ((0, 1, 8, 2, 64), (1025, 1, 8, 2, 64), (1, 0, 8, 2, 64), (1, 4097, 8, 2, 64), (1, 1, 9, 2, 64), (1, 1, 8, 2, 72),
                 (1, 1, 8, 2, 272), (1, 4096, 128, 2, 64), (1, 1, 0, 2, 64), (1, 1, 8, 0, 64)):
        assert size(*args) == 0, args


def test_rope_phases(lib):
    """phase = frac(inv_freq / 2 pi) in units of 2^-64 turns, to a double's
    precision of the quotient."""
    f = [1.0, 1.0e6 ** -0.5, 3.0e-7, 0.0, 7.5, 2 * math.pi]
    src, dst = (ctypes.c_double * len(f))(*f), (ctypes.c_uint64 * len(f))()
    assert lib.mfd_rope_phases(ctypes.addressof(src), len(f), ctypes.addressof(dst)) == mfd.MFD_OK
    pi = Fraction(314159265358979323846264338327950288419716939937510, 10 ** 50)
    for x, got in zip(f, dst):
        turns = Fraction(x) / (2 * pi)
        off = (Fraction(got, 1 << 64) - turns) % 1
        assert min(off, 1 - off) <= max(turns, 1) * Fraction(1, 1 << 51), x
    assert lib.mfd_rope_phases(None, 1, ctypes.addressof(dst)) == INV
    assert lib.mfd_rope_phases(ctypes.addressof(src), 0, ctypes.addressof(dst)) == INV
    for bad in (-1.0, math.nan, math.inf):
        one = (ctypes.c_double * 1)(bad)
        assert lib.mfd_rope_phases(ctypes.addressof(one), 1, ctypes.addressof(dst)) == INV
