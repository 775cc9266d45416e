"""CPU checks of the recurrent layers' entry points: argument errors that
return before any CUDA call, and what the binding refuses before any address is
taken.  No kernel runs."""
import ctypes
import math
from types import SimpleNamespace

import pytest
import torch

from tree_verified_speculative_gb300 import build as mfd_build
from tree_verified_speculative_gb300 import mfd

P = 0x100000
INV, UNS = mfd.MFD_ERR_INVALID_ARG, mfd.MFD_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    mfd_build.build()
    return mfd.load()


def state(**kw):
    f = dict(s=P, n_slots=4, Hv=4, Dk=64, Dv=64)
    f.update(kw)
    return mfd._DeltaStateStruct(*[f[n] for n, _ in mfd._DeltaStateStruct._fields_])


def rule(lib, c, q=P, qs=128, k=P, ks=128, v=P, vs=256, dtype=mfd.MFD_BF16, R=1, N=1, Hk=2, g=P, beta=P, norm=1, eps=1e-6, scale=0.1,
         nodes=None, out=P, src=None, dst=None, status=P):
    return lib.mfd_delta_rule(q, qs, k, ks, v, vs, dtype, R, N, Hk, g, beta, norm, eps, scale, nodes, out,
                              ctypes.byref(c) if c else None, src, dst, status, None)


def tree(lib, c, q=P, qs=128, k=P, ks=128, v=P, vs=256, dtype=mfd.MFD_BF16, R=1, N=1, Hk=2, g=P, beta=P, norm=1, eps=1e-6, scale=0.1,
         parent=P, nodes=None, out=P, src=None, dst=None, status=P):
    return lib.mfd_delta_tree(q, qs, k, ks, v, vs, dtype, R, N, Hk, g, beta, norm, eps, scale, parent, nodes, out,
                              ctypes.byref(c) if c else None, src, status, None)


def commit(lib, c, k=P, ks=128, v=P, vs=256, dtype=mfd.MFD_BF16, R=1, N=1, Hk=2, g=P, beta=P, norm=1, eps=1e-6, L=15, accept=P, path=P,
           nodes=None, src=None, dst=None, status=P):
    return lib.mfd_delta_commit(k, ks, v, vs, dtype, R, N, Hk, g, beta, norm, eps, L, accept, path, nodes,
                                ctypes.byref(c) if c else None, src, dst, status, None)


@pytest.mark.parametrize("kw,code", [(dict(s=None), INV), (dict(s=P + 8), INV), (dict(n_slots=0), INV), (dict(Hv=0), INV), (dict(Dk=0), INV),
                                     (dict(Dv=-16), INV), (dict(Dk=72), UNS), (dict(Dk=144), UNS), (dict(Dv=40), UNS), (dict(Dv=272), UNS),
                                     (dict(Hv=1026), UNS), (dict(Hv=3), UNS)])
def test_every_form_refuses_bad_states(lib, kw, code):
    c = state(**kw)
    wide = dict(ks=4096, vs=1 << 20)
    assert rule(lib, c, qs=4096, **wide) == code and tree(lib, c, qs=4096, **wide) == code and commit(lib, c, **wide) == code


COMMON = [
    (dict(k=None), INV), (dict(v=None), INV), (dict(k=P + 8), INV), (dict(ks=120), INV), (dict(ks=132), INV), (dict(vs=248), INV),
    (dict(dtype=mfd.MFD_E4M3), INV), (dict(dtype=-1), INV), (dict(R=0), INV), (dict(N=0), INV), (dict(Hk=0), INV), (dict(g=None), INV),
    (dict(beta=None), INV), (dict(g=P + 2), INV), (dict(norm=2), INV), (dict(eps=-1.0), INV), (dict(eps=math.nan), INV), (dict(eps=math.inf), INV),
    (dict(status=None), INV), (dict(nodes=P + 1), INV), (dict(src=P + 2), INV), (dict(R=1 << 27), UNS), (dict(Hk=3), UNS),
]


@pytest.mark.parametrize("i", range(len(COMMON)))
def test_every_form_refuses(lib, i):
    kw, code = COMMON[i]
    assert commit(lib, state(), **kw) == code
    assert rule(lib, state(), **kw) == code and tree(lib, state(), **kw) == code


def test_refusals_of_each_form(lib):
    for f in (rule, tree):
        for kw in (dict(q=None), dict(q=P + 2), dict(qs=120), dict(out=None), dict(out=P + 8), dict(scale=math.nan), dict(scale=math.inf)):
            assert f(lib, state(), **kw) == INV, kw
        assert f(lib, None) == INV
    assert rule(lib, state(), R=1 << 16, N=1 << 15) == UNS
    assert rule(lib, state(), dst=P + 1) == INV and commit(lib, state(), dst=P + 1) == INV
    assert tree(lib, state(), parent=None) == INV and tree(lib, state(), parent=P + 2) == INV and tree(lib, state(), N=514) == UNS
    for kw, code in ((dict(accept=None), INV), (dict(path=None), INV), (dict(L=0), INV), (dict(L=17), UNS), (dict(path=P + 2), INV)):
        assert commit(lib, state(), **kw) == code, kw
    assert commit(lib, None) == INV


def test_norm_refusals(lib):
    def gated(x=P, xs=256, z=P, zs=256, dtype=mfd.MFD_BF16, T=1, heads=4, D=64, w=P, eps=1e-6, act=2, out=P):
        return lib.mfd_gated_norm(x, xs, z, zs, dtype, T, heads, D, w, eps, act, out, None)
    for kw, code in ((dict(x=None), INV), (dict(z=None), INV), (dict(w=None), INV), (dict(out=None), INV), (dict(x=P + 8), INV), (dict(w=P + 2), INV),
                     (dict(xs=248), INV), (dict(zs=260), INV), (dict(T=0), INV), (dict(heads=0), INV), (dict(D=0), INV), (dict(dtype=2), INV),
                     (dict(eps=-1.0), INV), (dict(eps=math.nan), INV), (dict(act=3), INV), (dict(act=-1), INV), (dict(D=60), UNS),
                     (dict(D=264, xs=4096, zs=4096), UNS), (dict(heads=1025, xs=1 << 20, zs=1 << 20), UNS), (dict(T=1 << 30), UNS)):
        assert gated(**kw) == code, kw

    def block(y=P, r=P, dtype=mfd.MFD_BF16, T=1, H=64, wa=P, z=None, zs=0, act=0, scale=1.0, wb=P, eps=1e-6, ro=P, xo=2 * P):
        return lib.mfd_residual_norm(y, r, dtype, T, H, wa, z, zs, act, scale, wb, eps, ro, xo, None)
    for kw, code in ((dict(y=None), INV), (dict(r=None), INV), (dict(ro=None), INV), (dict(xo=None), INV), (dict(wb=None), INV), (dict(y=P + 8), INV),
                     (dict(wa=P + 2), INV), (dict(z=P + 2), INV), (dict(z=P, zs=56), INV), (dict(z=P, zs=68), INV), (dict(T=0), INV), (dict(H=0), INV),
                     (dict(dtype=2), INV), (dict(eps=-1.0), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV), (dict(act=3), INV),
                     (dict(H=60), UNS), (dict(H=16392), UNS), (dict(xo=P), INV)):
        assert block(**kw) == code, kw


def _call(form, **kw):
    R, N, Hk, Hv, Dk, Dv = 2, 3, 2, 4, 64, 32
    a = dict(q=torch.zeros((R, N, Hk, Dk), dtype=torch.bfloat16), k=torch.zeros((R, N, Hk, Dk), dtype=torch.bfloat16),
             v=torch.zeros((R, N, Hv, Dv), dtype=torch.bfloat16), g=torch.zeros((R, N, Hv)), beta=torch.zeros((R, N, Hv)),
             nodes=torch.zeros(R, dtype=torch.int32), out=torch.zeros((R, N, Hv, Dv), dtype=torch.bfloat16), src=None, dst=None,
             state=SimpleNamespace(n_slots=2, Hv=Hv, Dk=Dk, Dv=Dv, _c=None, device=0, s=torch.zeros(1)), status=torch.zeros(1, dtype=torch.int32),
             parent=torch.zeros((R, N), dtype=torch.int32), accept=torch.zeros(R, dtype=torch.int32),
             path=torch.zeros((R, 4), dtype=torch.int32))
    a.update(kw)
    if form == "rule":
        mfd.mfd_delta_rule(a["q"], a["k"], a["v"], a["g"], a["beta"], 1e-6, 0.1, a["nodes"], a["out"], a["state"], a["src"], a["dst"], a["status"])
    elif form == "tree":
        mfd.mfd_delta_tree(a["q"], a["k"], a["v"], a["g"], a["beta"], 1e-6, 0.1, a["parent"], a["nodes"], a["out"], a["state"], a["src"], a["status"])
    else:
        mfd.mfd_delta_commit(a["k"], a["v"], a["g"], a["beta"], 1e-6, a["accept"], a["path"], a["nodes"], a["state"], a["src"], a["dst"], a["status"])


BAD = [(dict(k=torch.zeros((2, 3, 2, 64))), "bf16 or fp16"), (dict(v=torch.zeros((2, 3, 4, 32), dtype=torch.float16)), "bf16 or fp16"),
       (dict(k=torch.zeros((2, 3, 2, 32), dtype=torch.bfloat16)), "k .n_req"), (dict(v=torch.zeros((2, 3, 2, 32), dtype=torch.bfloat16)), "k .n_req"),
       (dict(g=torch.zeros((2, 3, 4), dtype=torch.float64)), "g and beta"), (dict(beta=torch.zeros((2, 3, 2))), "g and beta"),
       (dict(nodes=torch.zeros(2, dtype=torch.int64)), "n_nodes"), (dict(src=torch.zeros(1, dtype=torch.int32)), "n_nodes"),
       (dict(status=torch.zeros(1)), "status"),
       (dict(state=SimpleNamespace(n_slots=1, Hv=4, Dk=64, Dv=32, _c=None, device=0, s=torch.zeros(1))), "slot for each")]


@pytest.mark.parametrize("form", ["rule", "tree", "commit"])
@pytest.mark.parametrize("i", range(len(BAD)))
def test_the_binding_refuses(form, i):
    kw, match = BAD[i]
    with pytest.raises(AssertionError, match=match):
        _call(form, **kw)


@pytest.mark.parametrize("form", ["rule", "tree", "commit"])
def test_the_right_types_go_on_to_the_device_check(form):
    with pytest.raises(AssertionError, match="device"):
        _call(form)


def test_states_refuse():
    for bad in (torch.zeros((2, 4, 64)), torch.zeros((2, 4, 64, 64), dtype=torch.bfloat16)):
        with pytest.raises(AssertionError, match="states"):
            mfd.DeltaState.from_tensor(bad)
    with pytest.raises(AssertionError, match="device"):
        mfd.DeltaState.from_tensor(torch.zeros((2, 4, 64, 64)))
