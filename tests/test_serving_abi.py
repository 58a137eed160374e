"""Refusals of the serving entry points, on the host before any CUDA call. CPU only."""

import pytest
import torch

import jagged_pointwise_attention_b200 as hstu
from jagged_pointwise_attention_b200 import _native
from jagged_pointwise_attention_b200.build import build

INV, UNS, OK = _native.HSTU_ERR_INVALID_ARG, _native.HSTU_ERR_UNSUPPORTED, _native.HSTU_OK


@pytest.fixture(scope="module")
def lib():
    build()
    return _native.load()


def test_cache_plan(lib):
    def call(ctx=16, off=16, B=2, T=4, page=16, free=16, nf=4, start=16, table=16, stride=8, maxp=8,
             slots=16, end=32):
        return lib.hstu_cache_plan(ctx, off, B, T, page, free, nf, start, table, stride, maxp, slots,
                                   end, None)
    for kw in (dict(ctx=None), dict(off=None), dict(start=None), dict(table=None), dict(end=None),
               dict(slots=None), dict(free=None), dict(B=0), dict(B=-1), dict(T=-1), dict(nf=-1),
               dict(maxp=0), dict(stride=7), dict(end=16)):
        assert call(**kw) == INV, kw
    for page in (0, 8, 15, 48, 2048, -16):
        assert call(page=page) == UNS
    assert call(maxp=1 << 28, stride=1 << 28) == UNS


def test_cache_append(lib):
    def call(dt=1, k=16, ks=128, v=16, vs=128, ts=16, slots=16, T=4, H=2, dqk=64, dv=64, kc=16,
             kp=2048, kt=128, vc=16, vp=2048, vt=128, tsc=16, tsp=16, n=4, page=16):
        return lib.hstu_cache_append(dt, k, ks, v, vs, ts, slots, T, H, dqk, dv, kc, kp, kt, vc, vp,
                                     vt, tsc, tsp, n, page, None)
    for kw in (dict(dt=5), dict(k=None), dict(v=None), dict(slots=None), dict(kc=None), dict(vc=None),
               dict(ts=None), dict(tsc=None), dict(T=-1), dict(H=0), dict(dqk=0), dict(ks=127),
               dict(vs=127), dict(kt=127), dict(vt=127), dict(kp=2047), dict(vp=2047), dict(tsp=15),
               dict(n=0), dict(n=1 << 28), dict(k=17)):
        assert call(**kw) == INV, kw
    assert call(page=24) == UNS
    assert call(T=0) == OK
    assert call(T=0, ts=None, tsc=None) == OK


def cached(lib, **kw):
    a = dict(dt=1, q=16, qs=128, kc=16, kp=2048, kt=128, vc=16, vp=2048, vt=128, tsc=16, tsp=16, n=4,
             page=16, table=16, tstride=8, maxp=8, ctx=16, off=16, B=2, T=4, max_new=2, H=2, dqk=64,
             dv=64, ts=16, par=None, pos=16, P=8, tb=16, NB=8, N=64, out=16, os=128, ws=16,
             wsb=1 << 28)
    a.update(kw)
    return lib.hstu_attn_cached_fwd(
        a["dt"], a["q"], a["qs"], a["kc"], a["kp"], a["kt"], a["vc"], a["vp"], a["vt"], a["tsc"],
        a["tsp"], a["n"], a["page"], a["table"], a["tstride"], a["maxp"], a["ctx"], a["off"], a["B"],
        a["T"], a["max_new"], a["H"], a["dqk"], a["dv"], a["ts"], a["par"], a["pos"], a["P"],
        a["tb"], a["NB"], a["N"], a["out"], a["os"], a["ws"], a["wsb"], None)


def test_attn_cached(lib):
    for kw in (dict(dt=9), dict(q=None), dict(kc=None), dict(vc=None), dict(table=None),
               dict(ctx=None), dict(off=None), dict(out=None), dict(ws=None), dict(wsb=1000),
               dict(ws=24), dict(q=24), dict(kc=24), dict(out=8), dict(qs=127), dict(qs=132),
               dict(kt=120), dict(kt=132, kp=16 * 132), dict(kp=2047), dict(vp=2040), dict(os=127),
               dict(tstride=7), dict(maxp=0), dict(B=-1), dict(T=-1), dict(max_new=0), dict(N=0),
               dict(N=131073), dict(H=0), dict(P=0), dict(NB=0), dict(NB=1025), dict(tsp=15),
               dict(n=0), dict(n=1 << 28)):
        assert cached(lib, **kw) == INV, kw
    for kw in (dict(page=8), dict(page=100), dict(par=16, max_new=257), dict(dqk=48, dv=48),
               dict(dv=32), dict(dqk=256, dv=256, qs=512),
               dict(dt=0, dqk=129, qs=258, kt=258, kp=16 * 258), dict(H=65536)):
        assert cached(lib, **kw) == UNS, kw
    assert cached(lib, B=0, T=0) == OK and cached(lib, T=0) == OK
    assert lib.hstu_attn_cached_workspace_bytes(1, 1, 64) > 0
    assert lib.hstu_attn_cached_workspace_bytes(0, 1, 64) > 0
    assert lib.hstu_attn_cached_workspace_bytes(1, 0, 64) == 0
    assert lib.hstu_attn_cached_workspace_bytes(7, 1, 64) == 0
    assert lib.hstu_attn_cached_workspace_bytes(1, 1, 129) == 0


def test_quant_and_linear_w4(lib):
    def quant(W=16, ldw=256, N=4, K=256, G=64, c=16, ldc=128, s=16, lds=4):
        return lib.hstu_quant_groups_w4(W, ldw, N, K, G, c, ldc, s, lds, None)
    for kw in (dict(W=None), dict(c=None), dict(s=None), dict(ldw=255), dict(ldc=127), dict(lds=3),
               dict(N=-1), dict(K=0), dict(W=17)):
        assert quant(**kw) == INV, kw
    for kw in (dict(G=16), dict(G=0), dict(G=256), dict(K=224, G=64)):
        assert quant(**kw) == UNS, kw
    assert quant(N=0) == OK

    def lin(x=16, ldx=256, M=2, K=256, c=16, ldc=128, s=16, lds=4, G=64, N=8, b=None, ep=0, r=None,
            ldr=8, y=16, ldy=8):
        return lib.hstu_linear_w4_fwd(x, ldx, M, K, c, ldc, s, lds, G, N, b, ep, r, ldr, y, ldy, None)
    for kw in (dict(x=None), dict(c=None), dict(s=None), dict(y=None), dict(ep=2), dict(ep=7),
               dict(M=-1), dict(K=0), dict(N=0), dict(ldx=248), dict(ldx=260), dict(ldc=112),
               dict(ldc=136), dict(lds=3), dict(ldy=7), dict(ep=2, r=16, ldr=7), dict(x=24),
               dict(c=24), dict(y=17), dict(b=18)):
        assert lin(**kw) == INV, kw
    for kw in (dict(G=16), dict(K=192, ldx=192, ldc=96)):
        assert lin(**kw) == UNS, kw
    assert lin(M=0) == OK


def test_binding_refuses(lib):
    z = torch.zeros
    cpu = z(2, 1, 64)
    off = torch.tensor([0, 2])
    with pytest.raises((ValueError, RuntimeError, AssertionError)):      # no CUDA device or CPU tensors
        hstu.hstu_cache_append(cpu, cpu, None, z(2, dtype=torch.int64), z(1, 16, 1, 64),
                               z(1, 16, 1, 64), None)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        hstu.hstu_cache_plan(z(1, dtype=torch.int32), off, z(1, dtype=torch.int32),
                             z(1, dtype=torch.int32), z(1, 4, dtype=torch.int32), 16, 2)


def test_arrays_off_their_elements_alignment(lib):
    """An address between two elements would fault on the device."""
    def plan(ctx=16, off=16, free=16, start=16, table=16, slots=16, end=32):
        return lib.hstu_cache_plan(ctx, off, 2, 4, 16, free, 4, start, table, 8, 8, slots, end, None)
    for kw in (dict(ctx=18), dict(off=20), dict(free=17), dict(start=18), dict(table=18), dict(slots=20),
               dict(end=34)):
        assert plan(**kw) == INV, kw

    def append(ts=16, slots=16):
        return lib.hstu_cache_append(1, 16, 128, 16, 128, ts, slots, 4, 2, 64, 64, 16, 2048, 128, 16, 2048,
                                     128, 16, 16, 4, 16, None)
    for kw in (dict(ts=20), dict(slots=20)):
        assert append(**kw) == INV, kw
    for kw in (dict(off=20), dict(ts=20), dict(table=18), dict(ctx=17), dict(par=18), dict(pos=18),
               dict(tb=18), dict(dt=0, q=18), dict(dt=0, kc=18), dict(dt=0, vc=17), dict(dt=0, out=18)):
        assert cached(lib, **kw) == INV, kw
