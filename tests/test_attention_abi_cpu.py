"""Host-side checks of the attention calls that need no GPU: bad arguments are
refused before the device is touched (fake pointers), empty calls are no-ops,
workspaces are sized, and the Python extension refuses what is not a device
tensor."""
import ctypes

import pytest
import torch

from ring_collectives_amd import _native as N
from ring_collectives_amd import attention as A

L = N.lib()
WS = (0x100000, 1 << 40)


def ptrs(P, base, step=0x1000000):
    return N.ptr_array([base + r * step for r in range(P)])[0]


def plan(**kw):
    d = dict(lengths=0x1000, new=0x2000, free=0x3000, used=0x4000, table=0x5000, after=0x6000, cu=0x7000, pos=0x8000,
             slots=0x9000, ua=0xA000, B=4, n_free=8, stride=4, page=16, cap=10, prefix=0)
    d.update(kw)
    return L.kv_plan(*[d[k] for k in ("lengths", "new", "free", "used", "table", "after", "cu", "pos", "slots", "ua", "B",
                                      "n_free", "stride", "page", "cap", "prefix")], None)


@pytest.mark.parametrize("kw", [dict(B=-1), dict(n_free=-1), dict(stride=-1), dict(cap=-1), dict(prefix=-1), dict(page=0),
                                dict(page=24), dict(page=1 << 21), dict(lengths=None), dict(new=None), dict(used=None),
                                dict(free=None), dict(table=None), dict(after=None), dict(cu=None), dict(pos=None),
                                dict(slots=None), dict(ua=None), dict(slots=0x9004), dict(pos=0x8002), dict(ua=0x4000),
                                dict(after=0x1000), dict(after=0x2000)])
def test_plan_refusals(kw):
    assert plan(**kw) == N.RING_EINVAL


def test_plan_limits():
    assert plan(B=0) == N.RING_OK
    assert plan(B=8193) == N.RING_EUNSUPPORTED


def rope(P=2, T=3, Hq=4, Hkv=2, D=64, rot=64, rows=100, crows=50, stride=512, eps=1e-6, dt=N.RING_BF16, **kw):
    d = dict(x=ptrs(max(P, 1), 0x10000000), gq=ptrs(max(P, 1), 0x1000, 0x400), gk=ptrs(max(P, 1), 0x9000, 0x400), cs=0x20000,
             pos=0x30000, q=ptrs(max(P, 1), 0x30000000), k=ptrs(max(P, 1), 0x40000000), v=ptrs(max(P, 1), 0x50000000),
             kc=None, vc=None, slots=None)
    d.update(kw)
    return L.tp_qk_norm_rope(*[d[k] for k in ("x", "gq", "gk", "cs", "pos", "q", "k", "v", "kc", "vc", "slots")], P, T, Hq, Hkv,
                             D, rot, rows, crows, stride, eps, dt, None)


@pytest.mark.parametrize("kw,code", [
    (dict(P=0), N.RING_EINVAL), (dict(P=65), N.RING_EINVAL), (dict(T=-1), N.RING_EINVAL), (dict(Hq=0), N.RING_EINVAL),
    (dict(eps=-1.0), N.RING_EINVAL), (dict(eps=float("nan")), N.RING_EINVAL), (dict(dt=N.RING_I32), N.RING_EUNSUPPORTED),
    (dict(D=96), N.RING_EUNSUPPORTED), (dict(Hq=3), N.RING_EUNSUPPORTED), (dict(rot=24), N.RING_EINVAL),
    (dict(rot=80), N.RING_EINVAL), (dict(rot=-16), N.RING_EINVAL), (dict(stride=511), N.RING_EINVAL),
    (dict(stride=516), N.RING_EINVAL), (dict(stride=1 << 21), N.RING_EINVAL), (dict(k=None), N.RING_EINVAL),
    (dict(kc=ptrs(2, 0x60000000)), N.RING_EINVAL), (dict(gq=None), N.RING_EINVAL), (dict(pos=None), N.RING_EINVAL),
    (dict(cs=None), N.RING_EINVAL), (dict(cs=0x20004), N.RING_EINVAL), (dict(q=None), N.RING_EINVAL),
    (dict(x=ptrs(2, 0x10000008)), N.RING_EINVAL), (dict(q=ptrs(2, 0)), N.RING_EINVAL),
    (dict(Hq=1 << 20, Hkv=1 << 20, stride=(1 << 21) - 8), N.RING_EUNSUPPORTED)])
def test_rope_refusals(kw, code):
    assert rope(**kw) == code


def test_rope_grad_refusals():
    a = [ptrs(2, 0x10000000 * (i + 1)) for i in range(4)]
    g = [ptrs(2, 0x1000 * (i + 1), 0x400) for i in range(2)]

    def call(T=3, gains=True, dg=True, ws=WS, dt=N.RING_F32, D=64):
        return L.tp_qk_norm_rope_grad(*a, *(g if gains else (None, None)), 0x20000, 0x30000, ptrs(2, 0x70000000),
                                      *(g if dg else (None, None)), 2, T, 4, 2, D, D, 100, 8 * D, 1e-6, dt, *ws, None)

    assert call(dg=False) == N.RING_EINVAL
    assert call(dt=7) == N.RING_EUNSUPPORTED
    assert call(D=32) == N.RING_EUNSUPPORTED
    assert call(ws=(0x100000, 256)) == N.RING_EWORKSPACE
    assert call(ws=(0x100010, 1 << 40)) == N.RING_EWORKSPACE
    assert call(ws=(None, 1 << 40)) == N.RING_EWORKSPACE
    assert call(T=0, gains=False) == N.RING_OK
    assert L.tp_qk_norm_rope_grad_workspace_bytes(2, 64) > 256
    assert L.tp_qk_norm_rope_grad_workspace_bytes(0, 64) == 0 == L.tp_qk_norm_rope_grad_workspace_bytes(2, 48)


def attn(P=2, B=3, Tq=10, Tk=10, Hq=4, Hkv=2, D=64, qs=256, ks=128, vs=128, os=256, scale=0.1, **kw):
    d = dict(q=ptrs(max(P, 1), 0x10000000), k=ptrs(max(P, 1), 0x20000000), v=ptrs(max(P, 1), 0x30000000),
             o=ptrs(max(P, 1), 0x40000000), lse=None, cq=0x1000, ck=0x2000)
    d.update(kw)
    return L.tp_attention(*[d[k] for k in ("q", "k", "v", "o", "lse", "cq", "ck")], P, B, Tq, Tk, Hq, Hkv, D, qs, ks, vs, os, 1,
                          scale, None)


BAD_ATTN = [
    (dict(P=0), N.RING_EINVAL), (dict(P=65), N.RING_EINVAL), (dict(B=-1), N.RING_EINVAL), (dict(Tq=-1), N.RING_EINVAL),
    (dict(Tk=-1), N.RING_EINVAL), (dict(Hkv=0), N.RING_EINVAL), (dict(scale=0.0), N.RING_EINVAL),
    (dict(scale=-1.0), N.RING_EINVAL), (dict(scale=float("inf")), N.RING_EINVAL), (dict(scale=float("nan")), N.RING_EINVAL),
    (dict(D=80), N.RING_EUNSUPPORTED), (dict(D=256, qs=1024, ks=512, vs=512, os=1024), N.RING_EUNSUPPORTED),
    (dict(Hq=5, qs=320, os=320), N.RING_EUNSUPPORTED), (dict(qs=248), N.RING_EINVAL), (dict(ks=132), N.RING_EINVAL),
    (dict(vs=1 << 21), N.RING_EINVAL), (dict(os=0), N.RING_EINVAL), (dict(q=None), N.RING_EINVAL), (dict(k=None), N.RING_EINVAL),
    (dict(o=None), N.RING_EINVAL), (dict(cq=None), N.RING_EINVAL), (dict(ck=None), N.RING_EINVAL),
    (dict(q=ptrs(2, 0x10000008)), N.RING_EINVAL), (dict(v=ptrs(2, 0)), N.RING_EINVAL), (dict(o=ptrs(2, 0x40000002)), N.RING_EINVAL),
    (dict(lse=ptrs(2, 0x50000002)), N.RING_EINVAL), (dict(P=8, Tq=(1 << 31) - 1, Hq=64, qs=4096, os=4096), N.RING_EUNSUPPORTED)]


@pytest.mark.parametrize("kw,code", BAD_ATTN)
def test_attention_refusals(kw, code):
    assert attn(**kw) == code


def test_attention_empty_calls():
    assert attn(Tq=0) == N.RING_OK
    assert attn(B=0) == N.RING_OK


def test_attention_grad_refusals():
    a = [ptrs(2, 0x10000000 * (i + 1)) for i in range(9)]

    def call(i=None, ws=WS, B=3, Tq=10, Tk=10, D=64, bad=None, scale=0.1):
        p = list(a)
        if i is not None:
            p[i] = bad
        s = [4 * D, 2 * D, 2 * D, 4 * D, 4 * D, 4 * D, 2 * D, 2 * D]
        return L.tp_attention_grad(*p, 0x1000, 0x2000, 2, B, Tq, Tk, 4, 2, D, *s, 1, scale, *ws, None)

    for i in range(9):
        assert call(i) == N.RING_EINVAL
        assert call(i, bad=ptrs(2, 0)) == N.RING_EINVAL
    assert call(0, bad=ptrs(2, 0x10000008)) == N.RING_EINVAL
    assert call(D=48) == N.RING_EUNSUPPORTED
    assert call(scale=0.0) == N.RING_EINVAL
    assert call(ws=(0x100000, 256)) == N.RING_EWORKSPACE
    assert call(ws=(0x100040, 1 << 40)) == N.RING_EWORKSPACE
    assert call(B=0) == N.RING_OK == call(Tq=0, Tk=0)
    assert L.tp_attention_grad_workspace_bytes(2, 10, 4) >= 256 + 2 * 10 * 4 * 8
    assert L.tp_attention_grad_workspace_bytes(65, 10, 4) == 0


def decode(P=2, B=3, Hq=4, Hkv=2, D=64, W=4, page=16, pages=20, prefix=0, qs=256, os=256, scale=0.1, ws=WS, **kw):
    d = dict(q=ptrs(max(P, 1), 0x10000000), k=ptrs(max(P, 1), 0x20000000), v=ptrs(max(P, 1), 0x30000000),
             o=ptrs(max(P, 1), 0x40000000), table=0x1000, lens=0x2000, pp=0x3000)
    d.update(kw)
    return L.tp_attention_decode(*[d[k] for k in ("q", "k", "v", "o", "table", "lens", "pp")], P, B, Hq, Hkv, D, W, page, pages,
                                 prefix, qs, os, scale, *ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(P=0), N.RING_EINVAL), (dict(B=-1), N.RING_EINVAL), (dict(Hkv=0), N.RING_EINVAL), (dict(W=-1), N.RING_EINVAL),
    (dict(pages=-1), N.RING_EINVAL), (dict(prefix=-1), N.RING_EINVAL), (dict(page=0), N.RING_EINVAL),
    (dict(page=12), N.RING_EINVAL), (dict(scale=0.0), N.RING_EINVAL), (dict(D=32), N.RING_EUNSUPPORTED),
    (dict(Hq=3), N.RING_EUNSUPPORTED), (dict(W=1 << 28), N.RING_EUNSUPPORTED), (dict(pages=1 << 28), N.RING_EUNSUPPORTED),
    (dict(B=(1 << 20) + 1), N.RING_EUNSUPPORTED), (dict(qs=255), N.RING_EINVAL), (dict(os=128), N.RING_EINVAL),
    (dict(q=None), N.RING_EINVAL), (dict(k=ptrs(2, 0)), N.RING_EINVAL), (dict(v=ptrs(2, 0x30000008)), N.RING_EINVAL),
    (dict(table=None), N.RING_EINVAL), (dict(lens=None), N.RING_EINVAL), (dict(lens=0x2001), N.RING_EINVAL),
    (dict(prefix=5, pp=None), N.RING_EINVAL), (dict(ws=(None, 0)), N.RING_EWORKSPACE),
    (dict(ws=(0x100000, 255)), N.RING_EWORKSPACE), (dict(prefix=5, ws=(0x100000, 256)), N.RING_EWORKSPACE)])
def test_decode_refusals(kw, code):
    assert decode(**kw) == code


def test_decode_empty_and_workspace():
    assert decode(B=0) == N.RING_OK
    f = L.tp_attention_decode_workspace_bytes
    assert f(2, 3, 4, 2, 64, 4, 16, 0) == 256                 # short caches: one part, nothing to join
    assert f(2, 3, 4, 2, 64, 4, 16, 100) >= 256 + 2 * 2 * 3 * 4 * 66 * 4
    assert f(1, 1, 1, 1, 128, 4096, 16, 0) > f(1, 1, 1, 1, 128, 64, 16, 0)
    assert f(0, 3, 4, 2, 64, 4, 16, 0) == 0 == f(2, 3, 4, 2, 64, 4, 24, 0)


def test_binding_refuses_what_is_not_a_device_tensor():
    c = A._binding()
    x = [torch.zeros(2, 2, 64, dtype=torch.bfloat16)]
    cu = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="current device"):
        c.tp_attention(x, x, x, x, cu, cu, None, 1, 1.0, 0, 0)
    with pytest.raises(TypeError, match="torch tensor"):
        c.tp_attention([1], x, x, x, cu, cu, None, 1, 1.0, 0, 0)
    with pytest.raises(TypeError, match="one tensor per rank"):
        c.tp_attention(5, x, x, x, cu, cu, None, 1, 1.0, 0, 0)
    with pytest.raises(ValueError, match="rank buffers"):
        c.tp_attention([], x, x, x, cu, cu, None, 1, 1.0, 0, 0)
    with pytest.raises(ValueError, match="dimensions"):
        c.tp_attention([x[0][0]], x, x, x, cu, cu, None, 1, 1.0, 0, 0)
    with pytest.raises(TypeError, match="arguments"):
        c.tp_attention(x, x, x)
    with pytest.raises(ValueError, match="current device"):
        c.kv_plan(cu, cu, cu, cu, cu, cu, cu, cu, cu, cu, 16, 0, 0, 0)


def test_ctypes_signatures_have_the_headers_parameter_counts():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "tp_attention.h")).read()
    src = re.sub(r"/\*.*?\*/", " ", src, flags=re.S)
    src = re.sub(r"#[^\n]*", " ", src)
    found = re.findall(r"\b([a-z_]\w*)\s*\(([^;{}]*)\)\s*;", src)
    assert len(found) == 9
    for name, args in found:
        assert len(N.SIGNATURES[name][1]) == len(args.split(",")), name
        assert isinstance(getattr(L, name), ctypes._CFuncPtr)
