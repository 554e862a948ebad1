"""Host-side checks of the beam search calls that need no GPU: bad arguments
are refused before the device is touched (fake pointers), empty calls are
no-ops, workspaces are sized, and the Python extension refuses what is not a
device tensor."""
import ctypes
import os
import re

import pytest
import torch

from ring_collectives_amd import _native as N
from ring_collectives_amd import attention as A
from ring_collectives_amd import search as S

L = N.lib()
WS = (0x100000, 1 << 40)


def ptrs(P, base, step=0x1000000):
    return N.ptr_array([base + r * step for r in range(P)])[0]


def beam(P=2, N_=3, W=4, K=4, width=128, vocab=200, stride=128, end=-1, dt=N.RING_F32, ws=WS, **kw):
    d = dict(x=ptrs(max(P, 1), 0x10000000), scores=0x1000, done=None, parents=0x2000, tokens=0x3000, after=0x4000, done_after=None)
    d.update(kw)
    return L.beam_select(*[d[k] for k in ("x", "scores", "done", "parents", "tokens", "after", "done_after")], P, N_, W, K, width,
                         vocab, stride, end, dt, *ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(P=0), N.RING_EINVAL), (dict(P=65), N.RING_EINVAL), (dict(N_=-1), N.RING_EINVAL), (dict(W=0), N.RING_EINVAL),
    (dict(K=0), N.RING_EINVAL), (dict(W=65), N.RING_EUNSUPPORTED), (dict(K=65), N.RING_EUNSUPPORTED),
    (dict(width=0), N.RING_EINVAL), (dict(vocab=0), N.RING_EINVAL), (dict(vocab=257), N.RING_EINVAL),
    (dict(stride=120), N.RING_EINVAL), (dict(stride=130), N.RING_EINVAL), (dict(stride=1 << 31), N.RING_EINVAL),
    (dict(dt=N.RING_I32), N.RING_EUNSUPPORTED), (dict(end=-2), N.RING_EINVAL), (dict(end=200), N.RING_EINVAL),
    (dict(done=0x5000), N.RING_EINVAL), (dict(done_after=0x5000), N.RING_EINVAL),
    (dict(done=0x5000, done_after=0x6000), N.RING_EINVAL), (dict(x=None), N.RING_EINVAL), (dict(x=ptrs(2, 0)), N.RING_EINVAL),
    (dict(x=ptrs(2, 0x10000008)), N.RING_EINVAL), (dict(scores=None), N.RING_EINVAL), (dict(scores=0x1002), N.RING_EINVAL),
    (dict(parents=None), N.RING_EINVAL), (dict(tokens=0x3001), N.RING_EINVAL), (dict(after=None), N.RING_EINVAL),
    (dict(ws=(None, 1 << 40)), N.RING_EWORKSPACE), (dict(ws=(0x100000, 256)), N.RING_EWORKSPACE),
    (dict(ws=(0x100080, 1 << 40)), N.RING_EWORKSPACE), (dict(N_=1 << 23), N.RING_EUNSUPPORTED),
    (dict(width=(1 << 28) + 8, stride=(1 << 28) + 8), N.RING_EUNSUPPORTED), (dict(N_=0), N.RING_OK)])
def test_beam_refusals(kw, code):
    assert beam(**kw) == code


def test_beam_workspace():
    f = L.beam_select_workspace_bytes
    assert f(2, 3, 4, 4, 128) >= 256 + 2 * 3 * 4 * 5 * 8
    assert f(0, 3, 4, 4, 128) == 0 == f(2, 3, 65, 4, 128) == f(2, 3, 4, 0, 128) == f(2, 3, 4, 4, 0)


def fork(B=4, B2=4, group=2, n_free=20, W=3, page=16, pages=30, ws=WS, **kw):
    d = dict(table=0x1000, lens=0x2000, parents=0x3000, keep=None, free=0x4000, used=0x5000, table2=0x6000, lens2=0x7000,
             copies=0x8000, n=0x9000, shared=0xA000, used2=0xB000)
    d.update(kw)
    return L.kv_fork(*[d[k] for k in ("table", "lens", "parents", "keep", "free", "used", "table2", "lens2", "copies", "n", "shared",
                                      "used2")], B, B2, group, n_free, W, page, pages, *ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), N.RING_EINVAL), (dict(B2=-2), N.RING_EINVAL), (dict(group=0), N.RING_EINVAL), (dict(group=3), N.RING_EINVAL),
    (dict(n_free=-1), N.RING_EINVAL), (dict(W=-1), N.RING_EINVAL), (dict(pages=-1), N.RING_EINVAL), (dict(page=0), N.RING_EINVAL),
    (dict(page=24), N.RING_EINVAL), (dict(page=1 << 21), N.RING_EINVAL), (dict(B=8193), N.RING_EUNSUPPORTED),
    (dict(B2=8194), N.RING_EUNSUPPORTED), (dict(W=1 << 27), N.RING_EUNSUPPORTED), (dict(table=None), N.RING_EINVAL),
    # counts that a loop's step would carry past 31 bits
    (dict(W=(1 << 27) - 1), N.RING_EUNSUPPORTED), (dict(W=(1 << 31) - (1 << 20), page=1), N.RING_EUNSUPPORTED),
    (dict(pages=(1 << 31) - (1 << 20)), N.RING_EUNSUPPORTED), (dict(lens=None), N.RING_EINVAL), (dict(parents=None), N.RING_EINVAL), (dict(free=None), N.RING_EINVAL),
    (dict(used=None), N.RING_EINVAL), (dict(table2=None), N.RING_EINVAL), (dict(lens2=None), N.RING_EINVAL),
    (dict(copies=None), N.RING_EINVAL), (dict(n=None), N.RING_EINVAL), (dict(used2=None), N.RING_EINVAL),
    (dict(used2=0x5000), N.RING_EINVAL), (dict(lens2=0x2000), N.RING_EINVAL), (dict(table2=0x1000), N.RING_EINVAL),
    (dict(shared=0xA002), N.RING_EINVAL), (dict(keep=0xC001), N.RING_EINVAL), (dict(copies=0x8002), N.RING_EINVAL),
    (dict(ws=(None, 1 << 40)), N.RING_EWORKSPACE), (dict(ws=(0x100000, 256)), N.RING_EWORKSPACE),
    (dict(ws=(0x100010, 1 << 40)), N.RING_EWORKSPACE)])
def test_fork_refusals(kw, code):
    assert fork(**kw) == code


def compact(B=4, n=20, W=3, page=16, first=0, ws=WS, **kw):
    d = dict(table=0x1000, lens=0x2000, table2=0x6000, free=0x4000, copies=0x8000, nc=0x9000, used2=0xB000)
    d.update(kw)
    return L.kv_compact(*[d[k] for k in ("table", "lens", "table2", "free", "copies", "nc", "used2")], B, n, W, page, first, *ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), N.RING_EINVAL), (dict(n=-1), N.RING_EINVAL), (dict(W=-1), N.RING_EINVAL), (dict(first=-1), N.RING_EINVAL),
    (dict(page=3), N.RING_EINVAL), (dict(B=8193), N.RING_EUNSUPPORTED), (dict(W=1 << 27), N.RING_EUNSUPPORTED),
    (dict(W=(1 << 31) - (1 << 20), page=1), N.RING_EUNSUPPORTED), (dict(n=(1 << 31) - (1 << 20)), N.RING_EUNSUPPORTED),
    (dict(first=(1 << 31) - 10), N.RING_EUNSUPPORTED), (dict(table=None), N.RING_EINVAL), (dict(lens=None), N.RING_EINVAL),
    (dict(table2=None), N.RING_EINVAL), (dict(table2=0x1000), N.RING_EINVAL), (dict(free=None), N.RING_EINVAL),
    (dict(copies=None), N.RING_EINVAL), (dict(nc=None), N.RING_EINVAL), (dict(used2=None), N.RING_EINVAL),
    (dict(used2=0xB001), N.RING_EINVAL), (dict(ws=(None, 0)), N.RING_EWORKSPACE), (dict(ws=(0x100000, 300)), N.RING_EWORKSPACE)])
def test_compact_refusals(kw, code):
    assert compact(**kw) == code


def copy(n=2, cap=5, pages=30, nbytes=4096, **kw):
    d = dict(caches=ptrs(max(n, 1), 0x10000000), copies=0x8000, nc=0x9000)
    d.update(kw)
    return L.kv_copy_pages(d["caches"], d["copies"], d["nc"], n, cap, pages, nbytes, None)


@pytest.mark.parametrize("kw,code", [
    (dict(n=0), N.RING_EINVAL), (dict(n=129), N.RING_EINVAL), (dict(cap=-1), N.RING_EINVAL), (dict(pages=-1), N.RING_EINVAL),
    (dict(nbytes=-16), N.RING_EINVAL), (dict(nbytes=4100), N.RING_EINVAL), (dict(nbytes=1 << 31), N.RING_EUNSUPPORTED),
    (dict(caches=None), N.RING_EINVAL), (dict(caches=ptrs(2, 0)), N.RING_EINVAL), (dict(caches=ptrs(2, 0x10000008)), N.RING_EINVAL),
    (dict(copies=None), N.RING_EINVAL), (dict(nc=None), N.RING_EINVAL), (dict(nc=0x9001), N.RING_EINVAL),
    (dict(cap=0, copies=None), N.RING_OK), (dict(pages=0), N.RING_OK), (dict(nbytes=0), N.RING_OK)])
def test_copy_refusals(kw, code):
    assert copy(**kw) == code


def kv4(f, P=2, T=3, Hkv=2, D=64, page=16, pages=8, ks=128, vs=128, **kw):
    d = dict(k=ptrs(max(P, 1), 0x10000000), v=ptrs(max(P, 1), 0x20000000), cache=ptrs(max(P, 1), 0x30000000), slots=0x1000)
    d.update(kw)
    order = ("k", "v", "cache", "slots") if f is L.tp_kv4_write else ("cache", "slots", "k", "v")
    return f(*[d[k] for k in order], P, T, Hkv, D, page, pages, ks, vs, None)


@pytest.mark.parametrize("kw,code", [
    (dict(P=0), N.RING_EINVAL), (dict(P=65), N.RING_EINVAL), (dict(T=-1), N.RING_EINVAL), (dict(Hkv=0), N.RING_EINVAL),
    (dict(pages=-1), N.RING_EINVAL), (dict(D=96), N.RING_EUNSUPPORTED), (dict(page=8), N.RING_EUNSUPPORTED),
    (dict(page=48), N.RING_EUNSUPPORTED), (dict(page=1 << 17), N.RING_EUNSUPPORTED), (dict(pages=1 << 27), N.RING_EUNSUPPORTED),
    (dict(ks=120), N.RING_EINVAL), (dict(vs=132), N.RING_EINVAL), (dict(k=None), N.RING_EINVAL), (dict(v=ptrs(2, 0)), N.RING_EINVAL),
    (dict(cache=ptrs(2, 0)), N.RING_EINVAL), (dict(cache=ptrs(2, 0x30000004)), N.RING_EINVAL), (dict(slots=None), N.RING_EINVAL),
    (dict(slots=0x1004), N.RING_EINVAL), (dict(k=ptrs(2, 0x10000002)), N.RING_EINVAL), (dict(T=0), N.RING_OK)])
@pytest.mark.parametrize("write", [True, False])
def test_kv4_refusals(kw, code, write):
    assert kv4(L.tp_kv4_write if write else L.tp_kv4_read, **kw) == code


def test_page_bytes():
    f = L.kv4_page_bytes
    assert f(2, 128, 16) == 2 * 16 * 136 and f(1, 64, 32) == 32 * 68
    assert f(0, 128, 16) == 0 == f(2, 96, 16) == f(2, 128, 8) == f(2, 128, 24)


def decode(P=2, B=4, group=2, Hq=4, Hkv=2, D=64, W=4, page=16, pages=20, qs=256, os=256, scale=0.1, ws=WS, **kw):
    d = dict(q=ptrs(max(P, 1), 0x10000000), cache=ptrs(max(P, 1), 0x20000000), o=ptrs(max(P, 1), 0x40000000), table=0x1000,
             lens=0x2000, shared=0x3000)
    d.update(kw)
    return L.tp_attention_decode_kv4(*[d[k] for k in ("q", "cache", "o", "table", "lens", "shared")], P, B, group, Hq, Hkv, D, W, page,
                                     pages, qs, os, scale, *ws, None)


@pytest.mark.parametrize("kw,code", [
    (dict(P=0), N.RING_EINVAL), (dict(B=-1), N.RING_EINVAL), (dict(group=0), N.RING_EINVAL), (dict(group=3), N.RING_EINVAL),
    (dict(Hkv=0), N.RING_EINVAL), (dict(W=-1), N.RING_EINVAL), (dict(pages=-1), N.RING_EINVAL), (dict(page=12), N.RING_EUNSUPPORTED),
    (dict(page=8), N.RING_EUNSUPPORTED), (dict(scale=0.0), N.RING_EINVAL), (dict(scale=float("nan")), N.RING_EINVAL),
    (dict(scale=3e38), N.RING_EINVAL), (dict(D=32), N.RING_EUNSUPPORTED), (dict(Hq=3), N.RING_EUNSUPPORTED),
    (dict(W=1 << 27), N.RING_EUNSUPPORTED), (dict(pages=1 << 27), N.RING_EUNSUPPORTED), (dict(B=8194), N.RING_EUNSUPPORTED),
    (dict(qs=248), N.RING_EINVAL), (dict(os=128), N.RING_EINVAL), (dict(q=None), N.RING_EINVAL), (dict(cache=ptrs(2, 0)), N.RING_EINVAL),
    (dict(o=ptrs(2, 0x40000008)), N.RING_EINVAL), (dict(table=None), N.RING_EINVAL), (dict(lens=None), N.RING_EINVAL),
    (dict(lens=0x2001), N.RING_EINVAL), (dict(shared=0x3002), N.RING_EINVAL), (dict(ws=(None, 0)), N.RING_EWORKSPACE),
    (dict(ws=(0x100000, 256)), N.RING_EWORKSPACE), (dict(B=0), N.RING_OK)])
def test_decode_refusals(kw, code):
    assert decode(**kw) == code


def test_decode_workspace_grows_with_the_batch():
    f = L.tp_attention_decode_kv4_workspace_bytes
    sizes = [f(4, b, 4, 8, 2, 128) for b in range(0, 600, 4)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])) and sizes[0] >= 256
    assert f(4, 8, 3, 8, 2, 128) == 0 == f(4, 8, 4, 8, 3, 128)


def test_binding_refuses_what_is_not_a_device_tensor():
    c = A._binding()
    i = torch.zeros(2, dtype=torch.int32)
    x = [torch.zeros(2, 2, 64, dtype=torch.bfloat16)]
    with pytest.raises(ValueError, match="current device"):
        c.beam_select([torch.zeros(2, 128)], torch.zeros(1, 2), i[None], i[None], torch.zeros(1, 2), 100, None, None, -1, i, 0, 0)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        c.beam_select([torch.zeros(2, 128).half()], torch.zeros(1, 2), i[None], i[None], torch.zeros(1, 2), 100, None, None, -1, i, 0, 0)
    with pytest.raises(ValueError, match="current device"):
        c.kv_fork(i[None], i, i, None, i, i, i[None], i, i[None], i, None, i, 1, 16, 4, i, 0, 0)
    with pytest.raises(ValueError, match="dimensions|rows"):
        c.kv_fork(i, i, i, None, i, i, i[None], i, i[None], i, None, i, 1, 16, 4, i, 0, 0)
    with pytest.raises(ValueError, match="current device"):
        c.kv_compact(i[None], i, i[None], i, i[None], i, i, 16, 0, i, 0, 0)
    with pytest.raises(ValueError, match="current device"):
        c.kv_copy_pages(x, i[None], i, 2, 0, 0)
    with pytest.raises(ValueError, match="current device"):
        c.tp_kv4_write(x, x, x, i, 16, 0, 0)
    with pytest.raises(TypeError, match="arguments"):
        c.tp_kv4_read(x, x)
    with pytest.raises(ValueError, match="current device"):
        c.tp_attention_decode_kv4(x, x, x, i[None], i, 16, None, 1, 1.0, i, 0, 0)
    with pytest.raises(ValueError, match="not supported"):
        S.kv4_cache(4, 2, 96, 16, device="cpu")


def test_ctypes_signatures_have_the_headers_parameter_counts():
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "tp_search.h")).read()
    src = re.sub(r"/\*.*?\*/", " ", src, flags=re.S)
    src = re.sub(r"#[^\n]*", " ", src)
    found = re.findall(r"\b([a-z_]\w*)\s*\(([^;{}]*)\)\s*;", src)
    assert len(found) == 12
    for name, args in found:
        assert len(N.SIGNATURES[name][1]) == len(args.split(",")), name
        assert isinstance(getattr(L, name), ctypes._CFuncPtr)
