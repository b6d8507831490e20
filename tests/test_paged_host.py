"""Refusals of the paged calls, before anything is launched (no GPU needed),
and the binding's own checks."""
import ctypes

import pytest
import torch

import linear_attention_serving_gb300 as kda
from linear_attention_serving_gb300 import paged

FAKE = ctypes.c_void_p(1 << 20)  # aligned dummy address; never dereferenced on these paths
ODD = ctypes.c_void_p((1 << 20) + 4)
OTHER = ctypes.c_void_p(1 << 21)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


def tables(**kw):
    a = dict(new=FAKE, ctx=FAKE, n=2, T=5, table=FAKE, width=4, free=FAKE, n_free=3, head=FAKE, head_next=OTHER, ps=16,
             pages=8, slots=FAKE, pos=FAKE, cu=FAKE, kv=FAKE, err=None, s=None)
    a.update(kw)
    return paged._lib().kda_paged_tables(*a.values())


def append(**kw):
    a = dict(k=FAKE, v=FAKE, slots=FAKE, T=5, hkv=2, D=128, dt=0, cdt=0, ks=None, vs=None, kc=FAKE, vc=FAKE, pages=8, ps=16,
             stride=2 * 16 * 128, err=None, s=None)
    a.update(kw)
    return paged._lib().kda_paged_append(*a.values())


def attn(**kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, cu=FAKE, kv=FAKE, n=2, T=5, max_q=3, hq=4, hkv=2, D=128, dt=0, cdt=0,
             ks=None, vs=None, pages=8, ps=16, stride=2 * 16 * 128, width=4, scale=0.1, window=0, o=FAKE, lse=None, ws=FAKE,
             wsb=0, err=None, s=None)
    a.update(kw)
    return paged._lib().kda_paged_attn(*a.values())


@pytest.mark.parametrize("kw,rc", [
    (dict(n=0), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(width=0), INVALID),
    (dict(n_free=-1), INVALID), (dict(pages=0), INVALID), (dict(ps=8), INVALID), (dict(ps=24), UNSUPPORTED),
    (dict(n=16385), UNSUPPORTED), (dict(width=1 << 27), INVALID), (dict(new=None), INVALID), (dict(ctx=None), INVALID),
    (dict(table=None), INVALID), (dict(free=None), INVALID), (dict(head=None), INVALID), (dict(head_next=None), INVALID),
    (dict(head_next=FAKE), INVALID), (dict(slots=None), INVALID), (dict(slots=ODD), INVALID), (dict(pos=ODD), INVALID),
    (dict(cu=None), INVALID), (dict(kv=None), INVALID)])
def test_tables_refusals(kw, rc):
    assert tables(**kw) == rc


@pytest.mark.parametrize("name", ["new", "ctx", "free", "head"])
@pytest.mark.parametrize("out", ["table", "head_next", "slots", "pos", "cu", "kv"])
def test_tables_refuses_an_input_as_output(out, name):
    """Blocks read the lengths and pages while others write already."""
    apart = {k: ctypes.c_void_p((i + 1) << 20) for i, k in enumerate(
        ["new", "ctx", "free", "head", "table", "head_next", "slots", "pos", "cu", "kv"])}
    assert tables(**{**apart, out: apart[name]}) == INVALID


@pytest.mark.parametrize("kw,rc", [
    (dict(D=64), UNSUPPORTED), (dict(dt=2), INVALID), (dict(cdt=7), INVALID), (dict(cdt=1), UNSUPPORTED),
    (dict(dt=1, cdt=2, ks=FAKE, vs=FAKE), UNSUPPORTED), (dict(cdt=2), INVALID), (dict(ks=FAKE, vs=FAKE), INVALID),
    (dict(cdt=2, ks=FAKE), INVALID), (dict(hkv=0), INVALID), (dict(pages=0), INVALID), (dict(ps=0), INVALID),
    (dict(ps=40), UNSUPPORTED), (dict(stride=4095), INVALID), (dict(stride=4097), INVALID), (dict(stride=1 << 40), INVALID),
    (dict(kc=None), INVALID), (dict(vc=ODD), INVALID), (dict(k=None), INVALID), (dict(v=ODD), INVALID), (dict(slots=None), INVALID),
    (dict(T=-1), INVALID), (dict(T=0), 0)])
def test_append_refusals(kw, rc):
    assert append(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(D=256), UNSUPPORTED), (dict(hq=5), INVALID), (dict(hq=1), INVALID), (dict(n=0), INVALID), (dict(width=0), INVALID),
    (dict(max_q=-1), INVALID), (dict(window=-1), INVALID), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID),
    (dict(width=1 << 27), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(table=None), INVALID), (dict(cu=None), INVALID), (dict(kv=None), INVALID),
    (dict(q=None), INVALID), (dict(o=None), INVALID), (dict(q=ODD), INVALID), (dict(o=ODD), INVALID), (dict(), WORKSPACE),
    (dict(ws=None, wsb=1 << 40), WORKSPACE), (dict(ws=ODD, wsb=1 << 40), WORKSPACE), (dict(T=0, wsb=1 << 40), 0)])
def test_attn_refusals(kw, rc):
    assert attn(**kw) == rc


def test_workspace_size():
    f = kda.paged_attn_workspace_size
    assert 0 < f(1, 1, 8, 8) < f(1, 1, 64, 1)
    assert f(-1, 1, 8, 8) == 0 and f(1, 0, 8, 8) == 0 and f(1, 1, 8, 3) == 0 and f(1, 1, 2, 4) == 0


@pytest.mark.parametrize("fails", [RuntimeError("g++ failed"), PermissionError("read-only"), ImportError("headers")])
def test_binding_without_the_compiled_way(fails, monkeypatch):
    """The plain binding stands alone, and says once that it does."""
    def no(*a, **k):
        raise fails

    monkeypatch.setattr(paged._build, "build_fast", no)
    monkeypatch.setattr(paged, "_declared", None)
    for f in ("tables", "append", "attn"):
        monkeypatch.setattr(paged, "_fast_" + f, paged._not_loaded)
    with pytest.warns(RuntimeWarning, match="plain binding") as said:
        assert kda.paged_attn_workspace_size(1, 1, 8, 8) > 0
        assert tables(n=0) == INVALID
        test_binding_refuses_host_tensors()
    assert len(said) == 1


def test_binding_refuses_host_tensors():
    z = torch.zeros
    i = z(2, dtype=torch.int32)
    c = z(4, 2, 16, 128, dtype=torch.bfloat16)
    x = z(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(kda.KDAError, match="CUDA"):
        kda.paged_tables(i, i, z(2, 4, dtype=torch.int32), i, z(1, dtype=torch.int32), 0, 16, 8)
    with pytest.raises(kda.KDAError, match="CUDA"):
        kda.paged_append(x, x, z(3, dtype=torch.int64), c, c)
    with pytest.raises(kda.KDAError, match="CUDA"):
        kda.paged_attn(x, c, c, z(1, 4, dtype=torch.int32), i, z(1, dtype=torch.int32))
