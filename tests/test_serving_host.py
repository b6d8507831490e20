"""Refusals of the rotary, sinks and verification calls before anything is launched (no GPU needed), the
frequencies, and the binding's own checks."""
import ctypes
import decimal
import math

import pytest
import torch

import linear_attention_serving_gb300 as kda
from linear_attention_serving_gb300 import paged
from serving_testutil import draft_inputs, frequencies_ref, verify_ref

FAKE = ctypes.c_void_p(1 << 20)  # aligned dummy addresses; never dereferenced on these paths
ODD = ctypes.c_void_p((1 << 20) + 4)
ADDR = [ctypes.c_void_p(i << 20) for i in range(2, 12)]
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


def rope(**kw):
    a = dict(q=ADDR[0], k=ADDR[1], pos=FAKE, freq=FAKE, amp=1.0, qw=None, kw=None, eps=1e-6, T=5, hq=4, hkv=2, D=128, rot=64, layout=0,
             dt=0, qs=512, ks=256, qo=ADDR[2], ko=ADDR[3], qos=512, kos=256, s=None)
    a.update(kw)
    return paged._lib().kda_qk_rope(*a.values())


def rope_append(**kw):
    a = dict(q=ADDR[0], k=ADDR[1], v=ADDR[2], pos=FAKE, slots=FAKE, freq=FAKE, amp=1.0, qw=None, kw=None, eps=1e-6, T=5, hq=4, hkv=2,
             D=128, rot=64, layout=0, dt=0, cdt=0, qs=512, ks=256, vs=256, qo=ADDR[3], qos=512, ksc=None, vsc=None, kc=FAKE, vc=FAKE,
             pages=8, ps=16, stride=2 * 16 * 128, err=None, s=None)
    a.update(kw)
    return paged._lib().kda_paged_rope_append(*a.values())


def sinks(**kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, table=FAKE, cu=FAKE, kv=FAKE, n=2, T=5, max_q=3, hq=4, hkv=2, D=128, dt=0, cdt=0,
             ks=None, vs=None, pages=8, ps=16, stride=2 * 16 * 128, width=4, scale=0.1, window=0, sinks=1, o=FAKE, lse=None, ws=FAKE,
             wsb=0, err=None, s=None)
    a.update(kw)
    return paged._lib().kda_paged_attn_sinks(*a.values())


def verify(**kw):
    a = dict(p=ADDR[0], q=ADDR[1], tokens=ADDR[2], u=ADDR[3], m=None, n=2, w=5, V=100, dt=1, ts=500, tr=100, ds=400, dr=100, acc=ADDR[4],
             out=ADDR[5], ws=None, wsb=0, err=None, s=None)
    a.update(kw)
    return paged._lib().kda_verify_drafts(*a.values())


SHARED = [
    (dict(D=64), UNSUPPORTED), (dict(dt=2), INVALID), (dict(layout=2), INVALID), (dict(layout=-1), INVALID), (dict(rot=-8), INVALID),
    (dict(rot=136), INVALID), (dict(rot=12), UNSUPPORTED), (dict(T=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(hq=0), INVALID),
    (dict(hkv=0), INVALID), (dict(hq=1 << 21, qs=1 << 30, qos=1 << 30), INVALID), (dict(eps=-1e-9), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(amp=float("inf")), INVALID), (dict(amp=float("nan")), INVALID), (dict(qs=511), INVALID),
    (dict(qs=516), INVALID), (dict(ks=128), INVALID), (dict(qos=256), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(pos=None), INVALID), (dict(freq=None), INVALID), (dict(qo=None), INVALID), (dict(q=ODD), INVALID), (dict(k=ODD), INVALID),
    (dict(qo=ODD), INVALID), (dict(qw=ODD), INVALID), (dict(kw=ODD), INVALID), (dict(freq=ODD), INVALID), (dict(T=0), 0),
    (dict(T=0, q=None, k=None, qo=None, pos=None), 0)]


@pytest.mark.parametrize("kw,rc", SHARED + [
    (dict(ko=None), INVALID), (dict(ko=ODD), INVALID), (dict(kos=128), INVALID), (dict(kos=260), INVALID), (dict(qo=ADDR[0], qos=520), INVALID),
    (dict(ko=ADDR[1], kos=264), INVALID), (dict(qo=ADDR[1]), INVALID), (dict(ko=ADDR[0]), INVALID), (dict(qo=ADDR[3]), INVALID)])
def test_rope_refusals(kw, rc):
    assert rope(**kw) == rc


@pytest.mark.parametrize("kw,rc", SHARED + [
    (dict(v=None), INVALID), (dict(v=ODD), INVALID), (dict(vs=128), INVALID), (dict(vs=260), INVALID), (dict(slots=None), INVALID),
    (dict(cdt=2), INVALID), (dict(cdt=1), UNSUPPORTED), (dict(dt=1, cdt=2, ksc=FAKE, vsc=FAKE), UNSUPPORTED), (dict(ksc=FAKE), INVALID),
    (dict(pages=0), INVALID), (dict(ps=24), UNSUPPORTED), (dict(stride=100), INVALID), (dict(kc=None), INVALID), (dict(vc=ODD), INVALID),
    (dict(qo=ADDR[0], qos=520), INVALID), (dict(qo=ADDR[1]), INVALID), (dict(qo=ADDR[2]), INVALID)])
def test_rope_append_refusals(kw, rc):
    assert rope_append(**kw) == rc


@pytest.mark.parametrize("kw,rc", [(dict(sinks=-1), INVALID), (dict(window=-1), INVALID), (dict(), WORKSPACE), (dict(T=0, wsb=1 << 40), 0)])
def test_sinks_refusals(kw, rc):
    assert sinks(**kw) == rc


@pytest.mark.parametrize("kw,rc", [
    (dict(dt=2), INVALID), (dict(n=0), INVALID), (dict(w=0), INVALID), (dict(V=0), INVALID), (dict(w=33), UNSUPPORTED),
    (dict(n=(1 << 24) + 1), UNSUPPORTED), (dict(V=2 ** 31 - 4096, tr=1 << 31, dr=1 << 31), UNSUPPORTED), (dict(p=None), INVALID), (dict(u=None), INVALID), (dict(acc=None), INVALID),
    (dict(out=None), INVALID), (dict(tokens=None), INVALID), (dict(p=ctypes.c_void_p((1 << 20) + 2)), INVALID),
    (dict(q=ctypes.c_void_p((1 << 20) + 1), dt=0), INVALID), (dict(tr=99), INVALID), (dict(dr=99), INVALID), (dict(ts=-1), INVALID),
    (dict(ds=-1), INVALID), (dict(acc=ADDR[5]), INVALID), (dict(out=ADDR[2]), INVALID), (dict(acc=ADDR[3]), INVALID),
    (dict(m=ADDR[4]), INVALID), (dict(out=ADDR[0]), INVALID), (dict(), WORKSPACE), (dict(ws=FAKE, wsb=15), WORKSPACE),
    (dict(ws=ODD, wsb=1 << 30), WORKSPACE)])
def test_verify_refusals(kw, rc):
    assert verify(**kw) == rc


@pytest.mark.parametrize("rot", [8, 64, 96, 128])
@pytest.mark.parametrize("kw", [dict(), dict(base=500000.0), dict(scaling="linear", factor=8.0), dict(scaling="ntk", factor=4.0),
                                dict(scaling="yarn", factor=16.0, original_len=4096),
                                dict(scaling="yarn", factor=40.0, original_len=8192, base=1e6, beta_fast=24.0, beta_slow=2.0)])
def test_frequencies(rot, kw):
    """In turns times 2^64; a power and a few products in 64 bits: a few times 2^-53 of the value, or half a unit."""
    freq, amp = kda.rope_frequencies(rot, **kw)
    ref, ref_amp = frequencies_ref(rot, **kw)
    assert freq.shape == (rot // 2,) and freq.dtype is torch.int64
    assert amp == pytest.approx(ref_amp, rel=2.0 ** -24)
    for a, b in zip(freq.tolist(), ref):
        turns = b / (2 * math.pi) * 2.0 ** 64
        assert abs(a - turns) <= 16 * 2.0 ** -53 * turns + 1


@pytest.mark.parametrize("kw", [dict(rot_dim=0), dict(rot_dim=136), dict(rot_dim=12), dict(base=1.0), dict(base=float("inf")),
                                dict(base=float("nan")), dict(scaling="other"), dict(scaling="linear", factor=0.5),
                                dict(scaling="linear", factor=float("inf")), dict(scaling="ntk", factor=1e300),
                                dict(scaling="yarn", factor=2.0), dict(scaling="yarn", factor=2.0, original_len=float("inf")),
                                dict(scaling="yarn", factor=2.0, original_len=100, beta_fast=1.0),
                                dict(scaling="yarn", factor=2.0, original_len=100, beta_slow=-1.0)])
def test_frequencies_refusals(kw):
    with pytest.raises(kda.KDAError):
        kda.rope_frequencies(**{"rot_dim": 64, **kw})


def test_verify_workspace_size():
    f = kda.verify_drafts_workspace_size
    assert 0 < f(1, 5, 32768) < f(500, 5, 32768) < f(500, 5, 65536) and f(500, 5, 65536, torch.bfloat16) > 0
    assert f(0, 5, 100) == f(5, 0, 100) == f(5, 33, 100) == f(5, 5, 0) == f(5, 5, 2 ** 31 - 4096) == f(500, 5, 100, torch.float16) == 0


def test_binding_refuses_host_tensors():
    z = torch.zeros
    q, k = z(3, 4, 128, dtype=torch.bfloat16), z(3, 2, 128, dtype=torch.bfloat16)
    c = z(4, 2, 16, 128, dtype=torch.bfloat16)
    i = z(3, dtype=torch.int32)
    freq, _ = kda.rope_frequencies(64)
    with pytest.raises(kda.KDAError, match="CUDA"):
        kda.qk_rope(q, k, i, freq)
    with pytest.raises(kda.KDAError, match="CUDA"):
        kda.paged_rope_append(q, k, k, i, i.long(), freq, c, c)
    with pytest.raises(kda.KDAError, match="CUDA"):
        kda.verify_drafts(z(3, 2, 9), z(3, 1, dtype=torch.int32), z(3, 2))


def test_law_of_the_plain_form():
    """The reference itself: over a fine grid of uniform numbers the token after a draft is the target's law."""
    p, q = [0.4, 0.35, 0.25], [0.2, 0.3, 0.5]
    steps = 40
    share = [0.0] * 3
    for d in range(3):
        us = torch.tensor([[(a + 0.5) / steps, (b + 0.5) / steps] for a in range(steps) for b in range(steps)])
        n = len(us)
        t = torch.tensor(p, dtype=torch.float64).view(1, 1, 3).repeat(n, 2, 1)
        f = torch.tensor(q, dtype=torch.float64).view(1, 1, 3).repeat(n, 1, 1)
        _, out = verify_ref(t, torch.full((n, 1), d, dtype=torch.int32), us, f)
        for row in out:
            share[row[0]] += q[d] / n
    assert all(abs(a - b) <= 1.5 / steps for a, b in zip(share, p))  # (a grid's cell on either border)


def test_plain_form_of_one_certain_draft():
    target, _, tokens, u = draft_inputs(20, 2, 6, seed=1, certain=True)
    acc, out = verify_ref(target, tokens, u)
    for a, row, d in zip(acc, out, tokens[:, 0].tolist()):
        assert row[0] == d if a else (row[0] != d and row[1] == -1)


@pytest.mark.parametrize("V,dtype", [(131_072, torch.float32), (32_768, torch.float32), (100_003, torch.bfloat16), (7, torch.float32),
                                     (5_000_000, torch.float32), (1_900_000, torch.bfloat16)])
def test_a_workspace_does_for_fewer_requests(V, dtype):
    """Sizes never fall as requests come (a server keeps one for its largest batch)."""
    size = [kda.verify_drafts_workspace_size(n, 5, V, dtype) for n in range(1, 700)]
    assert size[0] > 0 and all(a <= b for a, b in zip(size, size[1:]))


FAR = [2 ** 32 + 5, 2 ** 31, 2 ** 40, -2 ** 32 + 5]


@pytest.mark.parametrize("far", FAR)
def test_numbers_past_32_bits_on_the_host(far):
    """Not cut down to their last 32 bits."""
    assert kda.verify_drafts_workspace_size(5, 5, 100) > 0 and kda.paged_attn_workspace_size(5, 5, 8, 2) > 0
    for at in range(3):
        a = [5, 5, 100]
        a[at] = far
        assert kda.verify_drafts_workspace_size(*a) == 0
        a = [5, 8, 2]
        a[at] = far
        assert kda.paged_attn_workspace_size(5, *a) == 0
    assert kda.paged_attn_workspace_size(2 ** 64 + 5, 5, 8, 2) == 0
    with pytest.raises(kda.KDAError, match="rot_dim"):
        kda.rope_frequencies(far + 59)  # (64 in the last 32 bits of two of them)


@pytest.mark.parametrize("rot", [8, 96, 128])
@pytest.mark.parametrize("kw", [dict(), dict(base=1e6), dict(base=500000.0, scaling="ntk", factor=32.0),
                                dict(scaling="yarn", factor=16.0, original_len=4096)])
def test_frequencies_to_more_digits(rot, kw):
    """Within 2^-50 of the formula in 50 digits, and half a unit: the power, the ramp's two differences and quotient, the
    sum of its parts and the quotient by a turn are under 8 roundings of 2^-53 or their like."""
    d = decimal.Decimal
    with decimal.localcontext() as ctx:
        ctx.prec = 50
        turn = 2 * d("3.14159265358979323846264338327950288419716939937510582")
        base, factor = d(kw.get("base", 10000.0)), d(kw.get("factor", 1.0))
        if kw.get("scaling") == "ntk":
            base *= (factor.ln() * rot / (rot - 2)).exp()
        freq, _ = kda.rope_frequencies(rot, **kw)
        for i, got in enumerate(freq.tolist()):
            f = (base.ln() * -2 * i / rot).exp()
            if kw.get("scaling") == "yarn":
                g = min(d(1), max(d(0), (kw["original_len"] * f / turn - 1) / 31))
                f *= g + (1 - g) / factor
            want = f / turn * 2 ** 64
            assert abs(got - want) <= want * d(2) ** -50 + 1
