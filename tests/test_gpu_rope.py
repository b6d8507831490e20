"""Rotary positions and per-head norms against their 64-bit form, alone and with the append."""
import math

import pytest
import torch

import linear_attention_serving_gb300 as kda
from linear_attention_serving_gb300 import paged
from serving_testutil import D, FP32, rope_close, rope_ref
from test_gpu_canaries import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def inputs(T, hq, hkv, dtype, seed=0, top=5000):
    g = torch.Generator().manual_seed(seed)
    qkv = (2 * torch.randn(T, hq + 2 * hkv, D, generator=g)).to(dtype)
    pos = torch.randint(0, top, (T,), generator=g).int()
    w = 1 + 0.2 * torch.randn(2, D, generator=g)
    return qkv.to(DEV), pos.to(DEV), w[0].to(DEV).contiguous(), w[1].to(DEV).contiguous()


def split(qkv, hq, hkv):
    return qkv.split((hq, hkv, hkv), 1)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,hq,hkv,rot,interleaved,norm", [
    (1, 1, 1, 128, False, False), (1, 96, 8, 128, True, True), (3, 16, 2, 64, False, True), (257, 5, 1, 96, False, False),
    (33, 8, 8, 32, True, False), (50, 7, 3, 8, False, True), (50, 7, 3, 8, True, True), (21, 4, 2, 0, False, True),
    (64, 2, 2, 120, False, True), (64, 2, 2, 120, True, True), (1501, 32, 8, 128, False, True), (40, 3, 1, 56, True, False), (2, 300, 20, 128, False, True),
    (610, 70, 1, 16, True, True)])
def test_rope(T, hq, hkv, rot, interleaved, norm, dtype):
    qkv, pos, qw, kw = inputs(T, hq, hkv, dtype, seed=T + rot)
    q, k, _ = split(qkv, hq, hkv)
    freq, amp = kda.rope_frequencies(rot, device=DEV) if rot else (None, 1.0)
    if not norm:
        qw = kw = None
    before = qkv.clone()
    q2, k2 = kda.qk_rope(q, k, pos, freq, amplitude=amp, interleaved=interleaved, q_weight=qw, k_weight=kw, eps=1e-5)
    assert torch.equal(before, qkv)
    f = None if freq is None else freq.tolist()
    rope_close(q2, *rope_ref(q, pos, f, amp, interleaved, qw, 1e-5), dtype)
    rope_close(k2, *rope_ref(k, pos, f, amp, interleaved, kw, 1e-5), dtype)


def test_many_tokens_and_few_make_the_same_bits():
    """Four tokens to a block, one, or several blocks to one token: the rows are the same."""
    qkv, pos, qw, kw = inputs(9001, 24, 4, BF16, seed=3)
    q, k, _ = split(qkv, 24, 4)
    freq, _ = kda.rope_frequencies(128, device=DEV)
    q2, k2 = kda.qk_rope(q, k, pos, freq, q_weight=qw, k_weight=kw)
    for at in (0, 1, 4500, 9000):
        for n in (1, 60):
            s = slice(at, at + n)
            a, b = kda.qk_rope(q[s], k[s], pos[s].contiguous(), freq, q_weight=qw, k_weight=kw)
            assert torch.equal(a, q2[s]) and torch.equal(b, k2[s])


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_many_tokens_of_few_heads(interleaved, dtype, cache):
    """A token to each unit of a block: the bits of a block for each token."""
    T, hq, hkv, ps = 2501, 3, 1, 16
    qkv, pos, qw, kw = inputs(T, hq, hkv, dtype, seed=13)
    q, k, v = split(qkv, hq, hkv)
    freq, _ = kda.rope_frequencies(96, device=DEV)
    opts = dict(interleaved=interleaved, q_weight=qw, k_weight=kw)
    q2, k2 = kda.qk_rope(q, k, pos, freq, **opts)
    rope_close(q2[:50], *rope_ref(q[:50], pos[:50], freq.tolist(), 1.0, interleaved, qw, 1e-6), dtype)
    ks = vs = None
    if cache == E4M3:
        ks, vs = torch.full((hkv,), 0.02, device=DEV), torch.full((hkv,), 0.03, device=DEV)
    slots = torch.randperm(160 * ps, generator=torch.Generator().manual_seed(1))[:T].to(DEV)
    (kc, vc), (kc2, vc2) = caches(160, hkv, ps, cache), caches(160, hkv, ps, cache)
    q3 = kda.paged_rope_append(q, k, v, pos, slots, freq, kc, vc, k_scale=ks, v_scale=vs, **opts)
    assert torch.equal(q3, q2)
    for at in range(0, T, 500):
        s = slice(at, at + 500)
        a, b = kda.qk_rope(q[s], k[s], pos[s].contiguous(), freq, **opts)
        assert torch.equal(a, q2[s]) and torch.equal(b, k2[s])
        kda.paged_rope_append(q[s], k[s], v[s], pos[s].contiguous(), slots[s].contiguous(), freq, kc2, vc2, k_scale=ks, v_scale=vs, **opts)
    raw = torch.uint8 if cache == E4M3 else cache
    assert torch.equal(kc.view(raw), kc2.view(raw)) and torch.equal(vc.view(raw), vc2.view(raw))


def test_far_positions_stretched():
    """Angles are exact modulo a turn at any position, negative ones too."""
    pos = torch.tensor([0, 1, -1, 999_999, 16_777_217, 2 ** 31 - 1, -2 ** 31, 123_456_789], dtype=torch.int32, device=DEV)
    qkv, _, _, _ = inputs(len(pos), 2, 1, F32, seed=5)
    q, k, _ = split(qkv, 2, 1)
    for scaling in ("none", "linear", "ntk", "yarn"):
        freq, amp = kda.rope_frequencies(128, base=500000.0, scaling=scaling, factor=32.0, original_len=8192, device=DEV)
        assert (amp != 1) == (scaling == "yarn")
        q2, k2 = kda.qk_rope(q, k, pos, freq, amplitude=amp)
        rope_close(q2, *rope_ref(q, pos, freq.tolist(), amp, False, None, 0), F32)
        rope_close(k2, *rope_ref(k, pos, freq.tolist(), amp, False, None, 0), F32)


def test_in_place_on_the_projection():
    qkv, pos, qw, kw = inputs(300, 8, 2, BF16, seed=9)
    freq, _ = kda.rope_frequencies(64, device=DEV)
    q, k, v = split(qkv, 8, 2)
    want = kda.qk_rope(q, k, pos, freq, q_weight=qw, k_weight=kw)
    kept = v.clone()
    got = kda.qk_rope(q, k, pos, freq, q_weight=qw, k_weight=kw, q_out=q, k_out=k)
    assert got[0].data_ptr() == q.data_ptr()
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(v, kept)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_zeros_huge_and_not_finite(dtype):
    """A row of zeros stays zeros under a norm with eps; what is not finite stays in its pair (without a
    norm) or its row; channels that are not turned pass through as they are."""
    q = torch.zeros(1, 4, D, dtype=dtype, device=DEV)
    q[0, 1] = 1e18
    q[0, 2, 3] = float("inf")
    q[0, 3, 100] = float("nan")
    q[0, 3, 101] = float("inf")
    k = q[:, :1].clone()
    pos = torch.tensor([77], dtype=torch.int32, device=DEV)
    w = torch.ones(D, device=DEV)
    freq, _ = kda.rope_frequencies(64, device=DEV)
    a, b = kda.qk_rope(q, k, pos, freq, q_weight=w, k_weight=w)
    assert (a[0, 0] == 0).all() and (b == 0).all()
    rope_close(a[:, 1:2], *rope_ref(q[:, 1:2], pos, freq.tolist(), 1.0, False, w, 1e-6), dtype)
    a, b = kda.qk_rope(q, k, pos, freq)
    bad = ~torch.isfinite(a)
    assert bad[0, 2].nonzero().flatten().tolist() == [3, 35]
    assert bad[0, 3].nonzero().flatten().tolist() == [100, 101] and a[0, 3, 101] == float("inf")
    assert not bad[0, :2].any()


# ------------------------------------------------------------------ with the append
def caches(pages, hkv, ps, cache, seed=0, lie_apart=False):
    g = torch.Generator().manual_seed(seed)
    pool = torch.randn(pages, 2 if lie_apart else 1, hkv, ps, D, generator=g).to(cache).to(DEV)
    if lie_apart:
        return pool[:, 0], pool[:, 1]
    return pool[:, 0].contiguous(), pool[:, 0].flip(0).contiguous() if cache != E4M3 else pool[:, 0].contiguous().clone()


@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
@pytest.mark.parametrize("T,hq,hkv,ps,rot,interleaved,norm,apart", [
    (1, 4, 1, 16, 128, False, True, False), (37, 9, 3, 48, 64, True, True, False), (300, 16, 8, 64, 128, False, False, True),
    (5, 2, 2, 16, 0, False, True, False), (3001, 32, 8, 32, 128, True, True, False), (65, 8, 1, 128, 40, False, True, True)])
def test_rope_append(T, hq, hkv, ps, rot, interleaved, norm, apart, dtype, cache):
    """The same as the rotation alone and then the append: bit for bit, but for e4m3 keys, which are rounded once."""
    qkv, pos, qw, kw = inputs(T, hq, hkv, dtype, seed=T)
    q, k, v = split(qkv, hq, hkv)
    if not norm:
        qw = kw = None
    freq, amp = kda.rope_frequencies(rot, scaling="yarn", factor=4.0, original_len=1000, device=DEV) if rot else (None, 1.0)
    pages = -(-T // ps) + 4
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(pages * ps, generator=g)[:T].to(DEV)
    if T > 2:
        slots[T // 2] = -1
    kc, vc = caches(pages, hkv, ps, cache, seed=1, lie_apart=apart)
    kc2, vc2 = kc.clone(), vc.clone()
    ks = vs = None
    if cache == E4M3:
        ks, vs = (0.02 + torch.rand(hkv, generator=g).to(DEV) / 50 for _ in range(2))
    opts = dict(amplitude=amp, interleaved=interleaved, q_weight=qw, k_weight=kw, eps=1e-5)
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    q2 = kda.paged_rope_append(q, k, v, pos, slots, freq, kc, vc, k_scale=ks, v_scale=vs, error_word=err, **opts)
    want, k2 = kda.qk_rope(q, k, pos, freq, **opts)
    assert int(err) == 0 and torch.equal(q2, want)
    kda.paged_append(k2, v.contiguous(), slots, kc2, vc2, k_scale=ks, v_scale=vs)
    raw = torch.uint8 if cache == E4M3 else cache
    assert torch.equal(vc.view(raw), vc2.view(raw))
    if cache != E4M3:
        assert torch.equal(kc, kc2)
        return
    ref, size = rope_ref(k, pos, None if freq is None else freq.tolist(), amp, interleaved, kw, 1e-5)
    sc = ks.double().cpu()[None, :, None]
    live = (slots >= 0).cpu()
    got = kc[(slots // ps).clamp(min=0), :, (slots % ps)].float().double().cpu()[live]
    ref, size = (ref / sc)[live].clamp(-448, 448), (size / sc)[live]
    # half a step of e4m3: 2^-4 of the value, or of the smallest normal number's step (2^-9) below 2^-6
    tol = torch.maximum(2.0 ** -4 * ref.abs(), torch.full_like(ref, 2.0 ** -10)) + 1.1 * (FP32 + 2.0 ** -24) * size
    assert ((got - ref).abs() <= tol).all()
    untouched = torch.ones(pages * ps, dtype=torch.bool)
    untouched[slots[slots >= 0].cpu()] = False
    a, b = (x.view(raw).transpose(1, 2).reshape(pages * ps, -1).cpu()[untouched] for x in (kc, kc2))
    assert torch.equal(a, b)


def test_rope_append_writes_nothing_else():
    """Guards around every output, slots past the cache, and skipped ones."""
    T, hq, hkv, ps, pages = 70, 4, 2, 16, 6
    qkv, pos, qw, kw = inputs(T, hq, hkv, BF16, seed=2)
    q, k, v = split(qkv, hq, hkv)
    freq, _ = kda.rope_frequencies(128, device=DEV)
    slots = torch.arange(T, device=DEV)
    slots[3], slots[4], slots[5] = -1, pages * ps, 1 << 40
    gq, gk, gv = (Guarded(s, BF16) for s in ((T, hq, D), (pages, hkv, ps, D), (pages, hkv, ps, D)))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    gk.t.zero_()
    gv.t.zero_()
    kda.paged_rope_append(q, k, v, pos, slots, freq, gk.t, gv.t, q_weight=qw, k_weight=kw, q_out=gq.t, error_word=err)
    assert int(err) == paged.DEVERR_PAGE
    for x in (gq, gk, gv):
        assert x.intact()
    want, _ = kda.qk_rope(q, k, pos, freq, q_weight=qw, k_weight=kw)
    assert torch.equal(gq.t, want)
    for t in (gk.t, gv.t):
        rows = t.transpose(1, 2).reshape(pages * ps, -1).abs().sum(1) > 0
        live = torch.zeros(pages * ps, dtype=torch.bool, device=DEV)
        live[slots[(slots >= 0) & (slots < pages * ps)]] = True
        assert torch.equal(rows, live)


@pytest.mark.parametrize("cache", [BF16, E4M3])
def test_offsets_past_32_bits(cache):
    """Pages whose places in the cache pass 2^31 elements."""
    T, hq, hkv, ps, pages = 150, 4, 8, 64, 40_000
    qkv, pos, qw, kw = inputs(T, hq, hkv, BF16, seed=21)
    q, k, v = split(qkv, hq, hkv)
    freq, _ = kda.rope_frequencies(128, device=DEV)
    big, small = ([torch.empty(n, hkv, ps, D, device=DEV, dtype=cache) for _ in range(2)] for n in (pages, 4))
    near = torch.randperm(4 * ps, generator=torch.Generator().manual_seed(1))[:T].to(DEV)
    far = near + (pages - 4) * ps
    ks = vs = torch.full((hkv,), 0.03, device=DEV) if cache == E4M3 else None
    for kc, vc, slots in ((*big, far), (*small, near)):
        for c in (kc, vc):
            c[-4:].view(torch.uint8).zero_()
        kda.paged_rope_append(q, k, v, pos, slots, freq, kc, vc, q_weight=qw, k_weight=kw, k_scale=ks, v_scale=vs)
    for a, b in zip(big, small):
        assert torch.equal(a[-4:].view(torch.uint8), b.view(torch.uint8)) and (b.view(torch.uint8) != 0).any()


def test_no_tokens():
    q, k = (torch.empty(0, h, D, dtype=BF16, device=DEV) for h in (4, 2))
    pos = torch.empty(0, dtype=torch.int32, device=DEV)
    freq, _ = kda.rope_frequencies(128, device=DEV)
    a, b = kda.qk_rope(q, k, pos, freq)
    assert a.shape == q.shape and b.shape == k.shape
    kc, vc = caches(2, 2, 16, BF16)
    assert kda.paged_rope_append(q, k, k, pos, torch.empty(0, dtype=torch.int64, device=DEV), freq, kc, vc).shape == q.shape


def test_graph_and_other_stream():
    """Captured and replayed over new inputs; launched on the current stream."""
    qkv, pos, qw, kw = inputs(30, 8, 2, BF16, seed=4)
    freq, _ = kda.rope_frequencies(128, device=DEV)
    q, k, v = split(qkv, 8, 2)
    kc, vc = caches(4, 2, 16, BF16)
    slots = torch.arange(30, device=DEV)
    out = torch.empty(30, 8, D, dtype=BF16, device=DEV)
    call = lambda: kda.paged_rope_append(q, k, v, pos, slots, freq, kc, vc, q_weight=qw, k_weight=kw, q_out=out)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    fresh = inputs(30, 8, 2, BF16, seed=44)[0]
    qkv.copy_(fresh)
    out.zero_()
    kc.zero_()
    graph.replay()
    torch.cuda.synchronize()
    want = kda.qk_rope(q, k, pos, freq, q_weight=qw, k_weight=kw)
    assert torch.equal(out, want[0])
    assert torch.equal(kc.transpose(1, 2).reshape(-1, 2, D)[:30], want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a, _ = kda.qk_rope(q, k, pos, freq, q_weight=qw, k_weight=kw)
    s.synchronize()
    assert torch.equal(a, want[0])


def test_plain_binding_makes_the_same_calls(monkeypatch):
    qkv, pos, qw, kw = inputs(20, 8, 2, BF16, seed=6)
    freq, _ = kda.rope_frequencies(128, device=DEV)
    q, k, v = split(qkv, 8, 2)
    kc, vc = caches(4, 2, 16, BF16)
    slots = torch.arange(20, device=DEV)
    want = kda.qk_rope(q, k, pos, freq, q_weight=qw, k_weight=kw)
    q2 = kda.paged_rope_append(q, k, v, pos, slots, freq, kc, vc, q_weight=qw, k_weight=kw)
    kc2, vc2 = torch.zeros_like(kc), torch.zeros_like(vc)
    for name in ("_fast_rope", "_fast_rope_append"):
        monkeypatch.setattr(paged, name, lambda *a: None)
    got = kda.qk_rope(q, k, pos, freq, q_weight=qw, k_weight=kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    kc2.copy_(kc)
    vc2.copy_(vc)
    kc2.view(-1)[:] = 0
    q3 = kda.paged_rope_append(q, k, v, pos, slots, freq, kc2, vc2, q_weight=qw, k_weight=kw)
    rows = lambda x: x.transpose(1, 2).reshape(-1, 2, D)[:20]  # noqa: E731
    assert torch.equal(q3, q2) and torch.equal(rows(kc2), rows(kc)) and torch.equal(vc2, vc)


def test_binding_refusals():
    qkv, pos, qw, kw = inputs(4, 4, 2, BF16)
    freq, _ = kda.rope_frequencies(64, device=DEV)
    q, k, v = split(qkv, 4, 2)
    bad = [dict(q=q.half()), dict(q=q[..., :64]), dict(k=k[:3]), dict(k=k.float()), dict(positions=pos.long()),
           dict(positions=pos[:3]), dict(freq=freq.int()), dict(q_weight=qw[:64]), dict(q_weight=qw.double()), dict(eps=-1.0),
           dict(amplitude=float("nan")), dict(q_out=torch.empty(4, 3, D, dtype=BF16, device=DEV)),
           dict(q=q.transpose(0, 1)[:4]), dict(freq=freq[:3].contiguous()), dict(k_out=q[:, :2]), dict(q=q.cpu())]
    for kw_ in bad:
        a = dict(q=q, k=k, positions=pos, freq=freq)
        a.update(kw_)
        with pytest.raises(kda.KDAError):
            kda.qk_rope(**a)
    kc, vc = caches(2, 2, 16, BF16)
    slots = torch.arange(4, device=DEV)
    bad = [dict(v=v[:, :1]), dict(slot_map=slots.int()), dict(slot_map=slots[:3]), dict(k_cache=kc[:, :1]),
           dict(k_cache=kc.float(), v_cache=vc.float()), dict(k_scale=qw[:2].contiguous(), v_scale=qw[:2].contiguous()),
           dict(v=v.float()), dict(q_out=k)]
    for kw_ in bad:
        a = dict(q=q, k=k, v=v, positions=pos, slot_map=slots, freq=freq, k_cache=kc, v_cache=vc)
        a.update(kw_)
        with pytest.raises(kda.KDAError):
            kda.paged_rope_append(**a)


def test_frequencies_are_there_for_every_stream():
    """The table is read at once on a stream that nothing orders behind the one it was made on."""
    want, _ = kda.rope_frequencies(128)
    side, work = torch.cuda.Stream(), torch.cuda.Stream()
    got = torch.empty(20, 64, dtype=torch.int64, device=DEV)
    stale = [torch.full((64,), -1, dtype=torch.int64, device=DEV) for _ in range(40)]
    torch.cuda.synchronize()
    del stale  # (memory that holds something else)
    for i in range(20):
        with torch.cuda.stream(work):
            torch.cuda._sleep(20_000_000)
            freq, _ = kda.rope_frequencies(128, device=DEV)
        with torch.cuda.stream(side):
            got[i].copy_(freq)
    torch.cuda.synchronize()
    assert torch.equal(got.cpu(), want.expand(20, 64))


@pytest.mark.parametrize("plain", [False, True])
def test_norms_without_positions(plain, monkeypatch):
    """Nothing turns: no positions are needed; with a rotation they are."""
    if plain:
        monkeypatch.setattr(paged, "_fast_rope", lambda *a: None)
        monkeypatch.setattr(paged, "_fast_rope_append", lambda *a: None)
    qkv, pos, qw, kw = inputs(40, 4, 2, BF16, seed=31)
    q, k, v = split(qkv, 4, 2)
    slots = torch.arange(40, device=DEV)
    want = kda.qk_rope(q, k, pos, None, q_weight=qw, k_weight=kw)
    got = kda.qk_rope(q, k, None, None, q_weight=qw, k_weight=kw)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    rope_close(got[0], *rope_ref(q, pos, None, 1.0, False, qw, 1e-6), BF16)
    (kc, vc), (kc2, vc2) = caches(4, 2, 16, BF16), caches(4, 2, 16, BF16)
    want = kda.paged_rope_append(q, k, v, pos, slots, None, kc, vc, q_weight=qw, k_weight=kw)
    got = kda.paged_rope_append(q, k, v, None, slots, None, kc2, vc2, q_weight=qw, k_weight=kw)
    assert torch.equal(got, want) and torch.equal(kc, kc2) and torch.equal(vc, vc2)
    freq, _ = kda.rope_frequencies(64, device=DEV)
    with pytest.raises(kda.KDAError, match="positions"):
        kda.qk_rope(q, k, None, freq)
    with pytest.raises(kda.KDAError, match="positions"):
        kda.paged_rope_append(q, k, v, None, slots, freq, kc, vc)


@pytest.mark.parametrize("plain", [False, True])
@pytest.mark.parametrize("T", [1, 60, 2000])
def test_keys_do_not_hold_the_queries_memory(T, plain, monkeypatch):
    """A prompt's results are tensors of their own; small ones may share up to a megabyte."""
    if plain:
        monkeypatch.setattr(paged, "_fast_rope", lambda *a: None)
    qkv, pos, qw, kw = inputs(T, 16, 2, BF16, seed=T)
    q, k, _ = split(qkv, 16, 2)
    freq, _ = kda.rope_frequencies(128, device=DEV)
    want = rope_ref(k[-3:], pos[-3:], freq.tolist(), 1.0, False, kw, 1e-6)
    for x in kda.qk_rope(q, k, pos, freq, q_weight=qw, k_weight=kw):
        held = x.untyped_storage().nbytes()
        assert held == x.nbytes or (T < 2000 and held <= 1 << 20)
    rope_close(x[-3:], *want, BF16)


def test_a_table_of_the_models_own():
    """Frequencies whose ramp is linear in the pair's number (base 10^6, factor 4, 32,768 positions), as int64 turns
    times 2^64: the rotation by p f_i in 64 bits, whose own angles are off by 2^-53 of p f_i."""
    rot, base, factor, length = 128, 1e6, 4.0, 32768
    low, high = (rot * math.log(length / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0))
    low, high = math.floor(low), math.ceil(high)
    f = []
    for i in range(rot // 2):
        x, g = base ** (-2 * i / rot), 1 - min(1.0, max(0.0, (i - low) / (high - low)))
        f.append(x * (g + (1 - g) / factor))
    paper, amp = kda.rope_frequencies(rot, base=base, scaling="yarn", factor=factor, original_len=length)
    off = [abs(a / 2.0 ** 64 * 2 * math.pi / b - 1) for a, b in zip(paper.tolist(), f)]
    assert sum(x > 0.01 for x in off) == 16 and 0.41 < max(off) < 0.43  # (what include/kda.h says of the other ramp)
    table = torch.tensor([round(x / (2 * math.pi) * 2 ** 64) for x in f], dtype=torch.int64)
    qkv, pos, _, _ = inputs(500, 3, 1, F32, seed=41, top=131_072)
    q, k, _ = split(qkv, 3, 1)
    got, _ = kda.qk_rope(q, k, pos, table.to(DEV), amplitude=amp)
    angle = pos.cpu().double()[:, None] * torch.tensor(f, dtype=torch.float64)
    c, s = (amp * angle.cos())[:, None], (amp * angle.sin())[:, None]
    a, b = q.double().cpu().split(rot // 2, 2)
    size = amp * (a.abs() + b.abs()).repeat(1, 1, 2)
    rope_close(got, torch.cat((a * c - b * s, a * s + b * c), 2), size, F32)
