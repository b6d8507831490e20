"""Paged attention through a window beside sinks, against the plain 64-bit form."""
import pytest
import torch

import linear_attention_serving_gb300 as kda
from linear_attention_serving_gb300 import paged
from paged_testutil import D, attn_close, make
from serving_testutil import sinks_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def hide(d, ps, window, sinks):
    """Keys that no query sees become NaN, and pages without a seen key leave the table."""
    nan = float("nan")
    if d["k_cache"].dtype == E4M3:
        d["k_cache"], d["v_cache"] = d["k_cache"].float(), d["v_cache"].float()
    for i, kv in enumerate(d["kv"]):
        n = d["cu"][i + 1] - d["cu"][i]
        first = max(0, kv - n - window + 1) if n else kv
        for b in range(-(-kv // ps)):
            rows = range(b * ps, min(kv, b * ps + ps))
            gone = [j % ps for j in rows if j < first and j >= (sinks if n else 0)]
            for c in (d["k_cache"], d["v_cache"]):
                c[d["table"][i][b], :, gone] = nan
            if len(gone) == len(rows):
                d["table"][i][b] = -5


def run(new, ctx, hkv, g, ps, cache, window, sinks, seed=0, max_q=None, hidden=True, **kw):
    d = make(new, ctx, hkv, g, ps, cache=cache, seed=seed)
    if hidden:
        hide(d, ps, window, sinks)
    dev = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    dev["k_cache"], dev["v_cache"] = dev["k_cache"].to(cache), dev["v_cache"].to(cache)
    err = i32([0])
    o, lse = kda.paged_attn(dev["q"], dev["k_cache"], dev["v_cache"], i32(d["table"]), i32(d["cu"]), i32(d["kv"]),
                            max_q=max(new) if max_q is None else max_q, window=window, sinks=sinks, k_scale=dev["k_scale"],
                            v_scale=dev["v_scale"], error_word=err, **kw)
    assert int(err) == 0
    ref = sinks_ref(d["q"], dev["k_cache"].cpu(), dev["v_cache"].cpu(), d["table"], d["cu"], d["kv"], window=window, sinks=sinks,
                    k_scale=d["k_scale"], v_scale=d["v_scale"])
    attn_close(o, lse, ref, d["q"].dtype, cache)
    return o, lse


# (new, ctx, kv heads, group, page size, window, sinks)
CASES = [
    ([1], [0], 1, 1, 16, 1, 1), ([1], [700], 1, 1, 16, 1, 1), ([1], [5000], 2, 4, 64, 100, 4), ([1] * 5, [0, 3, 129, 1000, 127], 2, 3, 16, 64, 5),
    ([1, 1], [2000, 400], 1, 8, 128, 300, 128), ([1, 1], [2000, 400], 1, 8, 32, 300, 129), ([1, 1, 1], [255, 256, 257], 2, 2, 16, 128, 127),
    ([3, 5, 2], [1000, 0, 77], 2, 4, 16, 50, 17), ([5] * 3, [640, 383, 129], 1, 16, 64, 128, 64), ([2, 0, 4], [300, 500, 900], 1, 2, 48, 33, 200),
    ([4], [1500], 2, 2, 16, 7, 300), ([1], [1500], 2, 2, 16, 1499, 3), ([1], [1500], 2, 2, 16, 1400, 3), ([1], [1500], 2, 2, 16, 1200, 200),
]


@pytest.mark.parametrize("cache", [BF16, E4M3, F32])
@pytest.mark.parametrize("new,ctx,hkv,g,ps,window,sinks", CASES)
def test_few_rows(new, ctx, hkv, g, ps, window, sinks, cache):
    run(new, ctx, hkv, g, ps, cache, window, sinks, seed=len(ctx) + window)


@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 11)])
@pytest.mark.parametrize("rows,g", [(17, 1), (20, 4), (24, 8), (24, 1), (25, 5), (28, 4), (32, 16), (33, 3)])
def test_e4m3_windows_of_up_to_two_tiles_of_rows(rows, g, window, sinks):
    """Over 16 rows of a kv head: 24 columns of 32 are worked on where no request has more."""
    run([rows // g, 1, 2], [700, 130, 40], 2, g, 64, E4M3, window, sinks, seed=rows, hidden=window > 0)


TILES = [
    ([200], [0], 1, 1, 16, 64, 4), ([130], [1000], 2, 2, 64, 100, 20), ([300, 33], [700, 129], 1, 4, 16, 128, 128),
    ([65, 400], [513, 2], 1, 3, 32, 200, 129), ([257], [640], 2, 1, 128, 31, 64), ([40], [900], 1, 8, 48, 900, 10),
    ([500], [100], 1, 2, 16, 1, 1), ([77], [3000], 1, 5, 64, 250, 700),
]


@pytest.mark.parametrize("cache", [BF16, F32])
@pytest.mark.parametrize("new,ctx,hkv,g,ps,window,sinks", TILES)
def test_many_rows(new, ctx, hkv, g, ps, window, sinks, cache):
    run(new, ctx, hkv, g, ps, cache, window, sinks, seed=len(ctx) + window, hidden=cache is BF16)


def test_e4m3_over_32_rows():
    run([40], [900], 1, 2, 16, E4M3, 130, 70, hidden=False)


def test_mixed_batch():
    """Single tokens, windows and chunks in one call: both kernels, several blocks, cut items."""
    new, ctx = [1, 1, 300, 1, 5, 90, 1, 0, 1, 129], [3000, 0, 800, 127, 600, 2000, 1290, 44, 511, 0]
    run(new, ctx, 2, 4, 16, BF16, 333, 37)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32])
def test_long_window_is_cut_over_the_blocks(cache):
    """One item over many blocks: pieces that begin with a sink's tile, in one, and behind the last."""
    o, lse = run([1], [40000], 1, 2, 64, cache, 39000, 300, hidden=False)
    o2, lse2 = run([1], [40000], 1, 2, 64, cache, 39000, 300, hidden=False)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32])
def test_more_requests_than_threads(cache):
    n = 900
    run([1] * n, [(7 * i) % 290 for i in range(n)], 1, 1, 16, cache, 30, 6)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32])
@pytest.mark.parametrize("new,ctx", [([1, 1], [900, 3]), ([70], [500])])
def test_sinks_that_change_nothing(cache, new, ctx):
    """No window: sinks have no say.  No sinks: the window alone, the same bits.  Sinks past the context, or that
    meet the window: all keys."""
    def call(**kw):
        d = make(new, ctx, 2, 2, 16, cache=cache, seed=5)
        dev = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in d.items()}
        return kda.paged_attn(dev["q"], dev["k_cache"], dev["v_cache"], i32(d["table"]), i32(d["cu"]), i32(d["kv"]), max_q=max(new),
                              k_scale=dev["k_scale"], v_scale=dev["v_scale"], **kw)[0]

    plain = call()
    assert torch.equal(plain, call(sinks=9))
    assert torch.equal(plain, call(window=5, sinks=2 ** 31 - 1))
    assert torch.equal(plain, call(window=2 ** 31 - 1, sinks=3))
    assert torch.equal(call(window=50), call(window=50, sinks=0))
    assert not torch.equal(call(window=50), call(window=50, sinks=9))
    run(new, ctx, 2, 2, 16, cache, 50, 800, hidden=False)
    run(new, ctx, 2, 2, 16, cache, 450, 449, hidden=False)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32])
def test_queries_before_position_zero(cache):
    """More new tokens than the length says: those at negative positions see nothing."""
    d = make([40, 3], [0, 0], 2, 2, 16, cache=cache, seed=8)
    d["kv"] = [25, 1]
    dev = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in d.items()}
    o, lse = kda.paged_attn(dev["q"], dev["k_cache"], dev["v_cache"], i32(d["table"]), i32(d["cu"]), i32(d["kv"]), max_q=40, window=6,
                            sinks=3, k_scale=dev["k_scale"], v_scale=dev["v_scale"])
    ref = sinks_ref(d["q"], d["k_cache"], d["v_cache"], d["table"], d["cu"], d["kv"], window=6, sinks=3, k_scale=d["k_scale"],
                    v_scale=d["v_scale"])
    assert torch.isinf(lse[:15]).all() and (o[:15] == 0).all()
    attn_close(o, lse, ref, d["q"].dtype, cache)


def test_graph_and_short_wait_budget():
    """Replays give the same bits; a budget that looks at every wait (kernels of their own) too."""
    new, ctx = [1, 90, 4], [600, 300, 1000]
    for cache in (BF16, F32, E4M3):
        d = make(new, ctx, 2, 4, 16, cache=cache, seed=2)
        dev = {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in d.items()}
        t, cu, kv = i32(d["table"]), i32(d["cu"]), i32(d["kv"])
        ws = torch.empty(kda.paged_attn_workspace_size(sum(new), 3, 8, 2), dtype=torch.uint8, device=DEV)
        out = torch.empty_like(dev["q"])
        call = lambda: kda.paged_attn(dev["q"], dev["k_cache"], dev["v_cache"], t, cu, kv, max_q=90, window=100, sinks=20,  # noqa: E731
                                      k_scale=dev["k_scale"], v_scale=dev["v_scale"], out=out, workspace=ws)
        call()
        want = out.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
        was = kda.set_wait_budget(999_999)
        try:
            call()
            torch.cuda.synchronize()
        finally:
            kda.set_wait_budget(was)
        assert torch.equal(out, want)


@pytest.mark.parametrize("cache", [BF16, E4M3, F32])
def test_offsets_past_32_bits(cache):
    """The same content on pages whose places in the cache pass 2^31 elements: the same bits."""
    new, ctx, ps, hkv = [1, 70, 3], [900, 300, 500], 64, 8
    d = make(new, ctx, hkv, 2, ps, cache=cache, seed=6)
    n = d["k_cache"].shape[0]
    pages = 40_000 if cache != F32 else 34_000
    out = []
    for total in (n, pages):
        kc, vc = (torch.empty(total, hkv, ps, D, device=DEV, dtype=cache) for _ in range(2))
        for a, b in ((kc, d["k_cache"]), (vc, d["v_cache"])):
            a[-n:].view(torch.uint8).copy_(b.to(DEV).view(torch.uint8))
        table = [[x + total - n if x >= 0 else x for x in row] for row in d["table"]]
        sc = [None if d[k] is None else d[k].to(DEV) for k in ("k_scale", "v_scale")]
        out.append(kda.paged_attn(d["q"].to(DEV), kc, vc, i32(table), i32(d["cu"]), i32(d["kv"]), max_q=70, window=90, sinks=20,
                                  k_scale=sc[0], v_scale=sc[1]))
        del kc, vc
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])


@pytest.mark.parametrize("n", [20, 700])
def test_single_tokens_beside_a_chunk(n):
    """Where windows are short the tile kernel takes them all, else the kernel for few rows the single tokens."""
    new, ctx = [1] * n + [40], [(37 * i) % 500 for i in range(n)] + [77]
    for window in (20, 2500):
        run(new, ctx, 2, 2, 16, BF16, window, 9, hidden=False)


def test_bad_page_among_the_sinks():
    d = make([1], [900], 1, 1, 16, cache=BF16, seed=1)
    d["table"][0][0] = 10 ** 6
    err = i32([0])
    kda.paged_attn(d["q"].to(DEV), d["k_cache"].to(DEV), d["v_cache"].to(DEV), i32(d["table"]), i32(d["cu"]), i32(d["kv"]), window=50,
                   sinks=4, error_word=err)
    assert int(err) == paged.DEVERR_PAGE


def test_plain_binding_makes_the_same_call(monkeypatch):
    want = run([1, 3], [500, 90], 2, 2, 16, BF16, 60, 7)
    monkeypatch.setattr(paged, "_fast_attn", lambda *a: None)
    got = run([1, 3], [500, 90], 2, 2, 16, BF16, 60, 7)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refuses_negative_sinks():
    d = make([1], [9], 1, 1, 16)
    with pytest.raises(kda.KDAError):
        kda.paged_attn(d["q"].to(DEV), d["k_cache"].to(DEV), d["v_cache"].to(DEV), i32(d["table"]), i32(d["cu"]), i32(d["kv"]), window=5,
                       sinks=-1)


@pytest.mark.parametrize("window,sinks,hidden", [(300, 9, True), (257, 140, False)])
def test_single_tokens_by_the_kernel_for_few_rows_beside_chunks(window, sinks, hidden):
    """Over 16,384 key tiles of windows and sinks the single tokens have a launch of their own: the requests of up to 16
    rows of one kernel, the others' of the tile kernel, and the pieces of both in one join."""
    n = 700
    new, ctx = [1] * n + [150, 20], [400 + (37 * i) % 501 for i in range(n)] + [333, 805]
    for i in range(0, n, 90):
        new[i] = 1 + i // 90  # (up to 8 tokens of two heads)
    kda.profile_enable(True)
    try:
        kda.profile_collect()
        run(new, ctx, 8, 2, 16, BF16, window, sinks, seed=window, hidden=hidden)
        names = [name for name, _ in kda.profile_collect()]
    finally:
        kda.profile_enable(False)
    assert names == ["paged_few", "paged_tile", "paged_join"]
