"""The paged cache's operators against their plain 64-bit forms."""
import pytest
import torch

import linear_attention_serving_gb300 as kda
from linear_attention_serving_gb300 import paged
from paged_testutil import D, attn_close, attn_ref, cdiv, make, tables_ref
from test_gpu_canaries import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32, E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def errw():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ tables
TABLES = [
    ([1], [0], 16), ([1], [15], 16), ([1], [16], 16), ([0, 0], [5, 0], 16),
    ([3, 0, 17, 1], [14, 16, 0, 33], 16), ([64, 65, 63], [0, 1, 128], 64), ([1] * 700, list(range(700)), 32),
    ([0, 5, 0, 0, 9, 0], [1, 2, 3, 4, 5, 6], 48), ([700, 0, 801], [3, 9, 0], 16),
]


def run_tables(new, ctx, ps, head=2, spare_free=3, seed=0):
    g = torch.Generator().manual_seed(seed)
    width = max(1, max(cdiv(a + b, ps) for a, b in zip(new, ctx))) + 2
    need = sum(cdiv(a + b, ps) - cdiv(b, ps) for a, b in zip(new, ctx))
    had = [cdiv(c, ps) for c in ctx]
    pages = sum(had) + head + need + spare_free
    perm = torch.randperm(pages, generator=g).tolist()
    table, at = [], 0
    for h in had:
        table.append(perm[at:at + h] + [-3] * (width - h))
        at += h
    free = perm[at:]
    ref = tables_ref(new, ctx, table, free, head, ps)
    t = i32(table)
    e = errw()
    out = kda.paged_tables(i32(new), i32(ctx), t, i32(free), i32([head]), sum(new), ps, pages, error_word=e)
    return ref, t, out, int(e)


@pytest.mark.parametrize("new,ctx,ps", TABLES)
def test_tables(new, ctx, ps):
    ref, table, (slots, pos, cu, kv, head), e = run_tables(new, ctx, ps)
    assert e == 0
    assert table.tolist() == ref[0]
    assert slots.tolist() == ref[1] and pos.tolist() == ref[2]
    assert cu.tolist() == ref[3] and kv.tolist() == ref[4] and head.tolist() == [ref[5]]


def test_tables_many_tokens():
    """Over the size where a thread takes four tokens, with ends that are not multiples of four."""
    new, ctx = [120001, 0, 3, 80002, 1, 70006], [7, 2, 30, 0, 15, 100]
    ref, table, (slots, pos, cu, kv, head), e = run_tables(new, ctx, 16)
    assert e == 0 and table.tolist() == ref[0]
    assert torch.equal(slots.cpu(), torch.tensor(ref[1])) and torch.equal(pos.cpu().long(), torch.tensor(ref[2]))
    assert cu.tolist() == ref[3] and head.tolist() == [ref[5]]


def test_tables_many_requests():
    n = 5000
    new, ctx = [(i * 7) % 4 for i in range(n)], [(i * 13) % 50 for i in range(n)]
    ref, table, (slots, pos, cu, kv, head), e = run_tables(new, ctx, 16)
    assert e == 0 and table.tolist() == ref[0] and slots.tolist() == ref[1] and cu.tolist() == ref[3]


def _tables_fail(new, ctx, T, free_n, expect, head=0, table=None, pages=64):
    n, ps = len(new), 16
    t = i32(table or [[50] * 8] * n)
    before = t.clone()
    e = errw()
    out = kda.paged_tables(i32(new), i32(ctx), t, i32(list(range(free_n))), i32([head]), T, ps, pages, error_word=e)
    assert int(e) & expect, int(e)
    return before, t, out


@pytest.mark.parametrize("new,ctx,T,free_n,expect", [
    ([3, -1], [0, 0], 2, 9, paged.DEVERR_LENGTHS), ([3], [-2], 3, 9, paged.DEVERR_LENGTHS),
    ([3, 3], [0, 0], 7, 9, paged.DEVERR_LENGTHS), ([100], [100], 100, 99, paged.DEVERR_LENGTHS),
    ([40, 1], [0, 0], 41, 3, paged.DEVERR_NO_PAGES)])
def test_tables_refuses_on_the_device(new, ctx, T, free_n, expect):
    before, t, (_, _, _, _, head) = _tables_fail(new, ctx, T, free_n, expect)
    assert torch.equal(before, t) and head.tolist() == [0]


@pytest.mark.parametrize("new,ctx,T,free_n,expect", [
    ([3, -1], [0, 0], 2, 9, paged.DEVERR_LENGTHS), ([3], [-2], 3, 9, paged.DEVERR_LENGTHS),
    ([3, 3], [1, 7], 7, 9, paged.DEVERR_LENGTHS), ([100], [100], 100, 99, paged.DEVERR_LENGTHS),
    ([40, 1], [0, 5], 41, 2, paged.DEVERR_NO_PAGES), ([40, 1], [0, 0], 700001, 9, paged.DEVERR_LENGTHS),
    ([1] * 600, [16] * 600, 600, 599, paged.DEVERR_NO_PAGES)])
def test_tables_failed_call_leaves_an_empty_step(new, ctx, T, free_n, expect):
    """Whatever stood in the outputs: append writes nothing after it, attention has no rows, the lengths stay."""
    n, ps, pages = len(new), 16, 64
    nw, cx, table, free, head = i32(new), i32(ctx), i32([[50] * 8] * n), i32([i % pages for i in range(free_n)]), i32([0])
    slots = torch.arange(T, device=DEV) % (pages * ps)
    pos, cu, kv, nxt, e = i32([7] * T), i32(list(range(n + 1))), i32([9] * n), i32([5]), errw()
    p = lambda x: x.data_ptr()  # noqa: E731
    rc = paged._lib().kda_paged_tables(p(nw), p(cx), n, T, p(table), 8, p(free), free_n, p(head), p(nxt), ps, pages, p(slots),
                                       p(pos), p(cu), p(kv), p(e), torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and int(e) == expect and int(nxt) == 0 and (table == 50).all()
    assert (slots == -1).all() and (pos == 0).all() and (cu == 0).all() and kv.tolist() == ctx
    T = min(T, 600)
    kc = torch.randn(pages, 1, ps, D, device=DEV).bfloat16()
    vc, x = kc.clone(), torch.zeros(T, 1, D, device=DEV, dtype=BF16)
    before = kc.clone()
    kda.paged_append(x, x, slots[:T].contiguous(), kc, vc)
    out = torch.full_like(x, 7.0)
    kda.paged_attn(x, kc, vc, table, cu, kv, out=out)
    assert torch.equal(kc, before) and torch.equal(vc, before) and (out == 7).all()


def test_tables_bad_pages():
    """A page outside the cache: its tokens get slot -1 and nothing else changes."""
    t = i32([[2, -1, -1], [99, -1, -1]])
    e = errw()
    slots, *_ = kda.paged_tables(i32([10, 3]), i32([10, 4]), t, i32([1, 77, 3]), i32([1]), 13, 16, 8, error_word=e)
    assert int(e) == paged.DEVERR_PAGE
    assert slots.tolist() == [2 * 16 + 10 + j for j in range(6)] + [-1] * 7
    assert t.tolist() == [[2, -1, -1], [99, -1, -1]]


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype,cache", [(BF16, BF16), (BF16, E4M3), (F32, F32)])
@pytest.mark.parametrize("T,hkv,ps", [(1, 1, 16), (37, 3, 48), (300, 8, 64)])
def test_append(T, hkv, ps, dtype, cache):
    g = torch.Generator().manual_seed(T)
    pages = cdiv(T, ps) + 4
    slots = torch.randperm(pages * ps, generator=g)[:T]
    slots[T // 2] = -1
    k, v = (torch.randn(T, hkv, D, generator=g).to(dtype) for _ in range(2))
    if T > 1:
        k[0, 0, :4] = torch.tensor([float("inf"), -1e30, 0.0, 1e-30], dtype=dtype)
    sc = {}
    if cache == E4M3:
        sc = {"k_scale": 0.01 + torch.rand(hkv, generator=g) / 50, "v_scale": 0.01 + torch.rand(hkv, generator=g) / 50}
    raw = {BF16: torch.int16, F32: torch.int32, E4M3: torch.uint8}[cache]
    # K and V as the two halves of one pool: pages lie apart
    pool = torch.randint(0, 100, (pages, 2, hkv, ps, D), dtype=raw, generator=g).to(DEV)
    want = pool.cpu().clone()
    for half, x, s in ((0, k, sc.get("k_scale")), (1, v, sc.get("v_scale"))):
        y = x.float() / s.view(1, -1, 1) if s is not None else x
        y = (y.clamp(-448, 448) if s is not None else y).to(cache).view(raw)
        for t in range(T):
            if slots[t] >= 0:
                want[slots[t] // ps, half, :, slots[t] % ps] = y[t]
    halves = pool.view(cache)
    e = errw()
    kda.paged_append(k.to(DEV), v.to(DEV), slots.to(DEV), halves[:, 0], halves[:, 1],
                     **{n: x.to(DEV) for n, x in sc.items()}, error_word=e)
    assert int(e) == 0 and torch.equal(pool.cpu(), want)


def test_append_skips_slots_outside_the_cache():
    c = torch.zeros(2, 1, 16, D, dtype=BF16, device=DEV)
    x = torch.ones(3, 1, D, dtype=BF16, device=DEV)
    e = errw()
    kda.paged_append(x, x, torch.tensor([32, 5, 1 << 40], device=DEV), c, c.clone(), error_word=e)
    assert int(e) == paged.DEVERR_PAGE
    assert c.sum().item() == D and c[0, 0, 5].sum().item() == D


# ------------------------------------------------------------------ attention
def run_attn(d, window=0, max_q=0, scale=D ** -0.5, **kw):
    t = {n: (x.to(DEV) if isinstance(x, torch.Tensor) else x) for n, x in d.items()}
    e = errw()
    o, lse = kda.paged_attn(t["q"], t["k_cache"], t["v_cache"], i32(d["table"]), i32(d["cu"]), i32(d["kv"]), max_q=max_q,
                            window=window, sm_scale=scale, k_scale=t["k_scale"], v_scale=t["v_scale"], error_word=e, **kw)
    torch.cuda.synchronize()
    return o, lse, int(e)


def check(new, ctx, hkv, g, ps, cache, window=0, kv=None, scale=D ** -0.5, seed=0, **kw):
    d = make(new, ctx, hkv, g, ps, cache, seed)
    if kv is not None:
        d["kv"] = kv
    o, lse, e = run_attn(d, window, max(new), scale, **kw)
    assert e == 0
    ref = attn_ref(d["q"], d["k_cache"], d["v_cache"], d["table"], d["cu"], d["kv"], scale, window, d["k_scale"], d["v_scale"])
    attn_close(o, lse, ref, d["q"].dtype, cache)
    return d, o, lse


CACHES = [BF16, E4M3, F32]
NAMES = ["bf16", "e4m3", "f32"]


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 31, 32, 63, 64, 65, 127, 700])
def test_attn_one_token(ctx, cache):
    check([1], [ctx], 2, 4, 16, cache)


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
@pytest.mark.parametrize("hkv,g", [(1, 1), (3, 5), (2, 16), (1, 17), (1, 33), (2, 8), (1, 96)])
def test_attn_head_layouts(hkv, g, cache):
    check([1, 2, 1], [40, 3, 130], hkv, g, 32, cache)


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
@pytest.mark.parametrize("ps", [16, 32, 48, 64, 80, 128, 256])
def test_attn_page_sizes(ps, cache):
    check([1, 5, 20, 0, 3], [300, 0, 77, 50, 129], 2, 3, ps, cache)


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
@pytest.mark.parametrize("new,ctx", [([33], [0]), ([70, 1], [5, 200]), ([130], [131]), ([1, 140, 2, 65], [90, 0, 0, 64])])
def test_attn_chunks(new, ctx, cache):
    check(new, ctx, 2, 3, 16, cache)


@pytest.mark.parametrize("hkv,g,new,ctx,ps,window", [
    (1, 1, [129], [0], 16, 0), (1, 1, [128, 257], [1, 127], 128, 0), (2, 4, [32, 33, 64, 65], [300, 0, 127, 128], 64, 0),
    (1, 8, [513], [1000], 48, 0), (1, 12, [5, 21, 22, 10], [130, 700, 0, 256], 16, 0), (2, 3, [300, 1], [511, 511], 32, 200),
    (1, 5, [260], [40], 16, 64), (1, 128, [1, 3], [200, 129], 16, 0), (1, 100, [2], [383], 96, 130), (4, 2, [400, 7, 90], [0, 900, 33], 256, 0)])
def test_attn_row_tiles(hkv, g, new, ctx, ps, window):
    """bf16 chunks around the sizes where rows and key tiles of 128 begin and end."""
    check(new, ctx, hkv, g, ps, BF16, window=window)


@pytest.mark.parametrize("new,ctx", [([40, 3, 64], [20000, 9000, 0]), ([2] * 9 + [150], [3000] * 9 + [10])])
def test_attn_row_tiles_split(new, ctx):
    """Few row tiles over long contexts: every item is cut by block borders."""
    d = make(new, ctx, 1, 8, 64, BF16, seed=5)
    o, lse, e = run_attn(d, max_q=max(new))
    assert e == 0
    attn_close(o, lse, attn_ref(d["q"], d["k_cache"], d["v_cache"], d["table"], d["cu"], d["kv"]), BF16, BF16)


def test_attn_row_tiles_of_both_kinds_in_one_block():
    """So many items that each block has several of one half and of two halves in turn."""
    new, ctx = [70, 20, 64, 33, 1, 90] * 25, [10, 150, 0, 300, 40, 5] * 25
    d = make(new, ctx, 2, 4, 16, BF16, seed=7)
    o, lse, e = run_attn(d, max_q=max(new))
    assert e == 0
    attn_close(o, lse, attn_ref(d["q"], d["k_cache"], d["v_cache"], d["table"], d["cu"], d["kv"]), BF16, BF16)


@pytest.mark.parametrize("new,ctx", [([1], [40]), ([3, 0, 1], [0, 9, 200])])
@pytest.mark.parametrize("g", [16, 17, 24, 130])
def test_attn_wide_groups(g, new, ctx):
    """Groups at and over the rows of the kernel for few, and over a tile's: bf16."""
    check(new, ctx, 2, g, 16, BF16, seed=18)


@pytest.mark.parametrize("new,ctx", [([197, 100], [3, 19]), ([132, 20, 196, 32], [500, 700, 0, 1000])])
def test_attn_row_tiles_of_both_kinds_in_turn(new, ctx):
    """Items of one half, over several tiles, right before and after items of two halves,
    again and again: each kind's scores stay its own."""
    k = 6
    d = make(new * k, ctx * k, 8, 4, 16, BF16, seed=14)
    ref = attn_ref(d["q"], d["k_cache"], d["v_cache"], d["table"], d["cu"], d["kv"])
    first = None
    for _ in range(10):
        o, lse, e = run_attn(d, max_q=max(new))
        assert e == 0
        first = first or (o, lse)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1])
    attn_close(o, lse, ref, BF16, BF16)


@pytest.mark.parametrize("g", [3, 5, 7])
def test_attn_row_tiles_same_bits(g):
    """Rows of a tile that are no query's hold what an earlier call left there: it has no say."""
    d = make([300, 33], [40, 900], 2, g, 16, BF16, seed=15)
    other = make([200, 200], [300, 0], 4, 1, 16, BF16, seed=16, q_std=40.0)
    o, lse, _ = run_attn(d)
    for i in range(30):
        run_attn({**other, "q": other["q"] * (1 + i % 7)})
        o2, lse2, _ = run_attn(d)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_attn_row_tiles_rising_scores():
    """Scores that grow with the key: the running maximum moves at every tile."""
    d = make([3], [1500], 1, 16, 32, BF16, q_std=1.0)
    k = d["k_cache"].float()
    for j in range(1503):
        k[d["table"][0][j // 32], 0, j % 32] = 0.02 * j * d["q"][0, 0].float() / 11.3 + 0.1 * k[d["table"][0][j // 32], 0, j % 32]
    d["k_cache"] = k.bfloat16()
    o, lse, e = run_attn(d)
    attn_close(o, lse, attn_ref(d["q"], d["k_cache"], d["v_cache"], d["table"], d["cu"], d["kv"]), BF16, BF16)


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
@pytest.mark.parametrize("window", [1, 2, 16, 33, 100, 1000])
def test_attn_window(window, cache):
    check([1, 4, 90], [300, 150, 60], 1, 2, 16, cache, window=window)


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
@pytest.mark.parametrize("new,ctx,kv", [([2, 5, 1], [300, 40, 9], None), ([5, 3, 30], [0, 0, 0], [2, 0, 7]),
                                        ([1, 140, 3], [90, 0, 64], None)])
def test_attn_window_without_limit(new, ctx, kv, cache):
    """A window that no position reaches, up to the largest number, is none."""
    d = make(new, ctx, 2, 2, 16, cache, seed=23)
    if kv is not None:
        d["kv"] = kv
    o, lse, e = run_attn(d)
    room = 16 * len(d["table"][0])
    for window in (max(d["kv"]), room - 1, room, 2 ** 31 - 65536, 2 ** 31 - 1):
        o2, lse2, e2 = run_attn(d, window=window)
        assert e == 0 and e2 == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
def test_attn_window_as_wide_as_the_widest_table(cache):
    """Queries so far before position 0 that their distance to the window's end passes 2^31."""
    ps, T = 65536, 140000
    d = make([5], [0], 1, 1, ps, cache, seed=24)
    width = (2 ** 31 - 65537) // ps
    d["table"] = [[d["table"][0][0]] + [-1] * (width - 1)]
    d["q"] = torch.cat([torch.zeros(T - 5, 1, D, dtype=d["q"].dtype), d["q"]])
    d["cu"] = [0, T]
    o, lse, e = run_attn(d)
    o2, lse2, e2 = run_attn(d, window=width * ps - 1)
    assert e == 0 and e2 == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)
    assert (o[:-5] == 0).all() and torch.isinf(lse[:-5]).all() and torch.isfinite(lse[-5:]).all()


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
def test_attn_window_pages_given_back(cache):
    """Pages that hold no seen key may have left the table."""
    d = make([1, 3], [500, 201], 2, 2, 16, cache)
    d2 = {**d, "table": [list(r) for r in d["table"]]}
    for i, (n, kv) in enumerate(zip([1, 3], d["kv"])):
        for b in range((kv - n - 50 + 1) // 16):
            d2["table"][i][b] = -9
    o, lse, e = run_attn(d, window=50)
    o2, lse2, e2 = run_attn(d2, window=50)
    assert e == 0 and e2 == 0 and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
@pytest.mark.parametrize("new", [1, 3, 20])
@pytest.mark.parametrize("ps", [16, 128])
def test_attn_window_hides_what_is_not_finite(ps, new, cache):
    """Keys and values before the window of the first new token, in its page too, have no influence."""
    window, ctx = 50, 310
    d = make([new], [ctx], 2, 2, ps, cache, seed=22)
    o, lse, e = run_attn(d, window=window)
    for key in range(ctx - window + 1):
        for c, x in (("k_cache", float("nan")), ("v_cache", float("nan") if cache == E4M3 or key % 2 else float("-inf"))):
            d[c][d["table"][0][key // ps], :, key % ps] = x
    o2, lse2, e2 = run_attn(d, window=window)
    assert e == 0 and e2 == 0 and torch.isfinite(o).all() and torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
def test_attn_rows_that_see_nothing(cache):
    """Fewer keys than new tokens: the first queries stand before position 0."""
    d, o, lse = check([5, 3, 40], [0, 0, 0], 2, 3, 16, cache, kv=[2, 0, 7])
    assert (o[:3] == 0).all() and (o[5:8] == 0).all() and torch.isinf(lse[5:8]).all()


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
@pytest.mark.parametrize("new", [1, 5, 20])
def test_attn_items_without_keys_between_others(new, cache):
    """Lines so long that a block has an item with keys, several without any, and items with keys again."""
    n, kind = 1190, [0, 1, 1, 1, 2, 1, 1]
    ctx = [900 + i % 50 if kind[i % 7] == 0 else 0 for i in range(n)]
    kv = [c + new if kind[i % 7] == 0 else 0 if kind[i % 7] == 1 else min(new, 3) for i, c in enumerate(ctx)]
    check([new] * n, ctx, 1, 2, 64, cache, kv=kv, seed=19)


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
def test_attn_split_over_blocks(cache):
    """Long contexts beside short ones: items cut by many block borders, and whole ones between."""
    check([1, 1, 2, 1], [9000, 10, 4100, 0], 2, 4, 64, cache, seed=3)


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
def test_attn_large_scores(cache):
    """A wide softmax range: probabilities far below the largest, and a maximum that moves late."""
    d = make([2], [600], 1, 2, 16, cache, q_std=6.0)
    o, lse, e = run_attn(d)
    attn_close(o, lse, attn_ref(d["q"], d["k_cache"], d["v_cache"], d["table"], d["cu"], d["kv"], k_scale=d["k_scale"],
                                v_scale=d["v_scale"]), d["q"].dtype, cache)


def test_attn_small_queries_e4m3():
    """q far below fp16's range: scaled by powers of two, nothing is lost."""
    d = make([1], [100], 1, 4, 16, E4M3)
    d["q"] = (d["q"].float() * 2.0 ** -40).bfloat16()
    scale = D ** -0.5 * 2.0 ** 40
    o, lse, e = run_attn(d, scale=scale)
    attn_close(o, lse, attn_ref(d["q"], d["k_cache"], d["v_cache"], d["table"], d["cu"], d["kv"], scale, 0, d["k_scale"],
                                d["v_scale"]), BF16, E4M3)


@pytest.mark.parametrize("new", [2, 5])
@pytest.mark.parametrize("outlier", [2.0 ** 6, 2.0 ** 8, 2.0 ** 10, 2.0 ** 12, 2.0 ** 14])
def test_attn_e4m3_query_with_one_large_channel(outlier, new):
    """The other channels keep their bits (its keys are zero there, so the others decide)."""
    d = make([new], [300], 2, 4, 16, E4M3, seed=21)
    d["q"][..., 5] *= outlier
    d["k_cache"][..., 5] = 0
    o, lse, e = run_attn(d)
    assert e == 0
    attn_close(o, lse, attn_ref(d["q"], d["k_cache"], d["v_cache"], d["table"], d["cu"], d["kv"], k_scale=d["k_scale"],
                                v_scale=d["v_scale"]), BF16, E4M3)


def test_attn_large_queries_e4m3():
    """q near the end of bf16's range: scaled by powers of two, nothing is cut."""
    d = make([2], [100], 1, 4, 16, E4M3)
    d["q"] = (d["q"].float() * 2.0 ** 114).bfloat16()
    scale = D ** -0.5 * 2.0 ** -114
    o, lse, e = run_attn(d, scale=scale)
    attn_close(o, lse, attn_ref(d["q"], d["k_cache"], d["v_cache"], d["table"], d["cu"], d["kv"], scale, 0, d["k_scale"],
                                d["v_scale"]), BF16, E4M3)


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
def test_attn_nan_stays_in_its_request(cache):
    d = make([1, 2], [50, 70], 1, 2, 16, cache)
    o, lse, _ = run_attn(d)
    d["k_cache"][d["table"][1][1], 0, 3, 5] = float("nan")
    o2, lse2, _ = run_attn(d)
    assert torch.equal(o[0], o2[0]) and torch.equal(lse[0], lse2[0])
    assert torch.isnan(o2[1:]).all()


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
@pytest.mark.parametrize("new", [1, 20])
def test_attn_nan_query_of_a_cut_item(new, cache):
    """A row whose scores are all NaN is NaN, whole or cut by block borders."""
    d = make([new, 1], [20000, 30], 1, 2, 64, cache, seed=20)
    d["q"][0, 1, 7] = d["q"][new, 0, 3] = float("nan")
    o, lse, e = run_attn(d, max_q=new)
    bad = torch.zeros(new + 1, 2, dtype=torch.bool)
    bad[0, 1] = bad[new, 0] = True
    assert e == 0 and torch.equal(torch.isnan(lse).cpu(), bad)
    assert torch.equal(torch.isnan(o).cpu(), bad[..., None].expand(-1, -1, D))


@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
def test_attn_pages_apart_and_same_bits(cache):
    """K and V as halves of one pool give the same bits as separate caches, run after run."""
    d = make([1, 40, 3], [3000, 60, 500], 2, 4, 32, cache, filler=0.0)
    o, lse, _ = run_attn(d)
    pool = torch.stack([d["k_cache"].view(torch.uint8), d["v_cache"].view(torch.uint8)], 1).to(DEV).view(cache)
    d2 = {**d, "k_cache": pool[:, 0], "v_cache": pool[:, 1]}
    for _ in range(3):
        o2, lse2, _ = run_attn(d2)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("new", [1, 2, 12])
def test_attn_f32_same_bits(new):
    """Tiles that most warps pass over, short items and cut ones: the same bits run after run."""
    n = 150
    d = make([new] * n, [(37 * i) % 400 for i in range(n - 1)] + [6000], 2, 2, 16, F32, seed=25)
    first = run_attn(d)
    attn_close(first[0], first[1], attn_ref(d["q"], d["k_cache"], d["v_cache"], d["table"], d["cu"], d["kv"]), F32, F32)
    for _ in range(40):
        o, lse, e = run_attn(d)
        assert e == 0 and torch.equal(o, first[0]) and torch.equal(lse, first[1])


def test_attn_other_stream_and_graph():
    d = make([1, 33], [700, 100], 2, 4, 16, BF16)
    o, lse, _ = run_attn(d)
    t = {n: (x.to(DEV) if isinstance(x, torch.Tensor) else x) for n, x in d.items()}
    args = (t["q"], t["k_cache"], t["v_cache"], i32(d["table"]), i32(d["cu"]), i32(d["kv"]))
    ws = torch.empty(kda.paged_attn_workspace_size(34, 2, 8, 2), dtype=torch.uint8, device=DEV)
    out, ol = torch.empty_like(o), torch.empty_like(lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        kda.paged_attn(*args, out=out, lse=ol, workspace=ws)
    side.synchronize()
    assert torch.equal(out, o) and torch.equal(ol, lse)
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.paged_attn(*args, out=out, lse=ol, workspace=ws)
    for _ in range(2):
        out.zero_()
        ws.fill_(255)  # the workspace needs no initialisation
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(ol, lse)


def test_attn_bad_lengths_are_recorded():
    """A request that cannot be is left out or counts as empty; the others are untouched."""
    d = make([1, 2, 1], [40, 50, 60], 1, 2, 16, BF16)
    o, lse, _ = run_attn(d)
    d2 = {**d, "kv": [d["kv"][0], 10 ** 6, d["kv"][2]]}
    o2, lse2, e2 = run_attn(d2)
    assert e2 == paged.DEVERR_LENGTHS
    assert torch.equal(o2[0], o[0]) and torch.equal(o2[3], o[3]) and (o2[1:3] == 0).all() and torch.isinf(lse2[1:3]).all()
    out = torch.full_like(o, 7.0)
    o3, _, e3 = run_attn({**d, "cu": [0, 1, 300, 4]}, out=out)
    assert e3 == 1 and torch.equal(o3[0], o[0]) and (o3[1:] == 7).all()
    out = torch.full_like(o, 7.0)
    o4, _, e4 = run_attn(d, max_q=1, out=out)
    assert e4 == 1 and torch.equal(o4[0], o[0]) and torch.equal(o4[3], o[3]) and (o4[1:3] == 7).all()


def test_step_runs_together():
    """tables, append and attention as a serving step calls them, over several
    steps: the cache ends as if the whole stream had been given at once."""
    hkv, g, ps, n = 2, 4, 16, 3
    gen = torch.Generator().manual_seed(9)
    steps = [[20, 5, 1], [1, 1, 1], [4, 0, 30], [1, 1, 1]]
    total = [sum(s[i] for s in steps) for i in range(n)]
    k = [torch.randn(t, hkv, D, generator=gen).bfloat16() for t in total]
    v = [torch.randn(t, hkv, D, generator=gen).bfloat16() for t in total]
    pages = 12
    kc, vc = (torch.full((pages, hkv, ps, D), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    table = torch.full((n, 8), -1, dtype=torch.int32, device=DEV)
    free, head, ctx = i32(torch.randperm(pages, generator=gen).tolist()), i32([0]), i32([0] * n)
    done = [0] * n
    for s in steps:
        T = sum(s)
        slots, pos, cu, kv, head = kda.paged_tables(i32(s), ctx, table, free, head, T, ps, pages)
        pick = lambda x: torch.cat([x[i][done[i]:done[i] + s[i]] for i in range(n)]).to(DEV)  # noqa: E731
        kda.paged_append(pick(k), pick(v), slots, kc, vc)
        q = torch.randn(T, hkv * g, D, generator=gen).bfloat16()
        o, lse = kda.paged_attn(q.to(DEV), kc, vc, table, cu, kv, max_q=max(s))
        ref = attn_ref(q, kc, vc, table.tolist(), cu.tolist(), kv.tolist())
        attn_close(o, lse, ref, BF16, BF16)
        ctx, done = kv, [a + b for a, b in zip(done, s)]
    assert head.tolist() == [sum(cdiv(t, ps) for t in total)]
    for i in range(n):
        got = kc[table[i, :cdiv(total[i], ps)].long()].permute(0, 2, 1, 3).reshape(-1, hkv, D)[:total[i]]
        assert torch.equal(got.cpu(), k[i])


def test_attn_page_outside_the_cache():
    """Recorded and never read; the other requests keep their results."""
    d = make([1, 1], [100, 100], 1, 2, 16, BF16)
    o, lse, _ = run_attn(d)
    for bad in (-1, 10 ** 6, d["k_cache"].shape[0]):
        t = [list(r) for r in d["table"]]
        t[1][2] = bad
        o2, lse2, e = run_attn({**d, "table": t})
        assert e == paged.DEVERR_PAGE and torch.equal(o2[0], o[0]) and torch.equal(lse2[0], lse[0])


# ------------------------------------------------------------------ many requests, long contexts
@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
def test_attn_many_requests(cache):
    """More requests than a block has threads: the line is scanned in several rounds."""
    n = 1500
    check([1] * n, [(7 * i) % 40 for i in range(n)], 1, 2, 16, cache, seed=11)


def test_attn_many_requests_of_both_kinds():
    n = 1400
    check([40 if i % 90 == 3 else i % 3 for i in range(n)], [(5 * i) % 30 for i in range(n)], 1, 2, 16, BF16, seed=12)


def _attn_ref_one(q, k, v, pos0, window):
    """One request's (o, lse, sum p |v|, largest score magnitude) in 64 bits on the GPU; k, v [S, D] of its one kv head."""
    T, g, _ = q.shape
    q, k, v = q.double(), k.double(), v.double()
    s = D ** -0.5 * (q.reshape(T * g, D) @ k.T)
    j = torch.arange(len(k), device=q.device)[None]
    p = (pos0 + torch.arange(T, device=q.device)).repeat_interleave(g)[:, None]
    s.masked_fill_((j > p) | ((j <= p - window) if window else (j < 0)), float("-inf"))
    lse = torch.logsumexp(s, 1)
    w = torch.exp_(s - lse[:, None])
    mag = D ** -0.5 * torch.stack([(x.abs() @ k.abs().T).amax(1) for x in q])
    return tuple(x.view(T, g, -1).cpu() for x in (w @ v, lse, w @ v.abs(), mag))


@pytest.mark.parametrize("window", [0, 90001])
def test_attn_context_longer_than_the_cache_of_the_gpu_holds(window):
    """Keys and values that a block's work passes in several parts, beside a short request."""
    new, ctx, g, ps = [300, 70], [140003, 21], 8, 64
    d = make(new, ctx, 1, g, ps, BF16, seed=13)
    o, lse, e = run_attn(d, window=window, max_q=max(new))
    assert e == 0
    ref = []
    for i in range(2):
        pages = torch.tensor(d["table"][i][:cdiv(d["kv"][i], ps)])
        k, v = (d[x][pages, 0].reshape(-1, D)[:d["kv"][i]].to(DEV) for x in ("k_cache", "v_cache"))
        ref.append(_attn_ref_one(d["q"][d["cu"][i]:d["cu"][i + 1]].to(DEV), k, v, ctx[i], window))
    o_ref, l_ref, a, mag = (torch.cat(x) for x in zip(*ref))
    attn_close(o, lse, (o_ref, l_ref[..., 0], a, mag[..., 0]), BF16, BF16)


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("g,new,cache", [(4, [1] * 24, BF16), (4, [1] * 24, E4M3), (4, [7] * 24, E4M3), (130, [1] * 24, BF16),
                                         (4, [60] * 24, BF16), (4, [200, 1, 40] * 8, BF16), (2, [1] * 24, F32), (2, [9] * 24, F32)])
def test_attn_wait_times_out_then_recovers(g, new, cache):
    """Waits of every role run out, early and late: the call records it, stays in its buffers
    and returns, and the next call is right."""
    d = make(new, [3000, 9000, 17, 500] * 6, 1, g, 64, cache, seed=26)
    o, lse, e = run_attn(d, max_q=max(new))
    out, ol = Guarded(o.shape, o.dtype), Guarded(lse.shape, F32)
    ws = Guarded((kda.paged_attn_workspace_size(sum(new), len(new), g, 1),), torch.uint8)
    codes = []
    for budget in (1, 100, 300, 700, 1500, 3000, 6000, 12000, 50000):
        old = kda.set_wait_budget(budget)
        try:
            codes.append(run_attn(d, max_q=max(new), out=out.t, lse=ol.t, workspace=ws.t)[2])
        finally:
            kda.set_wait_budget(old)
        assert codes[-1] in (0, 4) and out.intact() and ol.intact() and ws.intact()
        assert codes[-1] or (torch.equal(out.t, o) and torch.equal(ol.t, lse))
    assert e == 0 and codes[0] == 4
    o2, lse2, e = run_attn(d, max_q=max(new), out=out.t, lse=ol.t, workspace=ws.t)
    assert e == 0 and torch.equal(o2, o) and torch.equal(lse2, lse)


# ------------------------------------------------------------------ the two ways into the library
@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
def test_compiled_and_plain_binding_agree(cache, monkeypatch):
    """What the compiled way returns is what the plain one returns, and it does take these calls."""
    def go():
        new, ctx, hkv, g, ps, pages = [3, 0, 20], [14, 5, 0], 2, 4, 16, 8
        table, e = i32([[6, -1, -1], [7, -1, -1], [-1, -1, -1]]), errw()
        slots, pos, cu, kv, head = kda.paged_tables(i32(new), i32(ctx), table, i32([3, 1, 2, 0, 4]), i32([1]), 23, ps, pages,
                                                    error_word=e)
        gen = torch.Generator().manual_seed(2)
        qt = F32 if cache is F32 else BF16
        q = torch.randn(23, hkv * g, D, generator=gen).to(qt).to(DEV)
        k, v = (torch.randn(23, hkv, D, generator=gen).to(qt).to(DEV) for _ in range(2))
        kc, vc = (torch.zeros(pages, hkv, ps, D, device=DEV).to(cache) for _ in range(2))
        sc = dict(k_scale=torch.full((hkv,), 0.02, device=DEV), v_scale=torch.full((hkv,), 0.03, device=DEV)) if cache is E4M3 else {}
        kda.paged_append(k, v, slots, kc, vc, error_word=e, **sc)
        o, lse = kda.paged_attn(q, kc, vc, table, cu, kv, max_q=20, error_word=e, **sc)
        out, ol = torch.empty_like(o), torch.empty_like(lse)
        o2, lse2 = kda.paged_attn(q, kc, vc, table, cu, kv, out=out, lse=ol, **sc)
        assert o2.data_ptr() == out.data_ptr() and lse2.data_ptr() == ol.data_ptr()
        return table, slots, pos, cu, kv, head, kc.view(torch.uint8), vc.view(torch.uint8), o, lse, o2, lse2, e

    paged._lib()
    taken = []
    for name in ("tables", "append", "attn"):
        f = getattr(paged, "_fast_" + name)
        monkeypatch.setattr(paged, "_fast_" + name, lambda *a, f=f: (taken.append(r := f(*a)), r)[1])
    compiled = go()
    assert len(taken) == 4 and all(r is not None for r in taken)
    for name in ("tables", "append", "attn"):
        monkeypatch.setattr(paged, "_fast_" + name, lambda *a: None)
    for x, y in zip(compiled, go()):
        assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x, y)


def test_plain_binding_launches_on_the_tensors_device(monkeypatch):
    """Every call of the library is made with the tensors' device current, whichever was."""
    entered, real = [], torch.cuda.device

    class Device(real):
        def __enter__(self):
            entered.append(self.idx)
            super().__enter__()

    for name in ("tables", "append", "attn"):
        monkeypatch.setattr(paged, "_fast_" + name, lambda *a: None)
    monkeypatch.setattr(torch.cuda, "device", Device)
    lib, made = paged._lib(), []

    class Library:
        def __getattr__(self, name):
            made.append((name, list(entered)))
            return getattr(lib, name)

    monkeypatch.setattr(paged, "_declared", Library())
    e = errw()
    table = i32([[0, -1]])
    slots, pos, cu, kv, head = kda.paged_tables(i32([2]), i32([3]), table, i32([1]), i32([0]), 2, 16, 2, error_word=e)
    x, c = torch.ones(2, 1, D, dtype=BF16, device=DEV), torch.ones(2, 1, 16, D, dtype=BF16, device=DEV)
    kda.paged_append(x, x, slots, c, c.clone(), error_word=e)
    o, lse = kda.paged_attn(x, c, c, table, cu, kv, sm_scale=1, error_word=e)
    calls = [(n, d) for n, d in made if n in ("kda_paged_tables", "kda_paged_append", "kda_paged_attn")]
    index = torch.cuda.current_device()
    assert [n for n, _ in calls] == ["kda_paged_tables", "kda_paged_append", "kda_paged_attn"]
    assert [d for _, d in calls] == [[index] * (k + 1) for k in range(3)]
    assert int(e) == 0 and (o == 1).all()


def test_refusals_of_both_ways():
    """What the compiled way leaves undone, the plain one refuses, with its message."""
    d = make([2], [20], 2, 2, 16, BF16)
    t = {n: d[n].to(DEV) for n in ("q", "k_cache", "v_cache")}
    args = dict(q=t["q"], k_cache=t["k_cache"], v_cache=t["v_cache"], block_table=i32(d["table"]), cu_q=i32(d["cu"]),
                kv_len=i32(d["kv"]))
    kda.paged_attn(**args)
    for change, says in [
            (dict(q=t["q"][:, :3]), "contiguous"), (dict(q=t["q"].half()), "unsupported dtype"),
            (dict(cu_q=args["cu_q"].long()), "int32"), (dict(kv_len=i32([1, 2])), "cu_q must be"),
            (dict(block_table=args["block_table"].cpu()), "CUDA"), (dict(v_cache=t["v_cache"].float()), "same dtype"),
            (dict(k_scale=torch.ones(2, device=DEV)), "e4m3"), (dict(out=torch.empty_like(t["q"], dtype=F32)), "out must"),
            (dict(workspace=torch.empty(256, dtype=torch.uint8, device=DEV)), "WORKSPACE"), (dict(window=-1), "kda_paged_attn"),
            (dict(q=t["q"][:, :3].contiguous()), "kda_paged_attn")]:
        with pytest.raises(kda.KDAError, match=says):
            kda.paged_attn(**{**args, **change})


# ------------------------------------------------------------------ guard bytes
@pytest.mark.parametrize("cache", CACHES, ids=NAMES)
@pytest.mark.parametrize("new,ctx", [([1, 1], [0, 3000]), ([37, 0, 1], [5, 9, 700]), ([130, 33], [2000, 0])])
def test_writes_only_its_buffers(new, ctx, cache):
    """The step's outputs, caches and workspace between pattern bytes, which stay; and the bits of a plain call."""
    hkv, g, ps, n, T = 2, 3, 16, len(new), sum(new)
    d = make(new, ctx, hkv, g, ps, cache, seed=17)
    qt = d["q"].dtype
    width, pages = len(d["table"][0]), d["k_cache"].shape[0]
    table = Guarded((n, width), torch.int32, i32(d["table"]))
    kc, vc = (Guarded(d[x].shape, cache, d[x].to(DEV)) for x in ("k_cache", "v_cache"))
    o, lse = Guarded(d["q"].shape, qt), Guarded((T, hkv * g), F32)
    ws = Guarded((kda.paged_attn_workspace_size(T, n, hkv * g, hkv),), torch.uint8)
    slots, pos = Guarded((T,), torch.int64), Guarded((T,), torch.int32)
    cu, kv, head = Guarded((n + 1,), torch.int32), Guarded((n,), torch.int32), Guarded((1,), torch.int32)
    err = Guarded((1,), torch.int32, i32([0]))
    bufs = [table, kc, vc, o, lse, ws, slots, pos, cu, kv, head, err]
    first_new = [t[cdiv(c, ps):cdiv(c + a, ps)] for t, a, c in zip(d["table"], new, ctx)]
    free = i32([p for ps_ in first_new for p in ps_] + [0])
    lib, stream, p = paged._lib(), torch.cuda.current_stream().cuda_stream, lambda x: x.t.data_ptr()
    nw, cx, h0 = i32(new), i32(ctx), i32([0])
    assert lib.kda_paged_tables(nw.data_ptr(), cx.data_ptr(), n, T, p(table), width, free.data_ptr(), free.numel(),
                                h0.data_ptr(), p(head), ps, pages, p(slots), p(pos), p(cu), p(kv), p(err), stream) == 0
    torch.cuda.synchronize()
    assert table.t.tolist() == d["table"] and kv.t.tolist() == d["kv"] and cu.t.tolist() == d["cu"] and int(err.t) == 0
    rest, lrest, _ = run_attn(d, max_q=max(new))
    k, v = (torch.randn(T, hkv, D, device=DEV).to(qt) for _ in range(2))
    ks, vs = (None if d[x] is None else d[x].to(DEV) for x in ("k_scale", "v_scale"))
    q = d["q"].to(DEV)
    o2, lse2 = kda.paged_attn(q, kc.t, vc.t, table.t, cu.t, kv.t, max_q=max(new), k_scale=ks, v_scale=vs, out=o.t, lse=lse.t,
                              workspace=ws.t, error_word=err.t)
    torch.cuda.synchronize()
    assert torch.equal(o2, rest) and torch.equal(lse2, lrest) and int(err.t) == 0
    kda.paged_append(k, v, slots.t, kc.t, vc.t, k_scale=ks, v_scale=vs, error_word=err.t)
    torch.cuda.synchronize()
    assert int(err.t) == 0 and all(b.intact() for b in bufs)
    assert torch.equal(q, d["q"].to(DEV))


# ------------------------------------------------------------------ together
def test_hybrid_example():
    """Chunks and single tokens through both kinds of layer against one pass: a few roundings
    to bf16 (2^-9 on average) on the way of each output."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "hybrid_serving.py")
    spec = importlib.util.spec_from_file_location("hybrid_serving", path)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    assert example.main() < 1e-2
