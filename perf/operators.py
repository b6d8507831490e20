"""The paged key/value cache of the full-attention layers that a hybrid model
puts between its linear-attention layers: what one serving step asks of it.

  tables  block tables, slot map, positions and offsets of a step's new tokens,
          built on the GPU from the requests' lengths and a list of free pages
  append  the new tokens' keys and values written into the cache's pages
  attn    attention of each request's chunk of new tokens (from a single token
          to a whole prompt) over its cached keys, through the block table

Caches are [pages, kv heads, page size, 128] (a head's part of a page is one
contiguous block); queries, new keys and new values are [tokens, heads, 128].
Request i's n new tokens stand at positions kv_len - n .. kv_len - 1; a query at
position p sees the keys at positions p - window + 1 .. p (all up to p without a
window).  An e4m3 cache holds x / scale, one scale for each kv head.
"""
import math

import numpy as np
import torch

own = False  # False: elementary torch operations; True: the library's kernels

DEV = "cuda"
HEAD = 128
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


# ----------------------------------------------------------------- the cases
def _case(op, **kw):
    c = {"op": op, "n": 1, "singles": 0, "new_lo": 1, "new_hi": 1, "ctx_lo": 0, "ctx_hi": 0, "hq": 16, "hkv": 2,
         "page": 64, "dtype": "bf16", "cache": "bf16", "window": 0, "lens": 1}
    c.update(kw)
    return c


def listed():
    return [
        # the bookkeeping of a decode step of 256 sequences: latency alone
        _case("tables", name="tables_decode", n=256, ctx_lo=512, ctx_hi=16384, lens=11),
        # the same for a million prompt tokens queued at once (pages of 16)
        _case("tables", name="tables_prefill_1m", n=150, new_lo=3000, new_hi=13000, page=16, lens=12),
        # a decode step with windows of five tokens (four drafts), e4m3 cache
        _case("append", name="append_mtp_e4m3", n=256, new_lo=5, new_hi=5, ctx_lo=100, ctx_hi=2000, hkv=8,
              cache="e4m3", lens=13),
        # 32768 packed prompt tokens of ragged documents
        _case("append", name="append_packed_32k", n=11, new_lo=600, new_hi=8192, hkv=8, page=16, lens=14),
        # one stream's next token: the smallest call
        _case("attn", name="attn_one_token", ctx_lo=8191, ctx_hi=8191, lens=15),
        # a batch of 256 sequences of very different lengths, one token each
        _case("attn", name="attn_decode_ragged", n=256, ctx_lo=512, ctx_hi=16384, hq=32, hkv=4, lens=16),
        # speculative windows of five tokens over 96 query heads
        _case("attn", name="attn_decode_mtp", n=256, new_lo=5, new_hi=5, ctx_lo=256, ctx_hi=4096, hq=96, hkv=8, lens=17),
        # long contexts in an e4m3 cache
        _case("attn", name="attn_decode_e4m3", n=64, ctx_lo=4096, ctx_hi=65535, hq=32, hkv=8, cache="e4m3", lens=18),
        # fp32 inputs, as the fp32 decode of the linear layers, no sharing of heads
        _case("attn", name="attn_decode_f32", n=16, ctx_lo=100, ctx_hi=3000, hq=16, hkv=16, page=16, dtype="f32",
              cache="f32", lens=19),
        # a whole prompt of 8192 tokens, 16 heads
        _case("attn", name="attn_prompt_8k", new_lo=8192, new_hi=8192, lens=20),
        # the last chunk of a 64k prompt: the largest
        _case("attn", name="attn_chunk_64k", new_lo=2048, new_hi=2048, ctx_lo=63488, ctx_hi=63488, hq=32, hkv=8, lens=21),
        # single tokens and odd chunks in one batch, a sliding-window layer, small pages
        _case("attn", name="attn_mixed_window", n=32, singles=24, new_lo=50, new_hi=1023, ctx_lo=1, ctx_hi=3000, hq=32,
              hkv=8, page=16, window=1024, lens=22),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["tables", "append", "attn", "attn", "attn", "attn"])
        page = rng.choice([16, 32, 64, 128])
        lens = rng.randrange(1 << 20)
        if op == "tables":
            n = _log_int(rng, 1, 512)
            hi = rng.choice([1, 5, _log_int(rng, 10, 8000)])
            c = _case(op, n=n, new_lo=1 if hi < 6 else hi // 3, new_hi=hi, ctx_hi=_log_int(rng, 1, 16384), page=page, lens=lens)
        elif op == "append":
            n = _log_int(rng, 1, 256)
            hi = _log_int(rng, 1, max(1, 20000 // n))
            c = _case(op, n=n, new_lo=max(1, hi // 3), new_hi=hi, ctx_hi=_log_int(rng, 1, 500), hkv=rng.choice([1, 2, 4, 8]),
                      page=page, cache=rng.choice(["bf16", "e4m3"]), lens=lens)
        else:
            hkv = rng.choice([1, 2, 4, 8])
            kind = rng.choice(["decode", "window", "chunk", "mixed", "f32"])
            kw = {"hkv": hkv, "hq": hkv * rng.choice([1, 2, 3, 4, 5, 8]), "page": page, "lens": lens,
                  "window": rng.choice([0, 0, 0, 512])}
            if kind == "decode":
                kw |= {"n": _log_int(rng, 1, 200), "ctx_lo": 64, "ctx_hi": _log_int(rng, 100, 16000),
                       "cache": rng.choice(["bf16", "e4m3"])}
            elif kind == "window":
                kw |= {"n": _log_int(rng, 1, 200), "new_lo": 2, "new_hi": rng.randint(2, 8),
                       "ctx_hi": _log_int(rng, 100, 8000), "cache": rng.choice(["bf16", "e4m3"])}
            elif kind == "chunk":
                hi = _log_int(rng, 33, 8192)
                kw |= {"n": rng.choice([1, 1, 2, 3, 5]), "new_lo": max(1, hi // 2), "new_hi": hi,
                       "ctx_hi": _log_int(rng, 1, 30000)}
            elif kind == "mixed":
                hi = _log_int(rng, 33, 1200)
                n = rng.randint(4, 32)
                kw |= {"n": n, "singles": rng.randint(1, n - 1), "new_lo": max(1, hi // 8), "new_hi": hi,
                       "ctx_hi": _log_int(rng, 10, 3000)}
            else:
                kw |= {"n": _log_int(rng, 1, 32), "new_hi": rng.choice([1, 5, 40]), "ctx_hi": _log_int(rng, 10, 3000),
                       "dtype": "f32", "cache": "f32"}
            c = _case(op, **kw)
            new, ctx = _lengths(c)
            kv = int((new + ctx).max())
            if c["n"] * c["hq"] * int(new.max()) * kv > 4.3e9 or c["n"] * hkv * kv * HEAD > 4e9:
                continue
        w, top = work(c), [work(x) for x in listed() if x["op"] == op]
        if w["bytes"] <= max(x["bytes"] for x in top) and w["flops"] <= max(x["flops"] for x in top):
            return c


def _lengths(case):
    """New tokens and tokens already cached, request by request (from the case alone)."""
    r = np.random.RandomState(case["lens"])

    def some(lo, hi):
        return np.clip(np.round(np.exp(r.uniform(np.log(lo + 1), np.log(hi + 1), case["n"]))) - 1, lo, hi).astype(np.int64)

    new, ctx = some(case["new_lo"], case["new_hi"]), some(case["ctx_lo"], max(case["ctx_lo"], case["ctx_hi"]))
    new[:case["singles"]] = 1
    return new, ctx


def _pairs(case, new, ctx):
    """Query/key pairs that the masks leave, one head."""
    total = 0
    for n, c in zip(new.tolist(), ctx.tolist()):
        lo, hi = c + 1, c + n  # keys seen by the first and the last query without a window
        w = case["window"] or hi
        full = max(0, hi - max(lo, w) + 1) if hi >= w else 0  # queries that see w keys
        part = n - full
        total += full * w + part * lo + part * (part - 1) // 2
    return total


def work(case):
    new, ctx = _lengths(case)
    T, n, h, page = int(new.sum()), case["n"], case["hkv"], case["page"]
    blocks = -(-(new + ctx) // page)
    fresh = int((blocks - -(-ctx // page)).sum())
    if case["op"] == "tables":  # lengths, free pages in; table entries, slots, positions, offsets out
        return {"bytes": 8 * n + 4 * fresh + 4 * fresh + 8 * T + 4 * T + 4 * (n + 1) + 4 * n, "flops": 0}
    if case["op"] == "append":
        return {"bytes": 2 * T * h * HEAD * (BYTES[case["dtype"]] + BYTES[case["cache"]]) + 8 * T, "flops": 0}
    seen = new + ctx
    if case["window"]:
        seen = np.minimum(seen, new + case["window"] - 1)
    byte = 2 * T * case["hq"] * HEAD * BYTES[case["dtype"]] + 4 * T * case["hq"] + 4 * int((-(-seen // page)).sum()) + 8 * n
    byte += 2 * int(seen.sum()) * h * HEAD * BYTES[case["cache"]]
    return {"bytes": byte, "flops": 4 * HEAD * case["hq"] * _pairs(case, new, ctx)}


# ----------------------------------------------------------------- the state
def prepare(case, seed):
    new, ctx = _lengths(case)
    n, page, h = case["n"], case["page"], case["hkv"]
    T, blocks, had = int(new.sum()), -(-(new + ctx) // page), -(-ctx // page)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    width = int(blocks.max())
    pages = int(blocks.sum()) + max(4, n)  # a few stay free
    shuffled = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    owned = had if case["op"] == "tables" else blocks
    col = torch.arange(width, device=DEV)
    start = torch.from_numpy(np.concatenate([[0], np.cumsum(owned)[:-1]])).to(DEV)
    at = start[:, None] + col[None, :]
    table = torch.where(col[None, :] < torch.from_numpy(owned).to(DEV)[:, None], shuffled[at.clamp(max=pages - 1)],
                        torch.full_like(at, -1, dtype=torch.int32))
    s = {"case": dict(case), "T": T, "pages": pages, "table": table, "max_new": int(new.max()), "max_kv": int((new + ctx).max())}
    s["new"] = torch.from_numpy(new).to(DEV, torch.int32)
    s["ctx"] = torch.from_numpy(ctx).to(DEV, torch.int32)
    s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).to(DEV, torch.int32)
    s["kv_len"] = s["new"] + s["ctx"]
    if case["op"] == "tables":
        s["free"] = shuffled[int(had.sum()):].contiguous()
        s["head"] = torch.randint(0, 3, (1,), generator=g, device=DEV, dtype=torch.int32)  # a few are taken already
        return s
    cache = TYPES[case["cache"]]
    x = lambda *size: torch.randn(size, generator=g, device=DEV)  # noqa: E731
    kc, vc = x(pages, h, page, HEAD), x(pages, h, page, HEAD)
    if case["cache"] == "e4m3":  # scales as a calibration on the layer's largest values gives them
        s["k_scale"] = (3.5 + x(h).abs()) / 448
        s["v_scale"] = (3.5 + x(h).abs()) / 448
        kc, vc = (t.div_(sc.view(1, h, 1, 1)).clamp_(-448, 448) for t, sc in ((kc, s["k_scale"]), (vc, s["v_scale"])))
    s["k_cache"], s["v_cache"] = kc.to(cache), vc.to(cache)
    del kc, vc
    if case["op"] == "append":
        i = torch.repeat_interleave(torch.arange(n, device=DEV), s["new"].long())
        pos = s["ctx"].long()[i] + torch.arange(T, device=DEV) - s["cu"].long()[i]
        s["slots"] = table[i, pos // page].long() * page + pos % page
        s["k"], s["v"] = x(T, h, HEAD).to(TYPES[case["dtype"]]), x(T, h, HEAD).to(TYPES[case["dtype"]])
        return s
    s["q"] = (2 * x(T, case["hq"], HEAD)).to(TYPES[case["dtype"]])
    if own:  # what a program keeps between calls
        import linear_attention_serving_gb300 as kda
        s["ws"] = torch.empty(kda.paged_attn_workspace_size(T, n, case["hq"], h), dtype=torch.uint8, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"tables": _tables_own, "append": _append_own, "attn": _attn_own}[op](s)
    return {"tables": _tables, "append": _append, "attn": _attn}[op](s)


def _tables_own(s):
    import linear_attention_serving_gb300 as kda
    slots, pos, cu, kv, head = kda.paged_tables(s["new"], s["ctx"], s["table"], s["free"], s["head"], s["T"],
                                                s["case"]["page"], s["pages"])
    return {"table": s["table"], "slots": slots, "pos": pos, "cu": cu, "kv_len": kv, "head": head}


def _append_own(s):
    import linear_attention_serving_gb300 as kda
    kda.paged_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attn_own(s):
    import linear_attention_serving_gb300 as kda
    o, lse = kda.paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"], max_q=s["max_new"],
                            window=s["case"]["window"], k_scale=s.get("k_scale"), v_scale=s.get("v_scale"), workspace=s["ws"])
    return {"o": o, "lse": lse}


def _tables(s):
    new, ctx, page, T, table = s["new"].long(), s["ctx"].long(), s["case"]["page"], s["T"], s["table"]
    had, have = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    first = s["head"].long() + torch.cumsum(have - had, 0) - (have - had)  # each request's first fresh page in the list
    cu = torch.nn.functional.pad(torch.cumsum(new, 0), (1, 0))
    col = torch.arange(table.shape[1], device=table.device)[None, :]
    fresh = (col >= had[:, None]) & (col < have[:, None])
    at = (first[:, None] + col - had[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], table)
    t = torch.arange(T, device=table.device)
    i = torch.repeat_interleave(torch.arange(new.numel(), device=table.device), new, output_size=T)
    pos = ctx[i] + t - cu[i]
    slots = table[i, pos // page].long() * page + pos % page
    return {"table": table, "slots": slots, "pos": pos.int(), "cu": cu.int(), "kv_len": (ctx + new).int(),
            "head": s["head"] + (have - had).sum().int()}


def _stored(x, scale, to):
    """Values as the cache holds them."""
    if scale is not None:
        x = (x.float() / scale.view(1, -1, 1)).clamp(-448, 448)
    return x.to(to)


def _append(s):
    page, slots = s["case"]["page"], s["slots"]
    for new, cache, scale in (("k", "k_cache", "k_scale"), ("v", "v_cache", "v_scale")):
        held = _stored(s[new], s.get(scale), s[cache].dtype)
        raw = torch.uint8 if held.dtype == torch.float8_e4m3fn else held.dtype  # rows are moved as they are
        s[cache].view(raw)[slots // page, :, slots % page] = held.view(raw)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _gathered(cache, table, scale):
    """A request's keys (or values) in order: [n, kv heads, width x page, 128] in 32 bits."""
    n, width = table.shape
    x = cache[table.clamp(min=0).long()].float()
    if scale is not None:
        x *= scale.view(1, 1, -1, 1, 1)
    return x.transpose(1, 2).reshape(n, cache.shape[1], width * cache.shape[2], HEAD)


def _attn(s):
    c, table, q, T = s["case"], s["table"], s["q"], s["T"]
    n, hq, hkv, m, kv = c["n"], c["hq"], c["hkv"], s["max_new"], s["max_kv"]
    g = hq // hkv
    kv_len, cu = s["kv_len"].long(), s["cu"].long()
    new = cu[1:] - cu[:-1]
    t = torch.arange(T, device=q.device)
    i = torch.repeat_interleave(torch.arange(n, device=q.device), new, output_size=T)
    row = t - cu[i]
    padded = torch.zeros(n, m, hq, HEAD, device=q.device)
    padded[i, row] = q.float()
    padded = padded.view(n, m, hkv, g, HEAD).permute(0, 2, 1, 3, 4).reshape(n, hkv, m * g, HEAD)
    k = _gathered(s["k_cache"], table, s.get("k_scale"))[:, :, :kv]
    x = torch.matmul(padded * HEAD ** -0.5, k.transpose(2, 3))  # [n, hkv, m g, kv]
    del k
    pos = (kv_len - new)[:, None] + torch.arange(m, device=q.device)[None, :]
    key = torch.arange(kv, device=q.device)
    hidden = key > pos[:, :, None]
    if c["window"]:
        hidden |= key <= pos[:, :, None] - c["window"]
    x.view(n, hkv, m, g, kv).masked_fill_(hidden[:, None, :, None, :], -math.inf)
    top = x.amax(3, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    x.sub_(top).exp_()
    total = x.sum(3, keepdim=True)
    v = _gathered(s["v_cache"], table, s.get("v_scale"))[:, :, :kv]
    o = torch.matmul(x, v) / torch.where(total > 0, total, torch.ones_like(total))
    lse = top + total.log()
    o = o.view(n, hkv, m, g, HEAD).permute(0, 2, 1, 3, 4).reshape(n, m, hq, HEAD)[i, row]
    lse = lse.view(n, hkv, m, g).permute(0, 2, 1, 3).reshape(n, m, hq)[i, row]
    return {"o": o.to(q.dtype), "lse": lse}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    page, d = case["page"], torch.float64
    if case["op"] == "append":
        out = {}
        for new, cache, scale in (("k", "k_cache", "k_scale"), ("v", "v_cache", "v_scale")):
            x, y = s[new].to(d), s[cache].to(d)
            if scale in s:
                x = x / s[scale].to(d)[None, :, None]
            y[torch.div(s["slots"], page, rounding_mode="floor"), :, s["slots"] % page] = x
            out[cache] = y
        return out
    cu, lens = s["cu"].tolist(), s["kv_len"].tolist()
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    o = torch.zeros(s["T"], case["hq"], HEAD, dtype=d, device=DEV)
    lse = torch.full((s["T"], case["hq"]), -math.inf, dtype=d, device=DEV)
    for i in range(case["n"]):
        a, b, kv = cu[i], cu[i + 1], lens[i]
        pages = s["table"][i, :-(-kv // page)].long()
        pos = torch.arange(kv - (b - a), kv, device=DEV)
        key = torch.arange(kv, device=DEV)
        seen = key[None, :] <= pos[:, None]
        if case["window"]:
            seen &= pos[:, None] - key[None, :] < case["window"]
        for h in range(hkv):
            k = s["k_cache"][pages, h].to(d).reshape(-1, HEAD)[:kv]
            v = s["v_cache"][pages, h].to(d).reshape(-1, HEAD)[:kv]
            if "k_scale" in s:
                k, v = k * s["k_scale"][h].to(d), v * s["v_scale"][h].to(d)
            heads = slice(h * g, h * g + g)
            z = torch.einsum("thd,kd->htk", s["q"][a:b, heads].to(d), k) / math.sqrt(HEAD)
            z = torch.where(seen[None], z, torch.full((), -math.inf, dtype=d, device=DEV))
            l = torch.logsumexp(z, 2)
            p = torch.where(seen[None], torch.exp(z - l[..., None]), torch.zeros((), dtype=d, device=DEV))
            o[a:b, heads] = torch.einsum("htk,kd->thd", p, v)
            lse[a:b, heads] = l.T
    return {"o": o, "lse": lse}
