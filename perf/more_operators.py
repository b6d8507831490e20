"""What a served step with drafted tokens asks for beside the paged cache's append
and attention:

  rope    queries and keys normed for each head (RMS, with weights) and turned by
          their positions, from the packed projection
  append  the same, the keys written straight into the cache's pages with the values
  attn    attention over the paged cache through a sliding window, with the first
          few tokens (sinks) visible to every query
  verify  drafted tokens against the target's probabilities, by given uniform
          numbers: how many stand, and the token after them

Heads have 128 channels.  The projection is [tokens, q heads + 2 kv heads, 128];
caches are [pages, kv heads, page size, 128], an e4m3 cache holds x / scale.
"""
import math

import numpy as np
import torch

own = False  # False: elementary torch operations; True: the library's kernels

DEV = "cuda"
HEAD = 128
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "e4m3": 1}


# ----------------------------------------------------------------- the cases
def _case(op, **kw):
    c = {"op": op, "n": 1, "lens": 1, "dtype": "bf16"}
    if op == "verify":  # drafts w - 1; the draft's probabilities, or one certain token each; flat: how spread p is
        c |= {"w": 5, "vocab": 32768, "greedy": False, "ragged": False, "dtype": "f32", "flat": 3.0, "noise": 0.7}
    else:
        c |= {"singles": 0, "new_lo": 1, "new_hi": 1, "ctx_lo": 0, "ctx_hi": 0, "hq": 16, "hkv": 2}
    if op in ("rope", "append"):
        c |= {"rot": 128, "pairs": False, "norm": True, "base": 10000.0, "scaling": "none", "factor": 1.0, "original": 0}
    if op in ("append", "attn"):
        c |= {"page": 64, "cache": "bf16"}
    if op == "attn":
        c |= {"window": 1024, "sinks": 4}
    c.update(kw)
    return c


def listed():
    return [
        # one stream's next token: the smallest call
        _case("rope", name="rope_one_token", ctx_lo=8191, ctx_hi=8191, lens=31),
        # packed ragged prompts in fp32, half of the head turned, pairs side by side, no norm
        _case("rope", name="rope_packed_f32", n=7, new_lo=300, new_hi=2500, ctx_hi=30000, hq=16, hkv=16, dtype="f32", rot=64,
              pairs=True, norm=False, lens=32),
        # windows of five tokens (four drafts) of 256 requests far into a stretched context, e4m3 cache
        _case("append", name="append_mtp_e4m3", n=256, new_lo=5, new_hi=5, ctx_lo=100, ctx_hi=120000, hq=32, hkv=8, cache="e4m3",
              scaling="yarn", factor=16.0, original=8192, lens=33),
        # 32768 packed prompt tokens of ragged documents: the largest of its kind
        _case("append", name="append_packed_32k", n=11, new_lo=600, new_hi=8192, hq=32, hkv=8, page=16, lens=34),
        # a batch of 256 sequences of very different lengths, one token each, through a window
        _case("attn", name="attn_sinks_decode", n=256, ctx_lo=512, ctx_hi=16384, hq=32, hkv=4, window=2048, sinks=4, lens=35),
        # draft windows over long contexts in an e4m3 cache
        _case("attn", name="attn_sinks_mtp_e4m3", n=64, new_lo=5, new_hi=5, ctx_lo=4096, ctx_hi=65000, hq=32, hkv=8,
              cache="e4m3", window=4096, sinks=64, lens=36),
        # fp32, as the fp32 decode of the linear layers, no sharing of heads
        _case("attn", name="attn_sinks_f32", n=16, ctx_lo=100, ctx_hi=3000, hq=16, hkv=16, page=16, dtype="f32", cache="f32",
              window=500, sinks=10, lens=37),
        # single tokens and odd chunks in one batch, small pages
        _case("attn", name="attn_sinks_mixed", n=32, singles=24, new_lo=50, new_hi=1023, ctx_lo=1, ctx_hi=3000, hq=32, hkv=8,
              page=16, window=700, sinks=5, lens=38),
        # the last chunk of a 64k prompt: the largest
        _case("attn", name="attn_sinks_chunk_64k", new_lo=2048, new_hi=2048, ctx_lo=63488, ctx_hi=63488, hq=32, hkv=8,
              window=4096, sinks=4, lens=39),
        # four drafts of one stream
        _case("verify", name="verify_one", lens=40),
        # a batch of 256 with four drafts each
        _case("verify", name="verify_batch", n=256, vocab=131072, lens=41),
        # drafts without probabilities (a lookup's, say), some requests with fewer, an odd vocabulary, bf16
        _case("verify", name="verify_certain_ragged", n=64, w=8, vocab=100003, greedy=True, ragged=True, dtype="bf16", noise=0.3,
              lens=42),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    while True:
        op = rng.choice(["rope", "append", "attn", "attn", "verify"])
        lens = rng.randrange(1 << 20)
        if op == "verify":
            c = _case(op, n=_log_int(rng, 1, 256), w=rng.randint(2, 8), vocab=_log_int(rng, 1000, 200000),
                      greedy=rng.random() < 0.3, ragged=rng.random() < 0.4, dtype=rng.choice(["f32", "f32", "bf16"]),
                      flat=rng.uniform(1.0, 4.0), noise=rng.uniform(0.1, 1.5), lens=lens)
            if rng.random() < 0.5:
                c["vocab"] = max(16, c["vocab"] // 64 * 64)
        elif op in ("rope", "append"):
            hkv = rng.choice([1, 2, 4, 8])
            n = _log_int(rng, 1, 256)
            hi = _log_int(rng, 1, max(1, 20000 // n))
            kw = {"n": n, "new_lo": max(1, hi // 3), "new_hi": hi, "hkv": hkv, "hq": hkv * rng.choice([1, 2, 3, 4, 5, 8]),
                  "rot": rng.choice([32, 64, 96, 128, 128]), "pairs": rng.random() < 0.4, "norm": rng.random() < 0.6,
                  "base": rng.choice([10000.0, 500000.0]), "lens": lens}
            if rng.random() < 0.5:
                kw |= {"scaling": rng.choice(["linear", "ntk", "yarn"]), "factor": rng.choice([2.0, 8.0, 40.0]), "original": 4096}
            if op == "rope":
                c = _case(op, dtype=rng.choice(["bf16", "bf16", "f32"]), ctx_hi=_log_int(rng, 1, 900000), **kw)
            else:
                c = _case(op, page=rng.choice([16, 32, 64, 128]), ctx_hi=_log_int(rng, 1, 500), **kw)
                c["cache"] = rng.choice(["bf16", "e4m3", "f32"])
                if c["cache"] == "f32":
                    c["dtype"] = "f32"
        else:
            hkv = rng.choice([1, 2, 4, 8])
            kind = rng.choice(["decode", "window", "chunk", "mixed", "f32"])
            kw = {"hkv": hkv, "hq": hkv * rng.choice([1, 2, 3, 4, 5, 8]), "page": rng.choice([16, 32, 64, 128]), "lens": lens,
                  "window": _log_int(rng, 20, 8000), "sinks": _log_int(rng, 1, 600)}
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
            if c["n"] * c["hq"] * int(new.max()) * kv > 4.3e9 or c["n"] * hkv * kv * HEAD > 2.2e9:
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


def _drafts(case):
    """Drafts of each request."""
    m = case["w"] - 1
    if not case["ragged"]:
        return np.full(case["n"], m, dtype=np.int64)
    return np.random.RandomState(case["lens"]).randint(0, m + 1, case["n"]).astype(np.int64)


def _pairs(case, new, ctx):
    """Query/key pairs that the masks leave, one head."""
    total = 0
    for n, c in zip(new.tolist(), ctx.tolist()):
        p = np.arange(c, c + n)
        lo = np.maximum(0, p - case["window"] + 1)
        total += int((p + 1 - lo + np.minimum(lo, case["sinks"])).sum())
    return total


def work(case):
    if case["op"] == "verify":
        # the target's row that the token comes from, and the draft's where that is a refused draft's (as good
        # as every request of a long window has one); one number of each row for the tests
        m = int(_drafts(case).sum())
        rows = case["n"] * (1 if case["greedy"] else 2)
        es = BYTES[case["dtype"]]
        byte = rows * case["vocab"] * es + m * (4 + 4 + es * (1 if case["greedy"] else 2)) + case["n"] * (8 + 4 * case["w"])
        return {"bytes": byte, "flops": 3 * rows * case["vocab"]}
    new, ctx = _lengths(case)
    T, hq, hkv, es = int(new.sum()), case["hq"], case["hkv"], BYTES[case["dtype"]]
    if case["op"] in ("rope", "append"):
        byte = 2 * T * (hq + hkv) * HEAD * es + 4 * T
        if case["op"] == "append":  # values too; keys and values out as the cache holds them
            byte += T * hkv * HEAD * (2 * BYTES[case["cache"]]) + 8 * T
        return {"bytes": byte, "flops": T * (hq + hkv) * (6 * HEAD * case["norm"] + 3 * case["rot"])}
    seen = new + ctx
    lo = np.maximum(0, ctx - case["window"] + 1)  # the first query's window begins here
    seen = seen - lo + np.minimum(lo, case["sinks"])
    byte = 2 * T * hq * HEAD * es + 4 * T * hq + 4 * int((-(-seen // case["page"])).sum()) + 8 * case["n"]
    byte += 2 * int(seen.sum()) * hkv * HEAD * BYTES[case["cache"]]
    return {"bytes": byte, "flops": 4 * HEAD * hq * _pairs(case, new, ctx)}


def frequencies(case):
    """Radians a position for each pair, and what the turned pairs are multiplied by."""
    rot, base, s = case["rot"], case["base"], case["factor"]
    if case["scaling"] == "ntk":
        base *= s ** (rot / (rot - 2))
    f = [base ** (-2 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        return [x / s for x in f], 1.0
    if case["scaling"] == "yarn":  # slow pairs are stretched, fast ones (over 32 turns in the original length) are not
        keep = [min(1.0, max(0.0, (case["original"] * x / (2 * math.pi) - 1) / 31)) for x in f]
        return [x * k + x / s * (1 - k) for x, k in zip(f, keep)], 0.1 * math.log(s) + 1
    return f, 1.0


# ----------------------------------------------------------------- the state
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    if case["op"] == "verify":
        return _prepare_verify(case, g)
    new, ctx = _lengths(case)
    n, h, T = case["n"], case["hkv"], int(new.sum())
    x = lambda *size: torch.randn(size, generator=g, device=DEV)  # noqa: E731
    s = {"case": dict(case), "T": T, "max_new": int(new.max()), "max_kv": int((new + ctx).max())}
    s["cu"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)])).to(DEV, torch.int32)
    s["kv_len"] = torch.from_numpy(new + ctx).to(DEV, torch.int32)
    i = torch.repeat_interleave(torch.arange(n), torch.from_numpy(new))
    pos = (torch.from_numpy(ctx)[i] + torch.arange(T) - torch.from_numpy(np.cumsum(new) - new)[i]).to(DEV)
    if case["op"] in ("rope", "append"):
        s["qkv"] = (2 * x(T, case["hq"] + 2 * h, HEAD)).to(TYPES[case["dtype"]])
        s["positions"] = pos.to(torch.int32)
        if case["norm"]:
            s["q_weight"], s["k_weight"] = 1 + 0.2 * x(HEAD), 1 + 0.2 * x(HEAD)
        f, s["amplitude"] = frequencies(case)
        s["radians"] = torch.tensor(f, dtype=torch.float64, device=DEV)
        if own:  # what a program keeps between calls
            import linear_attention_serving_gb300 as kda
            s["freq"], s["amplitude"] = kda.rope_frequencies(case["rot"], base=case["base"], scaling=case["scaling"],
                                                             factor=case["factor"], original_len=case["original"], device=DEV)
    if case["op"] == "rope":
        return s
    page, blocks = case["page"], -(-(new + ctx) // case["page"])
    seen_from = np.zeros_like(ctx) if case["op"] == "attn" else ctx // page  # (the append needs no older pages)
    owned = blocks - seen_from
    pages, width = int(owned.sum()) + 4, int(blocks.max())
    shuffled = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)
    col = torch.arange(width, device=DEV)[None, :]
    d = lambda a: torch.from_numpy(a).to(DEV)[:, None]  # noqa: E731
    at = d(np.cumsum(owned) - owned) + col - d(seen_from)
    mine = (col >= d(seen_from)) & (col < d(blocks))
    s["table"] = torch.where(mine, shuffled[at.clamp(0, pages - 1)], torch.full_like(at, -1, dtype=torch.int32))
    cache = TYPES[case["cache"]]
    kc, vc = x(pages, h, page, HEAD), x(pages, h, page, HEAD)
    if case["cache"] == "e4m3":  # scales as a calibration on the layer's largest values gives them
        s["k_scale"] = (7 + 2 * x(h).abs()) / 448
        s["v_scale"] = (7 + 2 * x(h).abs()) / 448
        kc, vc = (t.div_(sc.view(1, h, 1, 1)).clamp_(-448, 448) for t, sc in ((kc, s["k_scale"]), (vc, s["v_scale"])))
    s["k_cache"], s["v_cache"] = kc.to(cache), vc.to(cache)
    del kc, vc
    if case["op"] == "append":
        s["slots"] = s["table"][i.to(DEV), pos // page].long() * page + pos % page
        return s
    s["q"] = (2 * x(T, case["hq"], HEAD)).to(TYPES[case["dtype"]])
    if own:
        import linear_attention_serving_gb300 as kda
        s["ws"] = torch.empty(kda.paged_attn_workspace_size(T, n, case["hq"], h), dtype=torch.uint8, device=DEV)
    return s


def _prepare_verify(case, g):
    n, w, V, to = case["n"], case["w"], case["vocab"], TYPES[case["dtype"]]
    s = {"case": dict(case)}
    s["target"] = torch.empty(n, w, V, dtype=to, device=DEV)
    s["draft"] = None if case["greedy"] else torch.empty(n, w - 1, V, dtype=to, device=DEV)
    s["tokens"] = torch.empty(n, w - 1, dtype=torch.int32, device=DEV)
    step = max(1, (1 << 27) // (w * V))
    for a in range(0, n, step):  # the draft model's logits are the target's, some way off
        logits = case["flat"] * torch.randn(min(step, n - a), w, V, generator=g, device=DEV)
        s["target"][a:a + step] = logits.softmax(2).to(to)
        logits = logits[:, :-1] + case["noise"] * torch.randn(min(step, n - a), w - 1, V, generator=g, device=DEV)
        if case["greedy"]:
            s["tokens"][a:a + step] = logits.argmax(2).int()
            continue
        q = logits.softmax(2).to(to)
        s["draft"][a:a + step] = q
        pick = torch.rand(*q.shape[:2], 1, generator=g, device=DEV, dtype=torch.float64)
        c = torch.cumsum(q.double(), 2)
        s["tokens"][a:a + step] = torch.searchsorted(c, pick * c[..., -1:], right=True)[..., 0].clamp(max=V - 1).int()
    s["uniform"] = torch.rand(n, w, generator=g, device=DEV)
    s["n_draft"] = torch.from_numpy(_drafts(case)).to(DEV, torch.int32) if case["ragged"] else None
    return s


# ------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return {"rope": _rope_own, "append": _append_own, "attn": _attn_own, "verify": _verify_own}[op](s)
    return {"rope": _rope, "append": _append, "attn": _attn, "verify": _verify}[op](s)


def _heads(s):
    return s["qkv"].split((s["case"]["hq"], s["case"]["hkv"], s["case"]["hkv"]), 1)


def _rope_own(s):
    import linear_attention_serving_gb300 as kda
    q, k, _ = _heads(s)
    q, k = kda.qk_rope(q, k, s["positions"], s["freq"], amplitude=s["amplitude"], interleaved=s["case"]["pairs"],
                       q_weight=s.get("q_weight"), k_weight=s.get("k_weight"), eps=EPS)
    return {"q": q, "k": k}


def _append_own(s):
    import linear_attention_serving_gb300 as kda
    q, k, v = _heads(s)
    q = kda.paged_rope_append(q, k, v, s["positions"], s["slots"], s["freq"], s["k_cache"], s["v_cache"],
                              amplitude=s["amplitude"], interleaved=s["case"]["pairs"], q_weight=s.get("q_weight"),
                              k_weight=s.get("k_weight"), eps=EPS, k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _attn_own(s):
    import linear_attention_serving_gb300 as kda
    o, lse = kda.paged_attn(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"], max_q=s["max_new"],
                            window=s["case"]["window"], sinks=s["case"]["sinks"], k_scale=s.get("k_scale"),
                            v_scale=s.get("v_scale"), workspace=s["ws"])
    return {"o": o, "lse": lse}


def _verify_own(s):
    import linear_attention_serving_gb300 as kda
    accepted, tokens = kda.verify_drafts(s["target"], s["tokens"], s["uniform"], draft=s["draft"], n_draft=s["n_draft"])
    return {"accepted": accepted, "tokens": tokens}


def _turned(x, weight, s):
    """Normed and turned, in 32 bits (the angles in 64)."""
    c, x = s["case"], x.float()
    if c["norm"]:
        x = x * torch.rsqrt((x * x).mean(2, keepdim=True) + EPS) * weight
    angle = s["positions"].double()[:, None] * s["radians"][None, :]
    cos, sin = (s["amplitude"] * torch.cos(angle)).float()[:, None], (s["amplitude"] * torch.sin(angle)).float()[:, None]
    rot = c["rot"]
    if c["pairs"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack((a * cos - b * sin, a * sin + b * cos), 3).flatten(2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat((a * cos - b * sin, a * sin + b * cos), 2)
    return torch.cat((turned, x[..., rot:]), 2)


def _rope(s):
    q, k, _ = _heads(s)
    return {"q": _turned(q, s.get("q_weight"), s).to(q.dtype), "k": _turned(k, s.get("k_weight"), s).to(k.dtype)}


def _append(s):
    q, k, v = _heads(s)
    page, slots = s["case"]["page"], s["slots"]
    for x, cache, scale in ((_turned(k, s.get("k_weight"), s), "k_cache", "k_scale"), (v.float(), "v_cache", "v_scale")):
        if scale in s:
            x = (x / s[scale].view(1, -1, 1)).clamp(-448, 448)
        held = x.to(s[cache].dtype)
        raw = torch.uint8 if held.dtype == torch.float8_e4m3fn else held.dtype  # rows are moved as they are
        s[cache].view(raw)[slots // page, :, slots % page] = held.view(raw)
    return {"q": _turned(q, s.get("q_weight"), s).to(q.dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


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
    pos = ((kv_len - new)[:, None] + torch.arange(m, device=q.device)[None, :])[:, :, None]
    key = torch.arange(kv, device=q.device)
    hidden = (key > pos) | ((key <= pos - c["window"]) & (key >= c["sinks"]))
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


def _verify(s):
    """In 64 bits: the token sought is where a sum over the whole vocabulary passes a bound."""
    p, q, d, u = s["target"], s["draft"], s["tokens"].long(), s["uniform"].double()
    n, w, V = p.shape
    m = torch.full((n,), w - 1, device=p.device) if s["n_draft"] is None else s["n_draft"].long()
    j = torch.arange(w - 1, device=p.device)
    pd = p[:, :-1].gather(2, d[..., None])[..., 0].double()
    qd = 1.0 if q is None else q.gather(2, d[..., None])[..., 0].double()
    stands = (u[:, :-1] * qd < pd) & (j < m[:, None])
    accepted = stands.int().cumprod(1).sum(1)
    i = torch.arange(n, device=p.device)
    row = p[i, accepted].double()
    at = accepted.clamp(max=w - 2)
    refused = accepted < m
    if q is None:
        rest = row.clone()
        rest[i, d[i, at]] = 0
    else:
        rest = (row - q[i, at].double()).clamp(min=0)
    rest = torch.where((refused & (rest.sum(1) > 0))[:, None], rest, row)
    c = rest.cumsum(1)
    token = (c <= u[:, -1:] * c[:, -1:]).sum(1).clamp(max=V - 1)
    col = torch.arange(w, device=p.device)
    out = torch.where(col < accepted[:, None], torch.nn.functional.pad(d, (0, 1)), -1)
    out = torch.where(col == accepted[:, None], token[:, None], out)
    return {"accepted": accepted.int(), "tokens": out.int()}


# ------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    if case["op"] == "verify":
        return None  # whole numbers
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] in ("rope", "append"):
        q, k, v = (t.to(d) for t in _heads(s))
        f, amplitude = frequencies(case)
        half = case["rot"] // 2
        first = torch.arange(half, device=DEV) * (2 if case["pairs"] else 1)
        second = first + (1 if case["pairs"] else half)
        angle = torch.outer(s["positions"].to(d), torch.tensor(f, dtype=d, device=DEV))
        turn = torch.polar(torch.full_like(angle, amplitude), angle)[:, None]  # a complex number for each pair

        def turned(x, weight):
            if case["norm"]:
                x = x / torch.sqrt((x ** 2).sum(2, keepdim=True) / HEAD + EPS) * weight.to(d)
            z = torch.complex(x[..., first], x[..., second]) * turn
            x = x.clone()
            x[..., first], x[..., second] = z.real, z.imag
            return x

        q, k = turned(q, s.get("q_weight")), turned(k, s.get("k_weight"))
        if case["op"] == "rope":
            return {"q": q, "k": k}
        out, page = {"q": q}, case["page"]
        for x, cache, scale in ((k, "k_cache", "k_scale"), (v, "v_cache", "v_scale")):
            y = s[cache].to(d)
            if scale in s:
                x = x / s[scale].to(d)[None, :, None]
            y[torch.div(s["slots"], page, rounding_mode="floor"), :, s["slots"] % page] = x
            out[cache] = y
        return out
    page, cu, lens = case["page"], s["cu"].tolist(), s["kv_len"].tolist()
    hkv, g = case["hkv"], case["hq"] // case["hkv"]
    o = torch.zeros(s["T"], case["hq"], HEAD, dtype=d, device=DEV)
    lse = torch.full((s["T"], case["hq"]), -math.inf, dtype=d, device=DEV)
    for i in range(case["n"]):
        a, b, kv = cu[i], cu[i + 1], lens[i]
        pages = s["table"][i, :-(-kv // page)].long()
        p = torch.arange(kv - (b - a), kv, device=DEV)[:, None]
        key = torch.arange(kv, device=DEV)[None, :]
        seen = (key <= p) & ((p - key < case["window"]) | (key < case["sinks"]))
        some = seen.any(0).nonzero()[:, 0]  # keys of the request that any of its queries sees
        seen = seen[:, some]
        for h in range(hkv):
            k = s["k_cache"][pages, h].reshape(-1, HEAD)[some].to(d)
            v = s["v_cache"][pages, h].reshape(-1, HEAD)[some].to(d)
            if "k_scale" in s:
                k, v = k * s["k_scale"][h].to(d), v * s["v_scale"][h].to(d)
            heads = slice(h * g, h * g + g)
            z = torch.einsum("thd,kd->htk", s["q"][a:b, heads].to(d), k) / math.sqrt(HEAD)
            z = torch.where(seen[None], z, torch.full((), -math.inf, dtype=d, device=DEV))
            l = torch.logsumexp(z, 2)
            pr = torch.where(seen[None], torch.exp(z - l[..., None]), torch.zeros((), dtype=d, device=DEV))
            o[a:b, heads] = torch.einsum("htk,kd->thd", pr, v)
            lse[a:b, heads] = l.T
    return {"o": o, "lse": lse}
