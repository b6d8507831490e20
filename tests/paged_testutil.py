"""Plain 64-bit forms of the paged cache's operators, and inputs for them."""
import math

import torch

D = 128


def cdiv(a, b):
    return -(-a // b)


def tables_ref(new, ctx, table, free, head, ps):
    """(table, slots, positions, cu, kv_len, head) with Python integers."""
    table = [list(r) for r in table]
    slots, positions, cu, kv = [], [], [0], []
    for i, (n, c) in enumerate(zip(new, ctx)):
        for b in range(cdiv(c, ps), cdiv(c + n, ps)):
            table[i][b] = free[head]
            head += 1
        for p in range(c, c + n):
            slots.append(table[i][p // ps] * ps + p % ps)
            positions.append(p)
        cu.append(cu[-1] + n)
        kv.append(c + n)
    return table, slots, positions, cu, kv, head


def attn_ref(q, k_cache, v_cache, table, cu, kv_len, scale=D ** -0.5, window=0, k_scale=None, v_scale=None):
    """o, lse and, per output value, sum_j p_j |v_j| (the scale of rounding the
    probabilities), and per row max_j scale sum_c |q_c k_jc| (that of the scores)."""
    q, hkv, ps = q.double().cpu(), k_cache.shape[1], k_cache.shape[2]
    T, hq, _ = q.shape
    g = hq // hkv
    o, a = torch.zeros(T, hq, D, dtype=torch.float64), torch.zeros(T, hq, D, dtype=torch.float64)
    lse, mag = torch.full((T, hq), -math.inf, dtype=torch.float64), torch.zeros(T, hq, dtype=torch.float64)
    kc, vc = k_cache.cpu().to(torch.float32).double(), v_cache.cpu().to(torch.float32).double()
    for i in range(len(kv_len)):
        for t in range(cu[i], cu[i + 1]):
            pos = kv_len[i] - (cu[i + 1] - cu[i]) + t - cu[i]
            lo = max(0, pos - window + 1) if window else 0
            if pos < lo:
                continue
            keys = torch.arange(lo, pos + 1)
            pages = torch.tensor([table[i][j // ps] for j in range(lo, pos + 1)])
            for h in range(hkv):
                k, v = kc[pages, h, keys % ps], vc[pages, h, keys % ps]
                if k_scale is not None:
                    k, v = k * float(k_scale[h]), v * float(v_scale[h])
                x = q[t, h * g:(h + 1) * g]
                s = scale * x @ k.T
                l = torch.logsumexp(s, 1)
                p = torch.exp(s - l[:, None])
                rows = slice(h * g, (h + 1) * g)
                o[t, rows], lse[t, rows], a[t, rows] = p @ v, l, p @ v.abs()
                mag[t, rows] = (scale * x.abs() @ k.abs().T).amax(1)
    return o, lse, a, mag


def make(new, ctx, hkv, g, ps, cache=torch.bfloat16, seed=0, device="cpu", spare=3, q_std=1.5, filler=float("nan")):
    """A filled cache whose unused rows and pages hold `filler`, with shuffled
    pages; kv_len = ctx + new."""
    gen = torch.Generator().manual_seed(seed)
    n = len(new)
    kv = [a + b for a, b in zip(new, ctx)]
    blocks = [cdiv(x, ps) for x in kv]
    width = max(1, max(blocks)) + 1
    pages = sum(blocks) + spare
    perm = torch.randperm(pages, generator=gen).tolist()
    table, at = [], 0
    for b in blocks:
        table.append(perm[at:at + b] + [-7] * (width - b))
        at += b
    kc = torch.full((pages, hkv, ps, D), filler)
    vc = torch.full((pages, hkv, ps, D), filler)
    for i, x in enumerate(kv):
        for b in range(blocks[i]):
            m = min(ps, x - b * ps)
            kc[table[i][b], :, :m] = torch.randn(hkv, m, D, generator=gen)
            vc[table[i][b], :, :m] = torch.randn(hkv, m, D, generator=gen) + 0.25
    cu = [0]
    for x in new:
        cu.append(cu[-1] + x)
    qt = torch.float32 if cache == torch.float32 else torch.bfloat16
    q = (q_std * torch.randn(cu[-1], hkv * g, D, generator=gen)).to(qt)
    d = {"q": q, "table": table, "cu": cu, "kv": kv, "k_scale": None, "v_scale": None}
    if cache == torch.float8_e4m3fn:
        d["k_scale"] = (0.5 + torch.rand(hkv, generator=gen)) / 64
        d["v_scale"] = (0.5 + torch.rand(hkv, generator=gen)) / 64
        kc = (kc / d["k_scale"].view(1, -1, 1, 1)).clamp(-448, 448)
        vc = (vc / d["v_scale"].view(1, -1, 1, 1)).clamp(-448, 448)
    d["k_cache"], d["v_cache"] = kc.to(cache), vc.to(cache)
    return d


def attn_close(o, lse, ref, q_dtype, cache_dtype):
    """Holds every value to the roundings on its way: the scores' fp32 sums move log p
    by `ds`; each probability is rounded to bf16 (2^-8) or fp16 (2^-11) before its
    product, or, fp32, the sums over the keys are held to 2^-21; the output is rounded
    once."""
    o_ref, lse_ref, a, mag = ref
    assert torch.equal(torch.isinf(lse.double().cpu()), torch.isinf(lse_ref)), "rows that see no key"
    p_step = {torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -11, torch.float32: 2.0 ** -21}[cache_dtype]
    out_step = 2.0 ** -8 if q_dtype == torch.bfloat16 else 2.0 ** -24
    ds = 2.0 ** -19 * (1 + mag)[..., None]  # 128-term sums, the log2 scale, the hardware exponential
    off = (o.double().cpu() - o_ref).abs()
    tol = out_step * o_ref.abs() + (1 + out_step) * (p_step + 2 * ds) * a + 1e-30
    assert torch.isfinite(o).all()
    worst = (off / tol).max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"o: {worst:.2f} of its bound at {divmod(int((off / tol).argmax()), D)}"
    fin = torch.isfinite(lse_ref)
    d = (lse.double().cpu() - lse_ref).abs()[fin]
    t = (ds[..., 0] + 2.0 ** -22 * lse_ref.abs())[fin]
    assert (d <= t).all(), f"lse: {(d / t).max().item():.2f} of its bound"
