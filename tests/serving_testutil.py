"""Plain 64-bit forms of rotary positions with norms, window attention with sinks, and the
verification of drafts, and inputs for them."""
import math
from fractions import Fraction

import torch

D = 128


def frequencies_ref(rot, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0):
    """Radians a position, and the amplitude."""
    f = []
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" else base
        x = b ** (-2.0 * i / rot)
        if scaling == "linear":
            x /= factor
        if scaling == "yarn":
            turns = original_len * x / (2 * math.pi)
            g = min(1.0, max(0.0, (turns - beta_slow) / (beta_fast - beta_slow)))
            x = g * x + (1 - g) * x / factor
        f.append(x)
    return f, (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def rope_ref(x, positions, freq, amplitude, interleaved, weight, eps):
    """Normed and turned in 64 bits, and per value the size of the terms it is summed from.  freq:
    int64 turns a position times 2^64 (angles by Python's integers), or None."""
    x = x.double().cpu()
    y = x.clone()
    if weight is not None:
        y = x / torch.sqrt((x * x).mean(2, keepdim=True) + eps) * weight.double().cpu()
    mag = y.abs()
    if freq is None or len(freq) == 0:
        return y, mag
    f = [int(v) for v in freq]
    angle = torch.tensor([[(int(p) * v % (1 << 64)) / 2.0 ** 64 * 2 * math.pi for v in f] for p in positions.tolist()],
                         dtype=torch.float64).reshape(len(positions), len(f))
    c, s = (amplitude * torch.cos(angle))[:, None], (amplitude * torch.sin(angle))[:, None]
    half = len(f)
    i = torch.arange(half) * 2 if interleaved else torch.arange(half)
    j = i + 1 if interleaved else i + half
    a, b = y[..., i], y[..., j]
    out, size = y.clone(), mag.clone()
    out[..., i], out[..., j] = a * c - b * s, a * s + b * c
    size[..., i] = size[..., j] = abs(amplitude) * (a.abs() + b.abs())
    return out, size


# What fp32 does on the way, in units of 2^-24 of the terms' size: the mean of squares (8 products and sums in a
# lane, 4 across: 12, of which the root halves the effect: 6), the hardware's reciprocal root (2 ulp: 4), the product
# with the weight (2), the angle (2^-25 radians: 1), sine and cosine (2 ulp: 4), times the amplitude (1), the turned
# pair's two products and sum (3): 21, under 32.
FP32 = 2.0 ** -19


def rope_close(got, ref, size, dtype):
    half = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}[dtype]
    off = (got.double().cpu() - ref).abs()
    tol = half * ref.abs() + (1 + half) * FP32 * size + 1e-37
    assert torch.isfinite(got).all()
    assert (off <= tol).all(), f"{(off / tol).max().item():.2f} of its bound at {divmod(int((off / tol).argmax()), D)}"


def sinks_ref(q, k_cache, v_cache, table, cu, kv_len, scale=D ** -0.5, window=0, sinks=0, k_scale=None, v_scale=None):
    """As paged_testutil.attn_ref, a request at a time."""
    q, hkv, ps = q.double().cpu(), k_cache.shape[1], k_cache.shape[2]
    T, hq, _ = q.shape
    g = hq // hkv
    o, a = torch.zeros(T, hq, D, dtype=torch.float64), torch.zeros(T, hq, D, dtype=torch.float64)
    lse, mag = torch.full((T, hq), -math.inf, dtype=torch.float64), torch.zeros(T, hq, dtype=torch.float64)
    kc, vc = k_cache.cpu().to(torch.float32).double(), v_cache.cpu().to(torch.float32).double()
    for i in range(len(kv_len)):
        n, kv = cu[i + 1] - cu[i], kv_len[i]
        if n == 0 or kv == 0:
            continue
        p = torch.arange(kv - n, kv)[:, None]
        key = torch.arange(kv)[None, :]
        seen = key <= p
        if window:
            seen &= (key > p - window) | (key < sinks)
        some = seen.any(0)
        keys = torch.arange(kv)[some]
        seen = seen[:, some]
        pages = torch.tensor([table[i][j // ps] for j in keys.tolist()])
        for h in range(hkv):
            k, v = kc[pages, h, keys % ps], vc[pages, h, keys % ps]
            if k_scale is not None:
                k, v = k * float(k_scale[h]), v * float(v_scale[h])
            rows = slice(h * g, (h + 1) * g)
            x = q[cu[i]:cu[i + 1], rows]
            s = torch.einsum("tgd,kd->tgk", x, k) * scale
            s = s.masked_fill(~seen[:, None], -math.inf)
            l = torch.logsumexp(s, 2)
            w = torch.exp(s - torch.where(torch.isinf(l), torch.zeros_like(l), l)[..., None])
            w = torch.where(seen[:, None], w, torch.zeros_like(w))
            t = slice(cu[i], cu[i + 1])
            o[t, rows], lse[t, rows], a[t, rows] = w @ v, l, w @ v.abs()
            size = torch.einsum("tgd,kd->tgk", x.abs(), k.abs()) * scale
            mag[t, rows] = torch.where(seen[:, None], size, torch.zeros_like(size)).amax(2)
    return o, lse, a, mag


def verify_ref(target, tokens, uniforms, draft=None, n_draft=None):
    """In exact fractions: (num_accepted, tokens) as lists."""
    n, w, V = target.shape
    p = target.double().tolist()
    q = None if draft is None else draft.double().tolist()
    accepted, out = [], []
    for i in range(n):
        m = w - 1 if n_draft is None else int(n_draft[i])
        a = 0
        while a < m:
            d = int(tokens[i, a])
            qd = 1.0 if q is None else q[i][a][d]
            if not Fraction(float(uniforms[i, a])) * Fraction(qd) < Fraction(p[i][a][d]):
                break
            a += 1
        weights = [Fraction(x) for x in p[i][a]]
        if a < m:
            if q is None:
                rest = [x if k != int(tokens[i, a]) else Fraction(0) for k, x in enumerate(weights)]
            else:
                rest = [max(x - Fraction(y), Fraction(0)) for x, y in zip(weights, q[i][a])]
            weights = rest if any(rest) else weights
        bound = Fraction(float(uniforms[i, w - 1])) * sum(weights)
        total, k = Fraction(0), 0
        for k, x in enumerate(weights):
            total += x
            if total > bound:
                break
        accepted.append(a)
        out.append([int(t) for t in tokens[i, :a]] + [k] + [-1] * (w - 1 - a))
    return accepted, out


def draft_inputs(n, w, V, seed=0, spread=2.0, noise=0.7, dtype=torch.float32, certain=False):
    g = torch.Generator().manual_seed(seed)
    logits = spread * torch.randn(n, w, V, generator=g)
    target = logits.softmax(2).to(dtype)
    near = (logits[:, :-1] + noise * torch.randn(n, w - 1, V, generator=g)).softmax(2).to(dtype)
    if w == 1:
        tokens = torch.empty(n, 0, dtype=torch.int32)
    elif certain:
        tokens = near.float().argmax(2).int()
    else:
        tokens = torch.multinomial(near.float().reshape(-1, V), 1, generator=g).reshape(n, w - 1).int()
    return target, None if certain else near, tokens, torch.rand(n, w, generator=g)
