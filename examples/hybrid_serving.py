"""Serving steps of a small hybrid stack: one layer of Kimi Delta Attention, whose
cache is a state of fixed size, and one of softmax attention over a paged cache.

    python examples/hybrid_serving.py

Ragged prompts are taken in packed chunks, then every request decodes token by
token; each step's block tables, slot map and offsets are worked out on the GPU
from the requests' lengths alone.  At the end the whole streams are given once
more, as prompts, and have to give the same outputs up to rounding.  Random
weights, synthetic inputs.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import linear_attention_serving_gb300 as kda

DEV, BF16, I32, D = "cuda", torch.bfloat16, torch.int32, 128
HIDDEN, KDA_HEADS, HQ, HKV, PAGE = 512, 4, 8, 2, 16
OPTIONS = dict(qk_l2norm=True, beta_sigmoid=True, q_scale=True)


class Weights:
    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        w = lambda rows, cols: (torch.randn(rows, cols, generator=g) * rows ** -0.5).to(DEV, BF16)  # noqa: E731
        self.kda_in, self.kda_out = w(HIDDEN, KDA_HEADS * (4 * D + 1)), w(KDA_HEADS * D, HIDDEN)
        self.attn_in, self.attn_out = w(HIDDEN, (HQ + 2 * HKV) * D), w(HQ * D, HIDDEN)
        self.A = torch.zeros(KDA_HEADS, device=DEV)


class Server:
    """What a serving process keeps for n requests between steps."""

    def __init__(self, weights, n, max_len):
        self.w, self.n = weights, n
        blocks = -(-max_len // PAGE)
        self.pages = n * blocks
        self.k_cache, self.v_cache = (torch.empty(self.pages, HKV, PAGE, D, device=DEV, dtype=BF16) for _ in range(2))
        self.table = torch.full((n, blocks), -1, device=DEV, dtype=I32)
        self.free = torch.randperm(self.pages, device=DEV).to(I32)
        self.head = torch.zeros(1, device=DEV, dtype=I32)
        self.ctx = torch.zeros(n, device=DEV, dtype=I32)
        self.state = torch.zeros(n, KDA_HEADS, D, D, device=DEV)
        self.error = torch.zeros(1, device=DEV, dtype=I32)

    def step(self, x, new):
        """x [T, HIDDEN]: new[i] more inputs of each request i, packed.  Returns [T, HIDDEN]."""
        T = len(x)
        slots, positions, cu, kv_len, self.head = kda.paged_tables(
            torch.tensor(new, dtype=I32).to(DEV), self.ctx, self.table, self.free, self.head, T, PAGE, self.pages,
            error_word=self.error)
        x = x + self._kda(x, cu, single=max(new) == 1 and T == self.n)
        q, k, v = (x @ self.w.attn_in).view(T, HQ + 2 * HKV, D).split((HQ, HKV, HKV), 1)
        kda.paged_append(k.contiguous(), v.contiguous(), slots, self.k_cache, self.v_cache, error_word=self.error)
        o, _ = kda.paged_attn(q.contiguous(), self.k_cache, self.v_cache, self.table, cu, kv_len, max_q=max(new),
                              error_word=self.error)
        self.ctx = kv_len
        return x + o.view(T, HQ * D) @ self.w.attn_out

    def _kda(self, x, cu, single):
        T = len(x)
        y = x @ self.w.kda_in
        beta = y[:, 4 * KDA_HEADS * D:].float()
        q, k, v, z = (t.contiguous() for t in y[:, :4 * KDA_HEADS * D].view(T, 4, KDA_HEADS, D).unbind(1))
        if single:
            q, k, v, z, beta = (t.unsqueeze(1) for t in (q, k, v, z.float(), beta.contiguous()))
            o = kda.decode_step(self.state, q, k, v, z, beta, self.w.A, None, **OPTIONS)
        else:
            o, self.state = kda.chunk_fwd(q, k, v, z.float(), self.w.A, beta.contiguous(), cu_seqlens=cu,
                                          init_state=self.state, **OPTIONS)
        return o.reshape(T, KDA_HEADS * D) @ self.w.kda_out


def main(steps=12, chunks=((40, 7, 130), (25, 90, 1))):
    n = len(chunks[0])
    total = [sum(c[i] for c in chunks) + steps for i in range(n)]
    g = torch.Generator().manual_seed(1)
    streams = [torch.randn(t, HIDDEN, generator=g).to(DEV, BF16) for t in total]
    weights = Weights()
    server, done, out = Server(weights, n, max(total)), [0] * n, [[] for _ in range(n)]
    for new in list(chunks) + [(1,) * n] * steps:
        x = torch.cat([s[d:d + m] for s, d, m in zip(streams, done, new)])
        for i, y in enumerate(server.step(x, new).split(list(new))):
            out[i].append(y)
        done = [d + m for d, m in zip(done, new)]
    whole = Server(weights, n, max(total))
    ref = whole.step(torch.cat(streams), total).float()
    got = torch.cat([torch.cat(o) for o in out]).float()
    assert int(server.error) == 0 and int(whole.error) == 0
    off = ((got - ref).norm() / ref.norm()).item()
    print(f"{n} requests, {sum(total)} tokens in {len(chunks) + steps} steps; against one pass: relative difference {off:.1e}")
    return off


if __name__ == "__main__":
    sys.exit(0 if main() < 1e-2 else 1)
