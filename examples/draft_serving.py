"""Serving steps with drafted tokens of a small hybrid model: one layer of Kimi Delta
Attention and one of softmax attention (normed, turned queries and keys, a sliding
window beside the first tokens) over a paged cache.

    python examples/draft_serving.py

Each step takes a window of a token and its drafts for every request, and says on the
GPU alone how many drafts stand, which token follows, and where the requests then are: the
step is captured into a graph and replayed.  At the end the committed streams are given
once more, in one pass, and have to give the same probabilities up to rounding.  Random
weights; the draft model is a table.
"""
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import linear_attention_serving_gb300 as kda

DEV, BF16, F32, I32, D = "cuda", torch.bfloat16, torch.float32, torch.int32, 128
VOCAB, HIDDEN, KDA_HEADS, HQ, HKV, PAGE, WINDOW, SINKS = 24, 256, 2, 4, 2, 16, 24, 3
OPTIONS = dict(qk_l2norm=True, beta_sigmoid=True, q_scale=True)


class Weights:
    def __init__(self, seed=0):
        g = torch.Generator().manual_seed(seed)
        w = lambda rows, cols: (torch.randn(rows, cols, generator=g) * rows ** -0.5).to(DEV, BF16)  # noqa: E731
        self.embed = torch.randn(VOCAB, HIDDEN, generator=g).to(DEV, BF16)
        self.kda_in, self.kda_out = w(HIDDEN, KDA_HEADS * (4 * D + 1)), w(KDA_HEADS * D, HIDDEN)
        self.attn_in, self.attn_out, self.head = w(HIDDEN, (HQ + 2 * HKV) * D), w(HQ * D, HIDDEN), w(HIDDEN, VOCAB)
        self.q_norm, self.k_norm = (1 + 0.2 * torch.randn(2, D, generator=g)).to(DEV).unbind(0)
        self.A = torch.zeros(KDA_HEADS, device=DEV)
        self.draft = (0.6 * torch.randn(VOCAB, VOCAB, generator=g)).softmax(1).to(DEV)  # the draft model: by the last token
        self.freq, self.amplitude = kda.rope_frequencies(64, scaling="yarn", factor=4.0, original_len=64, device=DEV)


def kda_inputs(w, x):
    y = x @ w.kda_in
    q, k, v, z = (t.contiguous() for t in y[:, :4 * KDA_HEADS * D].view(-1, 4, KDA_HEADS, D).unbind(1))
    return q, k, v, z.float(), y[:, 4 * KDA_HEADS * D:].float().contiguous()


def attention(w, x, cache, table, slots, positions, cu, kv_len, max_q, error):
    q, k, v = (x @ w.attn_in).view(len(x), HQ + 2 * HKV, D).split((HQ, HKV, HKV), 1)
    q = kda.paged_rope_append(q, k, v, positions, slots, w.freq, *cache, amplitude=w.amplitude, q_weight=w.q_norm,
                              k_weight=w.k_norm, error_word=error)
    o, _ = kda.paged_attn(q, *cache, table, cu, kv_len, max_q=max_q, window=WINDOW, sinks=SINKS, error_word=error)
    return x + o.view(len(x), HQ * D) @ w.attn_out


class Server:
    """n requests, each with its next token at hand; a step commits that token and the drafts that stand."""

    def __init__(self, w, n, drafts, steps):
        self.w, self.n, self.W = w, n, drafts + 1
        blocks = -(-(steps + 1) * self.W // PAGE) + 1
        self.pages = n * (2 * steps + blocks)  # (a step's refused drafts may leave a page behind)
        self.cache = [torch.zeros(self.pages, HKV, PAGE, D, device=DEV, dtype=BF16) for _ in range(2)]
        i32 = dict(device=DEV, dtype=I32)
        self.table = torch.full((n, blocks), -1, **i32)
        self.free, self.head = torch.randperm(self.pages, device=DEV).to(I32), torch.zeros(1, **i32)
        self.new, self.ctx, self.accepted = torch.full((n,), self.W, **i32), torch.zeros(n, **i32), torch.zeros(n, **i32)
        self.token, self.error = torch.zeros(n, **i32), torch.zeros(1, **i32)
        self.state = torch.zeros(n, KDA_HEADS, D, D, device=DEV)
        row = (n, drafts, KDA_HEADS, D)
        self.kda_cache = tuple(torch.zeros(row, device=DEV, dtype=t) for t in (BF16, BF16, BF16, F32)) + (
            torch.zeros(row[:3], device=DEV),)

    def propose(self, u):
        """A draft for each u [n, W - 1], from the table; their probabilities."""
        tokens, rows = [self.token], []
        for j in range(self.W - 1):
            rows.append(self.w.draft[tokens[-1].long()])
            c = rows[-1].cumsum(1)
            tokens.append((c <= u[:, j:j + 1] * c[:, -1:]).sum(1).clamp(max=VOCAB - 1).to(I32))
        return torch.stack(tokens, 1), torch.stack(rows, 1)

    def step(self, u_draft, u):
        """Returns (window tokens [n, W], the model's probabilities [n, W, vocabulary], accepted [n], tokens [n, W])."""
        n, W, w = self.n, self.W, self.w
        window, q_draft = self.propose(u_draft)
        slots, positions, cu, kv_len, head = kda.paged_tables(self.new, self.ctx, self.table, self.free, self.head, n * W, PAGE,
                                                              self.pages, error_word=self.error)
        x = w.embed[window.long()].view(n * W, HIDDEN)
        inp = (t.view(n, W, *t.shape[1:]) for t in kda_inputs(w, x))
        o = kda.decode_step(self.state, *inp, w.A, self.kda_cache, num_accepted=self.accepted, error_word=self.error, **OPTIONS)
        x = x + o.reshape(n * W, KDA_HEADS * D) @ w.kda_out
        x = attention(w, x, self.cache, self.table, slots, positions, cu, kv_len, W, self.error)
        p = (x.float() @ w.head.float()).softmax(1).view(n, W, VOCAB)
        accepted, tokens = kda.verify_drafts(p, window[:, 1:].contiguous(), u, draft=q_draft, error_word=self.error)
        # where the requests are now: what the next step begins from
        self.head.copy_(head)
        self.ctx.add_(1 + accepted)
        self.accepted.copy_(accepted)
        self.token.copy_(tokens.gather(1, accepted.long()[:, None])[:, 0])
        return window, p, accepted, tokens


def one_pass(w, streams):
    """The probabilities after every token of the streams, all at once."""
    n, new = len(streams), [len(s) for s in streams]
    T, blocks = sum(new), -(-max(new) // PAGE)
    i32 = lambda v: torch.tensor(v, dtype=I32, device=DEV)  # noqa: E731
    pages, error = n * blocks, i32([0])
    table = torch.full((n, blocks), -1, dtype=I32, device=DEV)
    cache = [torch.zeros(pages, HKV, PAGE, D, device=DEV, dtype=BF16) for _ in range(2)]
    slots, positions, cu, kv_len, _ = kda.paged_tables(i32(new), i32([0] * n), table, torch.arange(pages, device=DEV).to(I32),
                                                       i32([0]), T, PAGE, pages, error_word=error)
    x = w.embed[torch.cat(streams).long()]
    q, k, v, z, beta = kda_inputs(w, x)
    o, _ = kda.chunk_fwd(q, k, v, z, w.A, beta, cu_seqlens=cu, **OPTIONS)
    x = x + o.view(T, KDA_HEADS * D) @ w.kda_out
    x = attention(w, x, cache, table, slots, positions, cu, kv_len, max(new), error)
    assert int(error) == 0
    return (x.float() @ w.head.float()).softmax(1)


def main(n=5, drafts=3, steps=40, replay=True):
    w = Weights()
    server = Server(w, n, drafts, steps)
    g = torch.Generator().manual_seed(3)
    u = torch.rand(steps, n, 2 * drafts + 1, generator=g).to(DEV)
    u_draft, u_test = torch.empty(n, drafts, device=DEV), torch.empty(n, drafts + 1, device=DEV)
    run = lambda: server.step(u_draft, u_test)  # noqa: E731
    streams, rows, stood = [[] for _ in range(n)], [[] for _ in range(n)], 0
    graph = None
    for i in range(steps):
        u_draft.copy_(u[i, :, :drafts])
        u_test.copy_(u[i, :, drafts:])
        if i < 2 or not replay:  # (the first steps load and set up)
            out = run()
        elif graph is None:
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                out = run()
            graph.replay()
        else:
            graph.replay()
        window, p, accepted = (t.cpu() for t in out[:3])
        for r in range(n):
            a = int(accepted[r]) + 1
            streams[r].append(window[r, :a])
            rows[r].append(p[r, :a])
            stood += a - 1
    assert int(server.error) == 0
    streams = [torch.cat(s).to(DEV) for s in streams]
    got, ref = torch.cat([torch.cat(r) for r in rows]).double(), one_pass(w, streams).cpu().double()
    off = ((got - ref).norm() / ref.norm()).item()
    print(f"{n} requests, {steps} steps, {len(got)} tokens, {stood} of {n * steps * drafts} drafts stood; probabilities against one "
          f"pass: relative difference {off:.1e}")
    return off, [s.tolist() for s in streams], stood / (n * steps * drafts)


if __name__ == "__main__":
    sys.exit(0 if main()[0] < 2e-2 else 1)
