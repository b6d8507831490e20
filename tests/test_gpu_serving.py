"""The calls of a served step with drafts together: projections turned and appended, attention through a
window beside sinks, verification, and the decode step that takes what it says."""
import importlib.util
import os

import pytest
import torch

import linear_attention_serving_gb300 as kda
from serving_testutil import verify_ref

pytestmark = pytest.mark.gpu


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "draft_serving.py")
    spec = importlib.util.spec_from_file_location("draft_serving", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_drafts_step_by_step_against_one_pass():
    """Refused drafts leave no trace: the committed streams' probabilities are those of one pass, up to a few
    roundings to bf16 (2^-9 of each value on average) on the way, and a replayed step commits the same tokens as a
    launched one."""
    e = example()
    off, streams, stood = e.main()
    assert off < 2e-2
    assert 0.05 < stood < 0.95  # both refused and accepted drafts are met
    off2, streams2, _ = e.main(replay=False)
    assert streams2 == streams and off2 < 2e-2


def test_each_step_verifies_as_the_plain_form_does():
    e = example()
    w = e.Weights(seed=4)
    server = e.Server(w, 3, 4, 12)
    g = torch.Generator().manual_seed(8)
    ctx = [0] * 3
    for _ in range(12):
        u = torch.rand(3, 9, generator=g).cuda()
        window, p, accepted, tokens = server.step(u[:, :4].contiguous(), u[:, 4:].contiguous())
        prob = torch.stack([w.draft[window[:, j].long()] for j in range(4)], 1)
        ref = verify_ref(p.cpu(), window[:, 1:].cpu(), u[:, 4:].cpu(), prob.cpu())
        assert accepted.tolist() == ref[0] and tokens.tolist() == ref[1]
        ctx = [c + 1 + a for c, a in zip(ctx, ref[0])]
        assert server.ctx.tolist() == ctx and server.token.tolist() == [t[a] for t, a in zip(ref[1], ref[0])]
    assert int(server.error) == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_windows_of_different_lengths_in_turn(dtype):
    """A decode step of a long window after one of a short window: the kernel keeps the shared memory that it was
    once given (the long window's launch failed after the short one's)."""
    def step(W):
        x = lambda *size: torch.randn(2, W, *size, device="cuda")  # noqa: E731
        row = (2, W - 1, 1, 128)
        cache = tuple(torch.zeros(row, device="cuda", dtype=t) for t in (dtype, dtype, dtype, torch.float32)) + (
            torch.zeros(row[:3], device="cuda"),)
        q, k, v = (x(1, 128).to(dtype) for _ in range(3))
        o = kda.decode_step(torch.zeros(2, 1, 128, 128, device="cuda"), q, k, v, x(1, 128), x(1), torch.zeros(1, device="cuda"),
                            cache, qk_l2norm=True, beta_sigmoid=True)
        assert torch.isfinite(o).all()

    for W in (7, 3, 7, 2, 6, 7):
        step(W)


def test_two_streams_do_not_mix():
    """Calls of two servers on streams of their own, enqueued in turn: each as alone."""
    e = example()
    w = e.Weights(seed=1)
    g = torch.Generator().manual_seed(2)
    u = torch.rand(10, 2, 4, 5, generator=g).cuda()

    def run(streams):
        torch.manual_seed(0)
        servers = [e.Server(w, 4, 2, 10) for _ in range(2)]
        torch.cuda.synchronize()
        out = [[], []]
        for i in range(10):
            for k in range(2):
                with torch.cuda.stream(streams[k]):
                    out[k].append(servers[k].step(u[i, k, :, :2].contiguous(), u[i, k, :, 2:].contiguous()))
        torch.cuda.synchronize()
        assert all(int(s.error) == 0 for s in servers)
        return [[t for step in o for t in step] for o in out]

    one = torch.cuda.current_stream()
    alone, beside = run([one, one]), run([torch.cuda.Stream(), torch.cuda.Stream()])
    for a, b in zip(alone, beside):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("far", [2 ** 32 + 5, 2 ** 40, 2 ** 31, -2 ** 32 + 5])
def test_numbers_past_32_bits_are_refused(far):
    """A window, sinks or a size that the library's 32 bits do not hold is not cut down to what they do."""
    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    new, ctx, table, free, head = i32(2), i32(3), i32(0, 1, -1, -1)[None], i32(1, 2, 3), i32(0)
    kda.paged_tables(new, ctx, table, free, head, 2, 16, 8)
    for page_size, n_pages in ((far - far % 16 + 16, 8), (16, far)):
        with pytest.raises(kda.KDAError, match="32 bits"):
            kda.paged_tables(new, ctx, table, free, head, 2, page_size, n_pages)
    q = torch.randn(2, 2, 128, device="cuda")
    cache = torch.randn(2, 1, 16, 128, device="cuda")
    a = (q, cache, cache.flip(0), i32(0, 1)[None], i32(0, 2), i32(20))
    kda.paged_attn(*a, max_q=2, window=5, sinks=5)
    for kw in (dict(window=far), dict(window=5, sinks=far), dict(max_q=far)):
        with pytest.raises(kda.KDAError, match="32 bits"):
            kda.paged_attn(*a, **kw)


def test_a_vocabulary_past_32_bits_is_refused():
    p = torch.empty(1, 1, 2 ** 32 + 5, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(kda.KDAError, match="32 bits"):
        kda.verify_drafts(p, torch.empty(1, 0, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, device="cuda"))
