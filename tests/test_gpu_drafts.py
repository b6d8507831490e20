"""Verification of drafted tokens against exact fractions, and its law."""
import pytest
import torch

import linear_attention_serving_gb300 as kda
from linear_attention_serving_gb300 import drafts, paged
from serving_testutil import draft_inputs, verify_ref
from test_gpu_canaries import Guarded

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def verify(target, draft, tokens, uniforms, n_draft=None):
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    t, q, d, u, m = dev(target, draft, tokens, uniforms, n_draft)
    acc, out = kda.verify_drafts(t, d, u, draft=q, n_draft=m, error_word=err)
    return acc.tolist(), out.tolist(), int(err)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("n,w,V", [(1, 1, 1), (1, 2, 1), (3, 1, 37), (5, 4, 16), (40, 5, 33), (7, 8, 1000), (2, 32, 64), (300, 3, 8),
                                   (3, 5, 4099)])
def test_against_fractions(n, w, V, certain, dtype):
    target, draft, tokens, u = draft_inputs(n, w, V, seed=n * w + V, dtype=dtype, certain=certain)
    if w == 1:
        draft = None
    acc, out, err = verify(target, draft, tokens, u)
    ref = verify_ref(target, tokens, u, draft)
    assert err == 0 and acc == ref[0] and out == ref[1]


def test_ragged_drafts():
    target, draft, tokens, u = draft_inputs(50, 6, 40, seed=1)
    m = (torch.arange(50) % 6).int()
    for q in (draft, None):
        acc, out, err = verify(target, q, tokens, u, m)
        ref = verify_ref(target, tokens, u, q, m)
        assert err == 0 and acc == ref[0] and out == ref[1]
        assert all(a <= b for a, b in zip(acc, m.tolist()))


def by_sums(target, draft, tokens, u):
    """64-bit sums, for large vocabularies."""
    n, w, V = target.shape
    p, i = target.double(), torch.arange(n, device=DEV)
    pd = p[:, :-1].gather(2, tokens.long()[..., None])[..., 0]
    qd = 1.0 if draft is None else draft.double().gather(2, tokens.long()[..., None])[..., 0]
    acc = (u.double()[:, :-1] * qd < pd).int().cumprod(1).sum(1)
    rest = p[i, acc].clone()
    refused = acc < w - 1
    at = acc.clamp(max=w - 2)
    if draft is None:
        rest[i[refused], tokens.long()[i, at][refused]] = 0
    else:
        rest = torch.where(refused[:, None], (rest - draft[i, at].double()).clamp(min=0), rest)
    c = rest.cumsum(1)
    return acc, (c <= u.double()[:, -1:] * c[:, -1:]).sum(1)


@pytest.mark.parametrize("n,w,V,certain,dtype", [
    (1, 5, 32768, False, F32), (1, 5, 200_003, False, F32), (3, 3, 1_000_001, False, F32), (300, 4, 5000, False, F32),
    (40, 5, 131_072, False, BF16), (700, 2, 20_000, True, F32), (9, 6, 50_001, True, BF16), (2, 2, 9_000_000, False, F32),
    (300, 3, 50_001, False, BF16), (100, 3, 60_003, False, F32), (100, 4, 60_002, True, BF16)])
def test_large_vocabularies(n, w, V, certain, dtype):
    """Every split of a row over blocks and segments; odd sizes go without vector loads."""
    g = torch.Generator(device=DEV).manual_seed(V + n)
    logits = 3 * torch.randn(n, w, V, generator=g, device=DEV)
    target = logits.softmax(2).to(dtype)
    near = (logits[:, :-1] + 0.5 * torch.randn(n, w - 1, V, generator=g, device=DEV)).softmax(2).to(dtype)
    draft = None if certain else near
    tokens = near.float().argmax(2).int()
    u = torch.rand(n, w, generator=g, device=DEV)
    u[: n // 2, :-1] = 0.999
    acc, out = kda.verify_drafts(target, tokens, u, draft=draft)
    ref, token = by_sums(target, draft, tokens, u)
    assert torch.equal(acc.long(), ref)
    assert torch.equal(out.gather(1, ref[:, None])[:, 0].long(), token)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("certain", [False, True])
@pytest.mark.parametrize("V", [3001, 2048, 5])
def test_padded_and_shifted_rows(V, certain, dtype):
    """Rows that lie apart, that begin on 16 bytes or not, p and q on the same place of them or not: the same tokens."""
    target, draft, tokens, u = draft_inputs(6, 4, V, seed=3, dtype=dtype, certain=certain)
    want = verify(target, draft, tokens, u)
    assert list(want[:2]) == list(verify_ref(target, tokens, u, draft))
    for pad, shift, other in ((7, 0, 0), (7, 1, 1), (1, 3, 0), (71, 2, 5), (0, 7, 6), (8, 0, 1), (13, 4, 4)):
        t = torch.full((6, 4, V + pad + shift), float("nan"), dtype=dtype)
        t[:, :, shift:shift + V] = target
        t, q = t.to(DEV)[:, :, shift:shift + V], None
        if draft is not None:
            q = torch.full((6, 3, V + pad + other), float("nan"), dtype=dtype)
            q[:, :, other:other + V] = draft
            q = q.to(DEV)[:, :, other:other + V]
        acc, out = kda.verify_drafts(t, tokens.to(DEV), u.to(DEV), draft=q)
        assert acc.tolist() == want[0] and out.tolist() == want[1]


def test_edges_of_the_uniform_numbers():
    """r = 0: the first token with weight; the largest number under 1, 1 and more: the last; below 0 and NaN: as 0."""
    p = torch.tensor([0.0, 0.25, 0.0, 0.5, 0.25, 0.0]).view(1, 1, 6).repeat(6, 1, 1)
    u = torch.tensor([0.0, 1 - 2.0 ** -24, 1.0, 7.0, -3.0, float("nan")]).view(6, 1)
    acc, out, err = verify(p, None, torch.empty(6, 0, dtype=torch.int32), u)
    assert err == 0 and acc == [0] * 6 and [x[0] for x in out] == [1, 4, 4, 4, 1, 1]
    # on a border the sum has to pass the bound
    p = torch.tensor([0.25, 0.25, 0.5]).view(1, 1, 3).repeat(4, 1, 1)
    u = torch.tensor([0.25, 0.5, 0.25 - 2.0 ** -26, 0.75]).view(4, 1)
    assert [x[0] for x in verify(p, None, torch.empty(4, 0, dtype=torch.int32), u)[1]] == [1, 2, 0, 2]


def test_edges_of_the_tests():
    """u q < p: equal is refused; p = 0 is refused even by u = 0; q = 0 stands where p > 0."""
    p = torch.tensor([[[0.5, 0.5], [0.5, 0.5]]]).repeat(4, 1, 1)
    q = torch.tensor([[[1.0, 0.0]]]).repeat(4, 1, 1)
    tokens = torch.tensor([[0], [0], [1], [0]], dtype=torch.int32)
    u = torch.tensor([[0.5, 0.3], [0.5 - 2.0 ** -25, 0.3], [0.9, 0.3], [0.0, 0.9]])
    acc, out, err = verify(p, q, tokens, u)
    assert err == 0 and acc == [0, 1, 1, 1] and out == [[1, -1], [0, 0], [1, 0], [0, 1]]
    zero = torch.tensor([[[0.0, 1.0], [1.0, 0.0]]])
    acc, out, err = verify(zero, None, torch.tensor([[0]], dtype=torch.int32), torch.zeros(1, 2))
    assert err == 0 and acc == [0] and out == [[1, -1]]


def test_nothing_left_beside_the_draft():
    """p covered by q all over (or on the certain draft alone): drawn from p itself."""
    p = torch.tensor([[[0.5, 0.5, 0.0], [0.0, 0.0, 1.0]]])
    acc, out, err = verify(p, p[:, :1] * 1.0, torch.tensor([[2]], dtype=torch.int32), torch.tensor([[0.5, 0.7]]))
    assert err == 0 and acc == [0] and out == [[1, -1]]
    p = torch.tensor([[[0.25, 0.0, 0.0], [0.0, 0.0, 1.0]]])
    acc, out, err = verify(p, None, torch.tensor([[0]], dtype=torch.int32), torch.tensor([[0.5, 0.7]]))
    assert err == 0 and acc == [0] and out == [[0, -1]]


def test_what_is_wrong_on_the_device():
    target, draft, tokens, u = draft_inputs(4, 3, 50, seed=7)
    tokens[0, 0], tokens[1, 1], u[1, 0] = 50, -1, 0.0
    for q in (draft, None):
        acc, out, err = verify(target, q, tokens, u)
        assert err == drafts.DEVERR_TOKEN
        assert acc[0] == 0 and acc[1] <= 1 and 0 <= out[0][0] < 50
        ref = verify_ref(target[2:], tokens[2:], u[2:], None if q is None else q[2:])
        assert acc[2:] == ref[0] and out[2:] == ref[1]
    target, draft, tokens, u = draft_inputs(4, 3, 50, seed=8)
    acc, out, err = verify(target, draft, tokens, u, torch.tensor([2, 3, -1, 0], dtype=torch.int32))
    assert err == 2  # KDA_DEVERR_NUM_ACCEPTED
    assert acc[1:3] == [0, 0] and out[1] == out[2] == [-1] * 3
    ref = verify_ref(target[[0, 3]], tokens[[0, 3]], u[[0, 3]], draft[[0, 3]], [2, 0])
    assert [acc[0], acc[3]] == ref[0] and [out[0], out[3]] == ref[1]
    target[2] = 0
    acc, out, err = verify(target, draft, tokens, u)
    assert err == drafts.DEVERR_PROBS and acc[2] == 0 and out[2] == [-1] * 3


def test_values_that_are_no_probabilities():
    """NaN and negative values weigh nothing, and a test against NaN is refused."""
    nan = float("nan")
    p = torch.tensor([[[nan, 0.5, -1.0, 0.5], [0.0, 0.0, nan, 1.0]]])
    q = torch.tensor([[[0.5, nan, 0.0, 0.5]]])
    acc, out, err = verify(p, q, torch.tensor([[0]], dtype=torch.int32), torch.tensor([[0.0, 0.9]]))
    assert err == 0 and acc == [0] and out == [[1, -1]]
    acc, out, err = verify(p, None, torch.tensor([[1]], dtype=torch.int32), torch.tensor([[0.1, 0.0]]))
    assert err == 0 and acc == [1] and out == [[1, 3]]


@pytest.mark.parametrize("n", [3, 100])
def test_rows_that_sum_to_too_much(n):
    """No answer, but a token or -1, and nothing read or written elsewhere."""
    target = torch.ones(n, 2, 5000, device=DEV)
    tokens = torch.zeros(n, 1, dtype=torch.int32, device=DEV)
    for draft in (None, 0.5 * target[:, :1]):
        for r in (0.0, 0.3, 0.77, 1.0):
            acc, out = kda.verify_drafts(target, tokens, torch.full((n, 2), r, device=DEV), draft=draft)
            assert ((out >= -1) & (out < 5000)).all() and ((acc >= 0) & (acc <= 1)).all()


@pytest.mark.parametrize("V", [7, 600, 5003])
@pytest.mark.parametrize("n", [77, 1000])
def test_many_requests(n, V):
    """Over the number that get a cluster each: a line of all their segments."""
    target, draft, tokens, u = draft_inputs(n, 3, V, seed=n + V)
    target[5], target[n - 1, 2] = 0, 0
    draft[7] = target[7, :2]  # (refused with nothing left beside: p itself)
    u[7, 0], tokens[9, 1] = 0.9999999, V
    m = (torch.arange(n) % 3).int()
    m[11], m[13] = 3, -1
    acc, out, err = verify(target, draft, tokens, u, m)
    keep = [i for i in range(min(n, 150)) if i not in (5, 9, 11, 13)]
    ref = verify_ref(target[keep], tokens[keep], u[keep], draft[keep], m[keep])
    assert [acc[i] for i in keep] == ref[0] and [out[i] for i in keep] == ref[1]
    assert acc[5] == 0 and out[5] == out[11] == out[13] == [-1] * 3
    assert err & ~drafts.DEVERR_TOKEN == 2 | drafts.DEVERR_PROBS
    # as in calls of few requests
    for at in range(0, n, 70):
        s = slice(at, at + 70)
        a, o, _ = verify(target[s], draft[s], tokens[s], u[s], m[s])
        assert a == acc[s] and o == out[s]
    p = draft_inputs(n, 3, V, seed=3, certain=True)
    assert list(verify(*p)[:2]) == [sum(x, []) for x in zip(*(verify(*(None if t is None else t[i:i + 60] for t in p))[:2]
                                                              for i in range(0, n, 60)))]


def test_the_law():
    """Whatever the draft, the first token is distributed as the target says: 200,000 requests, every share within
    5 standard deviations."""
    n = 200_000
    g = torch.Generator().manual_seed(12)
    p = torch.tensor([0.4, 0.3, 0.05, 0.2, 0.05, 0.0])
    q = torch.tensor([0.1, 0.5, 0.1, 0.0, 0.1, 0.2])
    tokens = torch.multinomial(q.repeat(n, 1), 1, generator=g).int()
    u = torch.rand(n, 2, generator=g)
    t, d = p.view(1, 1, 6).expand(n, 2, 6).contiguous(), q.view(1, 1, 6).expand(n, 1, 6).contiguous()
    acc, out = kda.verify_drafts(t.to(DEV), tokens.to(DEV), u.to(DEV), draft=d.to(DEV))
    share = torch.bincount(out[:, 0].cpu(), minlength=6).double() / n
    assert ((share - p.double()).abs() <= 5 * (p.double() * (1 - p.double()) / n).sqrt()).all()
    kept = torch.minimum(p, q).sum().item()  # accepted with this probability
    assert abs(acc.double().mean().item() - kept) <= 5 * (kept * (1 - kept) / n) ** 0.5


def test_writes_nothing_else_and_replays():
    target, draft, tokens, u = dev(*draft_inputs(9, 5, 20_000, seed=5))
    lib = paged._lib()
    acc, out = Guarded((9,), torch.int32), Guarded((9, 5), torch.int32)
    ws = Guarded((kda.verify_drafts_workspace_size(9, 5, 20_000),), torch.uint8)
    p = lambda x: x.data_ptr()  # noqa: E731

    def call():
        rc = lib.kda_verify_drafts(p(target), p(draft), p(tokens), p(u), None, 9, 5, 20_000, 1, 100_000, 20_000, 80_000, 20_000, p(acc.t),
                                   p(out.t), p(ws.t), ws.t.nbytes, None, torch.cuda.current_stream().cuda_stream)
        assert rc == 0

    call()
    want = kda.verify_drafts(target, tokens, u, draft=draft)
    assert acc.intact() and out.intact() and ws.intact()
    assert torch.equal(acc.t, want[0]) and torch.equal(out.t, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    fresh = draft_inputs(9, 5, 20_000, seed=6)
    for a, b in zip((target, draft, tokens, u), fresh):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    want = kda.verify_drafts(target, tokens, u, draft=draft)
    assert torch.equal(acc.t, want[0]) and torch.equal(out.t, want[1])


def test_plain_binding_and_refusals(monkeypatch):
    target, draft, tokens, u = dev(*draft_inputs(6, 4, 500, seed=2))
    want = kda.verify_drafts(target, tokens, u, draft=draft)
    bad = [dict(target=target.half()), dict(target=target[0]), dict(draft=draft.bfloat16()), dict(draft=draft[:, :2]),
           dict(draft_tokens=tokens.long()), dict(draft_tokens=tokens[:, :2].contiguous()), dict(uniforms=u.double()),
           dict(uniforms=u[:, :3].contiguous()), dict(n_draft=tokens[0].contiguous()), dict(n_draft=u[0].contiguous()),
           dict(target=target.cpu()), dict(target=target.transpose(1, 2)), dict(target=target[:, :, ::2].expand(6, 4, 250)),
           dict(target=torch.zeros(6, 33, 4, device=DEV), draft_tokens=torch.zeros(6, 32, dtype=torch.int32, device=DEV),
                uniforms=torch.zeros(6, 33, device=DEV), draft=None)]
    for kw in bad:
        a = dict(target=target, draft_tokens=tokens, uniforms=u, draft=draft)
        a.update(kw)
        with pytest.raises(kda.KDAError):
            kda.verify_drafts(**a)
    monkeypatch.setattr(paged, "_fast_verify", lambda *a: None)
    got = kda.verify_drafts(target, tokens, u, draft=draft)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_calls_on_two_streams_at_once():
    """Each with a workspace of its own (the binding's, or the caller's)."""
    sets = [dev(*draft_inputs(150, 4, 30_000, seed=i)) for i in range(2)]
    want = [kda.verify_drafts(t, d, u, draft=q) for t, q, d, u in sets]
    size = kda.verify_drafts_workspace_size(150, 4, 30_000)
    ws = [torch.empty(size, dtype=torch.uint8, device=DEV) for _ in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    out = [[], []]
    for i in range(20):
        for k, (t, q, d, u) in enumerate(sets):
            with torch.cuda.stream(streams[k]):
                out[k].append(kda.verify_drafts(t, d, u, draft=q, workspace=ws[k] if i % 2 else None))
    torch.cuda.synchronize()
    for k in range(2):
        for acc, tokens in out[k]:
            assert torch.equal(acc, want[k][0]) and torch.equal(tokens, want[k][1])


def test_requests_that_share_their_rows():
    """A stride of zero: one distribution for all requests."""
    p, q, tokens, u = draft_inputs(1, 3, 5000, seed=4)
    n = 200
    g = torch.Generator().manual_seed(1)
    u, tokens = torch.rand(n, 3, generator=g), tokens.repeat(n, 1)
    wide = verify(p.repeat(n, 1, 1), q.repeat(n, 1, 1), tokens, u)
    acc, out = kda.verify_drafts(p.to(DEV).expand(n, 3, 5000), tokens.to(DEV), u.to(DEV), draft=q.to(DEV).expand(n, 2, 5000))
    assert acc.tolist() == wide[0] and out.tolist() == wide[1]


def padded(x, pad, value, shift=0):
    """x on the device, its rows between others' values."""
    wide = torch.full((*x.shape[:2], shift + x.shape[2] + pad), value, dtype=x.dtype)
    wide[:, :, shift:shift + x.shape[2]] = x
    return wide.to(DEV)[:, :, shift:shift + x.shape[2]]


def with_no_token(x):
    """One place more, of no weight: what a drafted token outside the vocabulary stands for."""
    return torch.cat((x, x.new_zeros(*x.shape[:2], 1)), 2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("certain", [True, False])
@pytest.mark.parametrize("V", [1, 16, 50, 250, 1030])
def test_drafted_tokens_past_the_vocabulary(V, certain, dtype):
    """Refused, recorded, and without a say in the token that follows, whatever stands behind the row: places up to
    the end of its last piece, the next row's, far ones."""
    away = [V, V + 1, V + 2, 255, 256, 511, 512, 1023, 1024, 2047, 2048, 2 ** 31 - 1, 2 ** 31 - 8, -1, -2 ** 31]
    away = [d for d in away if d < 0 or d >= V]
    n, w = 3 * len(away), 3
    target, draft, tokens, u = draft_inputs(n, w, V, seed=V, dtype=dtype, certain=certain)
    for i, d in enumerate(3 * away):
        at = i % 2
        tokens[i, at], u[i, :at] = d, 0.0
        u[i, w - 1] = (1 - 2.0 ** -24, 0.5, 0.97)[i // len(away)]
    outside = (tokens < 0) | (tokens >= V)
    ref = verify_ref(with_no_token(target), torch.where(outside, V, tokens), u, None if draft is None else with_no_token(draft))
    assert all(a <= i % 2 for i, a in enumerate(ref[0]))
    for pad, value, shift in ((0, 0.0, 0), (40, 1.0, 0), (3, 1.0, 1), (2100, 0.25, 4), (2100, float("nan"), 0)):
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        acc, out = kda.verify_drafts(padded(target, pad, value, shift), tokens.to(DEV), u.to(DEV),
                                     draft=None if draft is None else padded(draft, pad, value), error_word=err)
        assert int(err) == drafts.DEVERR_TOKEN
        assert acc.tolist() == ref[0] and out.tolist() == ref[1]


@pytest.mark.parametrize("n,V,dtype", [(60, 70_001, F32), (110, 70_001, BF16), (3, 70_001, F32)])
def test_drafted_tokens_past_a_large_vocabulary(n, V, dtype):
    """The same in rows of many pieces, of either size."""
    g = torch.Generator(device=DEV).manual_seed(n)
    target = (2 * torch.randn(n, 2, V, generator=g, device=DEV)).softmax(2).to(dtype)
    tokens = (V + torch.arange(n, device=DEV) % 3 * 300).int()[:, None]
    u = torch.rand(n, 2, generator=g, device=DEV)
    u[: n // 2, 1] = 1 - 2.0 ** -24
    wide = torch.full((n, 2, V + 700), 0.5, dtype=dtype, device=DEV)
    wide[:, :, :V] = target
    acc, out = kda.verify_drafts(wide[:, :, :V], tokens, u)
    ref, token = by_sums(with_no_token(target), None, torch.full_like(tokens, V), u)
    assert (acc == 0).all() and (ref == 0).all()
    assert torch.equal(out[:, 0].long(), token)


def test_one_workspace_for_shrinking_batches():
    """That of 40 requests does for 28, which take smaller pieces and more of them, and for one."""
    V, w = 131_072, 2
    ws = torch.empty(kda.verify_drafts_workspace_size(40, w, V), dtype=torch.uint8, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    target = (2 * torch.randn(40, w, V, generator=g, device=DEV)).softmax(2)
    tokens, u = target[:, :1].argmax(2).int(), torch.rand(40, w, generator=g, device=DEV)
    u[:20, 0] = 0.9999
    ref, token = by_sums(target, None, tokens, u)
    for n in (40, 28, 29, 7, 1):
        acc, out = kda.verify_drafts(target[:n], tokens[:n], u[:n], workspace=ws)
        assert torch.equal(acc.long(), ref[:n]) and torch.equal(out.gather(1, ref[:n, None])[:, 0].long(), token[:n])
