"""moe_balance_loss and moe_router_backward against the formulas in float64.

Tolerances, with u = 2^-24 (half a step of float32).  An exponential of
v - max carries |v - max| u from its argument (at most 2^5 u here, the scores
lie within 32 of their maximum wherever p matters) and a few u of its own, a
row sum 16 + 6, so a probability is off by at most C = 64 roundings of its
value.  A loss adds non-negative terms: another T / 16 + 64 roundings for
the sums over the tokens.  lse is off by 8 u (|max| + log E), its square by
twice |lse| times that.  The gradient is a sum of a few such products."""

import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
C = 64


def make(T, E, k, S=1, mask=False, seed=0, spread=1.5, tail=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    scores = spread * torch.randn(T, E, generator=g, device="cuda")
    bias = 0.5 * torch.randn(E, generator=g, device="cuda")
    c = {"scores": scores, "ids": torch.topk(scores + bias, k, dim=1).indices.to(torch.int32),
         "mask": None, "offsets": None, "S": S}
    c["weights"] = torch.softmax(torch.gather(scores, 1, c["ids"].long()), 1)
    c["grad_weights"] = torch.randn(T, k, generator=g, device="cuda")
    c["grad_loss"] = torch.randn(S, 2, generator=g, device="cuda")
    if mask:
        c["mask"] = torch.rand(T, generator=g, device="cuda") < 0.7
    if S > 1:
        cuts = torch.sort((torch.rand(S + 1, generator=g, device="cuda") * (T + 1)).int()).values
        if not tail:
            cuts[0], cuts[-1] = 0, T
        c["offsets"] = cuts
    return c


def reference(c, grad_loss=True, grad_weights=True):
    s = c["scores"].double().cpu()
    ids = c["ids"].cpu().long()
    T, E = s.shape
    k, S = ids.shape[1], c["S"]
    ids = torch.where((ids >= 0) & (ids < E), ids, 0)
    valid = torch.ones(T, dtype=torch.bool) if c["mask"] is None else c["mask"].cpu().bool()
    cuts = [0, T] if c["offsets"] is None else c["offsets"].cpu().tolist()
    counts = torch.zeros(S, E, dtype=torch.int64)
    tokens = torch.zeros(S, dtype=torch.int64)
    loss, tol = torch.zeros(S, 2, dtype=torch.float64), torch.zeros(S, 2, dtype=torch.float64)
    grad, gtol = torch.zeros(T, E, dtype=torch.float64), torch.zeros(T, E, dtype=torch.float64)
    gl = c["grad_loss"].double().cpu()
    for q in range(S):
        rows = [t for t in range(cuts[q], cuts[q + 1]) if valid[t] and bool((s[t] > -math.inf).any())]
        n = len(rows)
        tokens[q] = n
        if n == 0:
            continue
        v = s[rows]
        counts[q] = torch.bincount(ids[rows].reshape(-1), minlength=E)
        p = torch.softmax(v, 1)
        m = v.max(1).values
        lse = torch.logsumexp(v, 1)
        f = counts[q].double() * E / (k * n)
        loss[q, 0] = (f * p.mean(0)).sum()
        loss[q, 1] = lse.square().mean()
        off = 8 * U * (m.abs() + math.log(E) + 1)
        adds = (C + n / 16 + 64) * U
        tol[q, 0] = adds * loss[q, 0]
        tol[q, 1] = adds * loss[q, 1] + (2 * lse.abs() * off + off * off).mean()
        if grad_loss:
            fp = (f * p).sum(1, keepdim=True)
            grad[rows] = p / n * (gl[q, 0] * (f - fp) + 2 * gl[q, 1] * lse[:, None])
            size = p / n * (gl[q, 0].abs() * (f + fp) + 2 * gl[q, 1].abs() * lse.abs()[:, None])
            gtol[rows] = 4 * C * U * size + p / n * 2 * gl[q, 1].abs() * off[:, None]
    if grad_weights:
        w, dw = c["weights"].double().cpu(), c["grad_weights"].double().cpu()
        d = w * (dw - (w * dw).sum(1, keepdim=True))
        grad.scatter_add_(1, ids, d)
        size = w * (dw.abs() + (w * dw).abs().sum(1, keepdim=True))
        gtol.scatter_add_(1, ids, (2 * k + 8) * U * size)
    return counts, tokens, loss, tol, grad, gtol + 2 * U * grad.abs() + 1e-37


def check(lib, c, backward=True):
    ref_counts, ref_tokens, ref_loss, tol, grad, gtol = reference(c)
    loss, counts, tokens = lib.balance_loss(c["scores"], c["ids"], mask=c["mask"],
                                            seq_offsets=c["offsets"])
    assert torch.equal(counts.cpu().long(), ref_counts)
    assert torch.equal(tokens.cpu().long(), ref_tokens)
    err = (loss.double().cpu() - ref_loss).abs()
    assert bool((err <= tol + 1e-37).all()), (err / tol, loss)
    if not backward:
        return loss, counts, tokens
    out = torch.full_like(c["scores"], 7.0)
    got = lib.router_backward(c["scores"], c["ids"], grad_loss=c["grad_loss"], counts=counts,
                              tokens=tokens, mask=c["mask"], seq_offsets=c["offsets"],
                              weights=c["weights"], grad_weights=c["grad_weights"], out=out)
    assert got is out
    err = (got.double().cpu() - grad).abs()
    assert bool((err <= gtol).all()), float((err / gtol).max())
    return loss, counts, tokens, got


SHAPES = [(1, 1, 1), (1, 128, 8), (2, 3, 2), (17, 64, 8), (32, 128, 8), (33, 70, 7), (64, 256, 8),
          (255, 257, 8), (300, 96, 6), (257, 255, 5), (129, 512, 8), (70, 513, 9), (40, 1024, 64),
          (1000, 8, 2), (2000, 128, 8), (700, 1001, 3), (513, 66, 64)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("S,mask", [(1, False), (3, True), (9, False)])
def test_against_the_formulas(lib, T, E, k, S, mask):
    check(lib, make(T, E, k, S, mask, seed=T + E + S))


@pytest.mark.parametrize("T,S", [(20000, 1), (16384, 40), (9001, 700)])
def test_many_tokens(lib, T, S):
    check(lib, make(T, 128, 8, S, True, seed=T, tail=False))


def test_even_routing_has_loss_one(lib):
    T, E, k = 128, 64, 4
    scores = torch.zeros(T, E, device="cuda")
    ids = (torch.arange(T * k, device="cuda", dtype=torch.int32) % E).view(T, k)
    loss, counts, tokens = lib.balance_loss(scores, ids)
    assert bool((counts == T * k // E).all()) and int(tokens[0]) == T
    assert abs(float(loss[0, 0]) - 1) <= (C + T) * U
    assert abs(float(loss[0, 1]) - math.log(E) ** 2) <= (C + T) * U * math.log(E) ** 2


def test_masked_rows_are_not_read(lib):
    c = make(300, 128, 8, 4, True, seed=3)
    want = check(lib, c)
    off = ~c["mask"]
    c["scores"][off] = float("nan")
    c["scores"][off.nonzero()[0]] = float("inf")
    got_loss, got_counts, _ = lib.balance_loss(c["scores"], c["ids"], mask=c["mask"],
                                               seq_offsets=c["offsets"])
    assert torch.equal(got_loss, want[0]) and torch.equal(got_counts, want[1])
    grad = lib.router_backward(c["scores"], c["ids"], grad_loss=c["grad_loss"], counts=want[1],
                               tokens=want[2], mask=c["mask"], seq_offsets=c["offsets"])
    assert not grad[off].any() and bool(torch.isfinite(grad).all())


def test_nothing_left(lib):
    """A mask without a token, and rows without a score."""
    c = make(50, 32, 4, 3, False, seed=5, tail=False)
    c["mask"] = torch.zeros(50, dtype=torch.bool, device="cuda")
    loss, counts, tokens, grad = check(lib, c)
    assert not loss.any() and not counts.any() and not tokens.any()
    c["mask"] = None
    c["scores"][7] = -math.inf
    c["scores"][8, 1:] = -math.inf
    c["ids"][8] = torch.tensor([0, 1, 2, 3])
    check(lib, c)


def test_experts_taken_out(lib):
    c = make(90, 100, 6, 2, False, seed=6)
    c["scores"][:, 40:60] = -math.inf
    c["scores"][:, 3] = torch.finfo(torch.float32).min
    c["ids"] = torch.topk(c["scores"], 6, dim=1).indices.to(torch.int32)
    loss, counts, tokens, grad = check(lib, c)
    assert not counts[:, 40:60].any() and not grad[:, 40:60].any() and not grad[:, 3].any()


def test_offsets_outside_and_empty_sequences(lib):
    c = make(100, 64, 4, 6, seed=7)
    c["offsets"] = torch.tensor([10, 10, 40, 40, 40, 90, 90], dtype=torch.int32, device="cuda")
    loss, counts, tokens, grad = check(lib, c)
    assert tokens.tolist() == [0, 30, 0, 0, 50, 0]
    only = lib.router_backward(c["scores"], c["ids"], grad_loss=c["grad_loss"], counts=counts,
                               tokens=tokens, seq_offsets=c["offsets"])
    assert not only[:10].any() and not only[90:].any()
    # the same in the form with more than one workgroup
    d = make(5000, 64, 4, 6, seed=8)
    d["offsets"] = torch.tensor([10, 10, 2040, 2040, 2040, 4090, 4090], dtype=torch.int32, device="cuda")
    check(lib, d)
    # bounds past the batch are read as its end
    c["offsets"] = torch.tensor([-5, 20, 40, 60, 80, 100, 1 << 30], dtype=torch.int32, device="cuda")
    got = lib.balance_loss(c["scores"], c["ids"], seq_offsets=c["offsets"])
    assert got[2].tolist() == [20, 20, 20, 20, 20, 0]


@pytest.mark.parametrize("T,E,k", [(40, 64, 8), (30, 300, 20), (9, 1000, 64)])
def test_repeated_and_foreign_ids(lib, T, E, k):
    """Two slots of one expert count twice and add their gradients; an id out
    of range is read as expert 0, as everywhere in the library."""
    c = make(T, E, k, seed=9)
    c["ids"][::2, 1] = c["ids"][::2, 0]
    c["ids"][::3, 2:6] = c["ids"][::3, 0:1]
    c["ids"][1::4, -1] = -1
    c["ids"][2::4, -1] = E
    a = check(lib, c)
    b = check(lib, c)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_parts_of_the_gradient(lib):
    c = make(77, 130, 5, 2, True, seed=10)
    loss, counts, tokens, both = check(lib, c)
    kw = dict(counts=counts, tokens=tokens, mask=c["mask"], seq_offsets=c["offsets"])
    one = lib.router_backward(c["scores"], c["ids"], grad_loss=c["grad_loss"], **kw)
    two = lib.router_backward(c["scores"], c["ids"], weights=c["weights"],
                              grad_weights=c["grad_weights"])
    _, _, _, _, g1, t1 = reference(c, grad_weights=False)
    _, _, _, _, g2, t2 = reference(c, grad_loss=False)
    assert bool(((one.double().cpu() - g1).abs() <= t1).all())
    assert bool(((two.double().cpu() - g2).abs() <= t2).all())
    assert bool(((one + two - both).abs() <= 4 * U * (one.abs() + two.abs()) + 1e-37).all())


def test_gradient_against_differences(lib):
    """Along a random direction, the float64 losses with the counts held and
    the float64 softmax over the selected scores; h^2 = 1e-8."""
    c = make(40, 96, 6, 2, seed=11, tail=False)
    loss, counts, tokens, grad = check(lib, c)
    gl, dw = c["grad_loss"].double(), c["grad_weights"].double()
    cuts = c["offsets"].tolist()

    def value(s):
        total = (torch.softmax(torch.gather(s, 1, c["ids"].long()), 1) * dw).sum()
        for q in range(2):
            rows = s[cuts[q]:cuts[q + 1]]
            n = rows.shape[0]
            f = counts[q].double() * 96 / (6 * n)
            total = total + gl[q, 0] * (f * torch.softmax(rows, 1).mean(0)).sum()
            total = total + gl[q, 1] * torch.logsumexp(rows, 1).square().mean()
        return float(total)

    gen = torch.Generator(device="cuda").manual_seed(1)
    v = torch.randn(40, 96, generator=gen, device="cuda", dtype=torch.float64)
    s = c["scores"].double()
    want = (value(s + 1e-4 * v) - value(s - 1e-4 * v)) / 2e-4
    have = float((grad.double() * v).sum())
    assert abs(have - want) <= 2e-6 * float((grad.double() * v).abs().sum()) + 1e-6


def test_unaligned_scores(lib):
    c = make(50, 128, 8, seed=12)
    want = check(lib, c)
    base = torch.empty(50 * 128 + 1, device="cuda")
    base[1:] = c["scores"].reshape(-1)
    c["scores"] = base[1:].view(50, 128)
    got = check(lib, c)
    assert torch.equal(got[1], want[1])


def test_no_tokens(lib):
    scores = torch.empty((0, 16), device="cuda")
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    loss, counts, tokens = lib.balance_loss(scores, ids, seq_offsets=off)
    assert loss.shape == (3, 2) and counts.shape == (3, 16) and tokens.shape == (3,)
    assert not loss.any() and not counts.any() and not tokens.any()
    g = lib.router_backward(scores, ids, grad_loss=torch.ones(1, 2, device="cuda"),
                            counts=counts[:1].contiguous(), tokens=tokens[:1].contiguous())
    assert g.shape == (0, 16)


def test_past_32_bit_offsets(lib):
    """More than 2^31 scores, all equal: closed forms."""
    T, E, k = 2 * 1024 * 1024 + 5, 1024, 2
    scores = torch.zeros((T, E), device="cuda")
    ids = (torch.arange(T * k, device="cuda") % 512).to(torch.int32).view(T, k)
    loss, counts, tokens = lib.balance_loss(scores, ids)
    want = torch.bincount(ids.view(-1).long(), minlength=E)
    assert torch.equal(counts[0].long(), want) and int(tokens[0]) == T
    # equal terms: the partial sums' roundings are at most one for each addition
    adds = (T / 16 / 256 + 512) * U
    lse = math.log(E)
    assert abs(float(loss[0, 0]) - 1) <= adds and abs(float(loss[0, 1]) / lse ** 2 - 1) <= adds
    gl = torch.tensor([[0.0, 1.0]], device="cuda")
    grad = lib.router_backward(scores, ids, grad_loss=gl, counts=counts, tokens=tokens)
    exact = 2 * lse / (T * E)
    for t in (0, T // 2, T - 1):
        assert bool(((grad[t].double() / exact - 1).abs() <= C * U).all())


def test_captured_and_replayed(lib):
    c = make(3000, 128, 8, 5, True, seed=13)
    out = torch.empty_like(c["scores"])

    def step():
        loss, counts, tokens = lib.balance_loss(c["scores"], c["ids"], mask=c["mask"],
                                                seq_offsets=c["offsets"])
        lib.router_backward(c["scores"], c["ids"], grad_loss=c["grad_loss"], counts=counts,
                            tokens=tokens, mask=c["mask"], seq_offsets=c["offsets"],
                            weights=c["weights"], grad_weights=c["grad_weights"], out=out)
        return loss, counts, tokens

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        d = make(3000, 128, 8, 5, True, seed=50 + i)
        for name in ("scores", "ids", "mask", "offsets", "weights"):
            c[name].copy_(d[name])
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held] + [out.clone()]
        want = list(step()) + [out]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_route_then_balance(lib):
    """Scores through the library's own router, its counts and its gradient."""
    from oracle import router as R
    rng = np.random.default_rng(2)
    scores = rng.standard_normal((200, 128)).astype(np.float32)
    bias = rng.normal(0, 0.5, 128).astype(np.float32)
    s = torch.from_numpy(scores).cuda()
    ids, w = lib.topk_route(s, 8, bias=torch.from_numpy(bias).cuda())
    ref_ids, _ = R.topk_route(scores, 8, bias)
    _, counts, _ = lib.balance_loss(s, ids)
    assert np.array_equal(counts[0].cpu().numpy(), np.bincount(ref_ids.reshape(-1), minlength=128))
    g = torch.Generator(device="cuda").manual_seed(0)
    c = {"scores": s, "ids": ids, "weights": w, "mask": None, "offsets": None, "S": 1,
         "grad_weights": torch.randn(200, 8, generator=g, device="cuda"),
         "grad_loss": torch.ones(1, 2, device="cuda")}
    check(lib, c)


def test_refusals(lib):
    c = make(8, 16, 2, seed=14)
    with pytest.raises(ValueError):
        lib.balance_loss(c["scores"].to(torch.bfloat16), c["ids"])
    with pytest.raises(ValueError):
        lib.balance_loss(c["scores"], c["ids"].long())
    with pytest.raises(ValueError):
        lib.balance_loss(c["scores"].t(), c["ids"])
    with pytest.raises(ValueError):
        lib.balance_loss(c["scores"], c["ids"], mask=torch.ones(7, dtype=torch.bool, device="cuda"))
    with pytest.raises(lib.MoeError):   # neither gradient
        lib.router_backward(c["scores"], c["ids"])
    with pytest.raises(lib.MoeError):   # weights without their gradient
        lib.router_backward(c["scores"], c["ids"], weights=c["weights"])


def test_no_tokens_many_sequences(lib):
    """An empty batch that is split over more sequences than one workgroup takes."""
    scores = torch.empty((0, 130), device="cuda")
    ids = torch.empty((0, 2), dtype=torch.int32, device="cuda")
    loss, counts, tokens = lib.balance_loss(scores, ids,
                                            seq_offsets=torch.zeros(8, dtype=torch.int32, device="cuda"))
    assert loss.shape == (7, 2) and not loss.any() and not counts.any() and not tokens.any()


@pytest.mark.parametrize("T,S", [(40, 2), (3000, 6)])
@pytest.mark.parametrize("other", [0.25, -math.inf])
def test_nan_scores_reach_their_sequence_alone(lib, T, S, other):
    c = make(T, 16, 2, S=S, tail=False, seed=5)
    cuts = c["offsets"].tolist()
    q = max(range(S), key=lambda i: cuts[i + 1] - cuts[i])
    row = (cuts[q] + cuts[q + 1]) // 2
    c["scores"][row] = other
    clean = lib.balance_loss(c["scores"], c["ids"], seq_offsets=c["offsets"])[0]
    c["scores"][row, 3] = float("nan")
    loss = lib.balance_loss(c["scores"], c["ids"], seq_offsets=c["offsets"])[0]
    for i in range(S):
        if i == q:
            assert bool(loss[i].isnan().all())
        else:
            assert torch.equal(loss[i], clean[i])


def test_first_tensor_by_keyword(lib):
    c = make(33, 16, 2)
    a = lib.balance_loss(c["scores"], c["ids"])
    b = lib.balance_loss(ids=c["ids"], scores=c["scores"], stream=torch.cuda.current_stream())
    assert all(torch.equal(x, y) for x, y in zip(a, b))
