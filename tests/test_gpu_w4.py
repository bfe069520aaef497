"""moe_w4_linear against the float64 product of the weights the codes stand for.

Tolerances, u = 2^-24 (half a step of float32).  code * x is exact.  A group's
two sums (of code x and of x) are added in at most G / 32 matrix instructions
of 32 products, the groups of a wavefront, then the wavefronts: a value takes
at most K / 32 + 32 roundings, of sums no larger than |s| (15 + z) sum |x| per
group.  SwiGLU and the routing weight add 16 roundings of their result, and
what their inputs were off by, times their slopes (|SiLU'| <= 1.1).  A BF16
result is off by half its step, 2^-8 of its value, more."""

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


def make(T, N, K, G, scale=BF16, zero=True, E=1, k=0, slots=False, weights=False, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = {"q": torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
         "scale": ((0.5 + torch.rand(E, N, K // G, generator=g, device="cuda")) / K ** 0.5).to(scale),
         "zero": None, "ids": None, "weights": None, "G": G}
    if zero:
        c["zero"] = torch.randint(0, 16, (E, N, K // G), generator=g, device="cuda", dtype=torch.uint8)
    c["x"] = torch.randn((T, k, K) if slots else (T, K), generator=g, device="cuda").to(BF16)
    if k:
        c["ids"] = torch.topk(torch.randn(T, E, generator=g, device="cuda"), k, dim=1).indices.int()
        if weights:
            c["weights"] = torch.rand(T, k, generator=g, device="cuda")
    return c


def dequantised(c):
    """Weights, and the sizes their rounding errors are measured by, float64."""
    q = c["q"].long()
    v = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.float64, device=q.device)
    v[..., 0::2], v[..., 1::2] = (q & 15).double(), (q >> 4).double()
    s = c["scale"].double().repeat_interleave(c["G"], -1)
    z = torch.full_like(s, 8.0) if c["zero"] is None else c["zero"].double().repeat_interleave(c["G"], -1)
    return (v - z) * s, (v + z) * s.abs()


def reference(c, swiglu):
    w, size = dequantised(c)
    x = c["x"].double()
    K = w.shape[-1]
    if c["ids"] is None:
        y, m = x @ w[0].t(), x.abs() @ size[0].t()
    else:
        T, k = c["ids"].shape
        E = w.shape[0]
        ids = c["ids"].long()
        ids = torch.where((ids >= 0) & (ids < E), ids, 0)
        rows = x if x.dim() == 3 else x[:, None].expand(T, k, K)
        y = torch.empty(T, k, w.shape[1], dtype=torch.float64, device=x.device)
        m = torch.empty_like(y)
        for t in range(T):
            for j in range(k):
                y[t, j] = w[ids[t, j]] @ rows[t, j]
                m[t, j] = size[ids[t, j]] @ rows[t, j].abs()
    tol = (K / 32 + 32) * U * m
    if swiglu:
        (g, u), (tg, tu) = y.chunk(2, -1), tol.chunk(2, -1)
        act = g * torch.sigmoid(g)
        y = act * u
        tol = 1.1 * tg * u.abs() + act.abs() * tu + 1.1 * tg * tu + (16 + 2 * g.abs()) * U * y.abs()
    if c["weights"] is not None:
        wt = c["weights"].double()[:, :, None]
        y, tol = y * wt, tol * wt + 2 * U * (y * wt).abs()
    return y, tol


def check(lib, c, swiglu=False, y_dtype="f32"):
    W = lib.W4Weights(c["q"], c["scale"], c["zero"])
    got = lib.w4_linear(W, c["x"], ids=c["ids"], weights=c["weights"], swiglu=swiglu, y_dtype=y_dtype)
    want, tol = reference(c, swiglu)
    assert got.shape == want.shape
    step = 2.0 ** -8 if y_dtype == "bf16" else 0.0
    err = (got.double() - want).abs()
    bound = tol + step * want.abs() + 1e-37
    assert bool((err <= bound).all()), float((err / bound).max())
    return got


DENSE = [(1, 1, 32, 32), (1, 16, 128, 128), (1, 17, 96, 32), (3, 33, 192, 64), (1, 4096, 2048, 128),
         (2, 100, 4096, 64), (5, 1001, 224, 32), (16, 48, 640, 128), (17, 257, 1024, 256),
         (32, 64, 2048, 32), (33, 31, 512, 64), (64, 515, 768, 128), (65, 80, 384, 128),
         (200, 130, 1024, 1024), (3, 40, 9216, 128), (20, 50, 5120, 64), (1, 33, 20480, 1024), (12, 20, 4224, 32),
         (4, 20000, 256, 64), (40, 17000, 160, 32), (20, 16500, 128, 128)]


@pytest.mark.parametrize("T,N,K,G", DENSE)
@pytest.mark.parametrize("scale,zero,y_dtype", [(BF16, False, "f32"), (F32, True, "f32"), (BF16, True, "bf16")])
def test_dense(lib, T, N, K, G, scale, zero, y_dtype):
    check(lib, make(T, N, K, G, scale, zero, seed=T + N + K), y_dtype=y_dtype)


@pytest.mark.parametrize("T,N,K,G", [(1, 2, 32, 32), (3, 70, 256, 64), (18, 96, 1024, 128), (50, 222, 448, 64)])
def test_dense_swiglu(lib, T, N, K, G):
    check(lib, make(T, N, K, G, F32, True, seed=N), swiglu=True)
    check(lib, make(T, N, K, G, BF16, False, seed=N), swiglu=True, y_dtype="bf16")


EXPERTS = [(1, 64, 128, 32, 8, 2), (5, 50, 256, 64, 3, 3), (32, 96, 512, 128, 16, 4), (40, 33, 224, 32, 4, 2),
           (64, 48, 256, 128, 2, 1), (200, 32, 128, 128, 5, 2), (1, 40, 128, 64, 1, 1), (256, 18, 96, 32, 64, 8),
           (2, 24, 18432, 128, 3, 2), (60, 20, 5120, 64, 4, 4)]


@pytest.mark.parametrize("T,N,K,G,E,k", EXPERTS)
@pytest.mark.parametrize("swiglu,slots", [(False, False), (True, False), (False, True)])
def test_experts(lib, T, N, K, G, E, k, swiglu, slots):
    if swiglu and N % 2:
        N += 1
    c = make(T, N, K, G, BF16, True, E, k, slots=slots, weights=slots, seed=T + E)
    check(lib, c, swiglu)
    check(lib, c, swiglu, "bf16")


def test_repeated_and_foreign_ids(lib):
    c = make(30, 64, 256, 64, BF16, True, 6, 4, seed=3)
    c["ids"][::2] = c["ids"][::2, :1]
    c["ids"][1::3, 2] = -7
    c["ids"][2::3, 3] = 6
    check(lib, c)


def test_all_entries_on_one_expert(lib):
    c = make(256, 48, 256, 128, BF16, False, 8, 8, seed=4)
    c["ids"].fill_(5)
    check(lib, c)


def test_same_bits_for_any_batch(lib):
    """A product's bits depend neither on the tokens beside it nor on the run."""
    c = make(12, 300, 1024, 128, seed=5)
    W = lib.W4Weights(c["q"], c["scale"], c["zero"])
    all_rows = lib.w4_linear(W, c["x"])
    for t in (0, 5, 11):
        assert torch.equal(lib.w4_linear(W, c["x"][t:t + 1])[0], all_rows[t])
    assert torch.equal(lib.w4_linear(W, c["x"]), all_rows)
    d = make(32, 96, 512, 128, BF16, True, 16, 4, seed=6)
    a, b = check(lib, d), check(lib, d)
    assert torch.equal(a, b)


def test_exact_integers(lib):
    """Unit scales and small integer x: every sum is an exact float32."""
    c = make(3, 64, 512, 128, F32, True, seed=7)
    c["scale"].fill_(1.0)
    c["x"] = torch.randint(-8, 9, (3, 512), device="cuda").to(BF16)
    got = lib.w4_linear(lib.W4Weights(c["q"], c["scale"], c["zero"]), c["x"])
    w, _ = dequantised(c)
    assert torch.equal(got.double(), c["x"].double() @ w[0].t())


def test_nan_stays_in_its_token(lib):
    c = make(6, 40, 256, 64, seed=8)
    W = lib.W4Weights(c["q"], c["scale"], c["zero"])
    clean = lib.w4_linear(W, c["x"])
    c["x"][2, 9] = float("nan")
    c["x"][4, 100] = float("inf")
    got = lib.w4_linear(W, c["x"])
    for t in (0, 1, 3, 5):
        assert torch.equal(got[t], clean[t])
    assert bool(torch.isnan(got[2]).all()) and not bool(torch.isfinite(got[4]).any())


def test_past_32_bit_offsets(lib):
    """More than 2^32 bytes of codes: the last rows of the last matrix."""
    E, N, K = 5, 262144, 8192
    q = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    scale = torch.ones((E, N, 1), dtype=BF16, device="cuda")
    scale = scale.expand(E, N, 1).contiguous()
    c = make(2, 64, K, K, BF16, False, seed=9)
    q[-1, -64:], scale[-1, -64:] = c["q"][0], c["scale"][0]
    W = lib.W4Weights(q, scale)
    ids = torch.tensor([[4], [4]], dtype=torch.int32, device="cuda")
    got = lib.w4_linear(W, c["x"], ids=ids)[:, 0]
    want, tol = reference(c, False)
    assert bool(((got[:, -64:].double() - want).abs() <= tol).all())
    # codes 0 stand for -8
    rest = -8 * c["x"].double().sum(1)
    near = (K / 32 + 32) * U * 8 * c["x"].double().abs().sum(1)
    assert bool(((got[:, :1000].double() - rest[:, None]).abs() <= near[:, None]).all())


def test_no_tokens(lib):
    c = make(4, 32, 64, 32)
    W = lib.W4Weights(c["q"], c["scale"], c["zero"])
    assert lib.w4_linear(W, c["x"][:0]).shape == (0, 32)


def test_captured_and_replayed(lib):
    c = make(8, 64, 256, 64, BF16, True, 8, 2, seed=10)
    W = lib.W4Weights(c["q"], c["scale"], c["zero"])
    y = torch.empty((8, 2, 32), device="cuda")

    def step():
        return lib.w4_linear(W, c["x"], ids=c["ids"], swiglu=True, y=y)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(4):
        d = make(8, 64, 256, 64, BF16, True, 8, 2, seed=60 + i)
        c["x"].copy_(d["x"])
        c["ids"].copy_(d["ids"])
        graph.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, step()), i


def test_a_layer_of_4_bit_experts(lib):
    """Router, gate and up products with SwiGLU, down products with the routing
    weights, and the library's combine, against float64.  h and the slots are
    rounded to BF16 in between: h by 2^-8 of its value, which the down product
    passes on, a slot by 2^-8 of its own."""
    T, E, k, H, I, G = 20, 16, 4, 256, 128, 64
    up = make(T, 2 * I, H, G, BF16, True, E, k, seed=11)
    down = make(T, H, I, G, BF16, True, E, k, seed=12)
    gen = torch.Generator(device="cuda").manual_seed(13)
    scores = torch.randn(T, E, generator=gen, device="cuda")
    ids, wts = lib.topk_route(scores, k)
    up["ids"] = ids
    h = check(lib, up, swiglu=True, y_dtype="bf16")
    down["ids"], down["weights"], down["x"] = ids, wts, h
    slots = check(lib, down, y_dtype="bf16")
    y = lib.combine(slots.view(T * k, H), T, k)
    w13, _ = dequantised(up)
    w2, _ = dequantised(down)
    for t in range(T):
        want, tol = torch.zeros(H, device="cuda").double(), torch.zeros(H, device="cuda").double()
        for j in range(k):
            e = int(ids[t, j])
            gu = w13[e] @ up["x"][t].double()
            a = gu[:I] * torch.sigmoid(gu[:I]) * gu[I:]
            s = float(wts[t, j]) * (w2[e] @ a)
            want += s
            tol += 2.0 ** -8 * (s.abs() + float(wts[t, j]) * (w2[e].abs() @ a.abs()))
        tol = 1.01 * tol + 1e-5
        assert bool(((y[t].double() - want).abs() <= tol).all())


def test_refusals(lib):
    c = make(4, 32, 64, 32)
    W = lib.W4Weights(c["q"], c["scale"], c["zero"])
    with pytest.raises(ValueError):
        lib.w4_linear(W, c["x"].float())
    with pytest.raises(ValueError):
        lib.w4_linear(W, c["x"][:, :32])
    with pytest.raises(ValueError):
        lib.W4Weights(c["q"], c["scale"][:, :5])
    with pytest.raises(ValueError):
        lib.W4Weights(c["q"], c["scale"].half())
    many = make(4, 32, 64, 32, E=3, k=1)
    with pytest.raises(ValueError):
        lib.w4_linear(lib.W4Weights(many["q"], many["scale"]), many["x"])
    odd = make(4, 31, 64, 32)
    with pytest.raises(lib.MoeError):
        lib.w4_linear(lib.W4Weights(odd["q"], odd["scale"]), odd["x"], swiglu=True)
    big = make(4, 32, 96, 96)
    with pytest.raises(lib.MoeError):   # groups of a power of two
        lib.w4_linear(lib.W4Weights(big["q"], big["scale"]), big["x"])


@pytest.mark.parametrize("T,bad", [(5, 2), (16, 15), (37, 20)])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_bad_row_of_x_stays_its_own(lib, T, bad, value):
    c = make(T, 40, 448, 64, zero=True)
    W = lib.W4Weights(c["q"], c["scale"], c["zero"])
    clean = lib.w4_linear(W, c["x"])
    c["x"][bad, 100] = value
    got = lib.w4_linear(W, c["x"])
    keep = torch.arange(T, device="cuda") != bad
    assert torch.equal(got[keep], clean[keep])
    assert not bool(got[bad].isfinite().any())
