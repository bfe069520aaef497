"""moe_block_norm and its backward pass against the formulas in float64.

Tolerances.  u = 2^-24 is half a step of float32.  A value computed in float32
from terms of magnitudes m_1, m_2, ... through at most c roundings on any way
from an input to it is off by at most about c u (m_1 + m_2 + ...), where a sum
over a row of H <= 16384 counts 16 (serial in a thread) + 6 (wavefront) + 16
(wavefronts) roundings, halved by the square root.  C_ROW = 64 covers the
longest way of the forward pass (two norms), 2 C_ROW that of the backward pass
(a sum of products of a normalised row).  A result stored in a type with step
eps is off by eps / 2 of its value more.  Sums over the T tokens add the
roundings of their additions: the tokens of one workgroup, then the
workgroups."""

import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
C_ROW = 64
EPS = 1e-6
BF16, F32 = torch.bfloat16, torch.float32


def make(T, H, x=BF16, y=BF16, gate="none", post=True, nxt=True, seed=0, x_pad=0, y_pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    c = {"x": normal(T, H + x_pad).to(x)[:, :H], "y": None, "w_post": None, "w_next": None, "gate": None}
    if y is not None:
        c["y"] = (0.3 * normal(T, H + y_pad)).to(y)[:, :H]
        c["w_post"] = (1 + 0.2 * normal(H)).to(x) if post else None
        if gate == "channel":
            c["gate"] = normal(H).to(x)
        elif gate == "token":
            c["gate"] = normal(T, 1)
        elif gate == "full":
            c["gate"] = normal(T, H).to(x)
    c["w_next"] = (1 + 0.2 * normal(H)).to(x) if nxt else None
    c["grad_out"], c["grad_n"] = normal(T, H).to(x), normal(T, H).to(x) if nxt else None
    return c


def args(c):
    return {k: c[k] for k in ("w_post", "w_next", "gate")}


def f64(t):
    return None if t is None else t.double()


def reference(c, a, eps=EPS):
    """out, n and the magnitudes their errors are measured by."""
    x, y, wp, wn, gate = (f64(c[k]) for k in ("x", "y", "w_post", "w_next", "gate"))
    out, mag = x, x.abs()
    if y is not None:
        b = y if wp is None else y / (y.square().mean(1, keepdim=True) + eps).sqrt() * wp
        b = b if gate is None else b * gate
        out, mag = a * x + b, (a * x).abs() + b.abs()
    if wn is None:
        return out, mag, None, None
    r = (out.square().mean(1, keepdim=True) + eps).rsqrt()
    n = out * r * wn
    spread = mag.norm(dim=1, keepdim=True) / out.norm(dim=1, keepdim=True).clamp(min=1e-30)
    return out, mag, n, n.abs() * (1 + spread) + mag * r * wn.abs()


def close(got, want, mag, roundings, what):
    step = torch.finfo(got.dtype).eps / 2 if got.dtype != F32 else 0.0
    err = (got.double() - want).abs()
    tol = roundings * U * mag + step * want.abs() + torch.finfo(got.dtype).tiny
    bad = err > tol
    assert not bool(bad.any()) and bool(torch.isfinite(got).all()), (
        what, float((err / tol).max()), int(bad.sum()))


def check_forward(lib, c, a=0.875, **kw):
    out, n = lib.block_norm(c["x"], c["y"], res_scale=a, eps=EPS, **args(c), **kw)
    ro, mo, rn, mn = reference(c, a)
    assert (out is None) == (c["y"] is None) and (n is None) == (rn is None)
    if out is not None:
        close(out, ro, mo, C_ROW, "out")
    if n is not None:
        close(n, rn, mn, C_ROW, "n")
    return out, n


def gradients(c, a, eps=EPS):
    """The backward formulas in float64, with x the stored out; and magnitudes."""
    o, y, wp, wn, gate, go, gn = (f64(c[k]) for k in ("x", "y", "w_post", "w_next", "gate", "grad_out",
                                                       "grad_n"))
    H = c["x"].shape[1]
    got, mag = {}, {}
    d = torch.zeros_like(o) if go is None else go
    md = d.abs()
    if wn is not None:
        r = (o.square().mean(1, keepdim=True) + eps).rsqrt()
        q = wn * gn
        d = d + r * q - o * r ** 3 / H * (q * o).sum(1, keepdim=True)
        md = md + r * q.abs() + o.abs() * r ** 3 / H * (q * o).abs().sum(1, keepdim=True)
        got["w_next"], mag["w_next"] = (gn * o * r).sum(0), (gn * o * r).abs().sum(0)
    s = a if y is not None else 1.0
    got["x"], mag["x"] = s * d, abs(s) * md
    if y is None:
        return got, mag
    r = 1.0 if wp is None else (y.square().mean(1, keepdim=True) + eps).rsqrt()
    b = y * r * (1.0 if wp is None else wp)
    g = torch.ones_like(d) if gate is None else gate.expand_as(d)
    q, mq = d * g, md * g.abs()
    if gate is not None:
        dg, mg = d * b, md * b.abs()
        dims = 0 if gate.dim() == 1 else 1 if gate.shape[1] == 1 and H > 1 else None
        if dims is None:
            got["gate"], mag["gate"] = dg, mg
        else:
            got["gate"], mag["gate"] = dg.sum(dims, keepdim=dims == 1), mg.sum(dims, keepdim=dims == 1)
    if wp is None:
        got["y"], mag["y"] = q, mq
    else:
        got["w_post"], mag["w_post"] = (q * y * r).sum(0), (mq * (y * r).abs()).sum(0)
        p, mp = q * wp, mq * wp.abs()
        got["y"] = r * p - y * r ** 3 / H * (p * y).sum(1, keepdim=True)
        mag["y"] = r * mp + y.abs() * r ** 3 / H * (mp * y.abs()).sum(1, keepdim=True)
    return got, mag


def check_backward(lib, c, a=0.875, **kw):
    got = lib.block_norm_backward(c["grad_out"], c["grad_n"], c["x"], c["y"], res_scale=a, eps=EPS,
                                  **args(c), **kw)
    want, mag = gradients(c, a)
    T = c["x"].shape[0]
    for k in ("x", "y", "gate", "w_post", "w_next"):
        assert (got[k] is None) == (k not in want), k
        if got[k] is None:
            continue
        # column sums: at most T additions in a workgroup, 64 + 16 over the workgroups
        over_tokens = k in ("w_post", "w_next") or (k == "gate" and c["gate"].dim() == 1)
        close(got[k], want[k], mag[k], 2 * C_ROW + (min(T, 1000) + 80 if over_tokens else 0), k)
    return got


SIZES = [(1, 1), (3, 7), (5, 8), (2, 64), (9, 511), (4, 512), (5, 520), (3, 1001), (1, 2048), (7, 2056),
         (2, 4096), (3, 4104), (2, 8192), (3, 8200), (2, 16384), (2, 16383)]
KINDS = [(BF16, BF16, "none", True, True), (BF16, F32, "channel", True, True),
         (F32, F32, "token", True, True), (BF16, BF16, "full", True, True),
         (BF16, F32, "token", False, True), (F32, F32, "full", False, False),
         (BF16, BF16, "channel", True, False), (BF16, None, "none", False, True),
         (F32, None, "none", False, True)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_forward(lib, T, H, kind):
    x, y, gate, post, nxt = KINDS[kind]
    check_forward(lib, make(T, H, x, y, gate, post, nxt, seed=T * 100 + kind))


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_backward(lib, T, H, kind):
    x, y, gate, post, nxt = KINDS[kind]
    check_backward(lib, make(T, H, x, y, gate, post, nxt, seed=T * 100 + kind))


@pytest.mark.parametrize("T,H", [(1000, 768), (3001, 264), (2500, 33), (700, 5000)])
def test_many_rows(lib, T, H):
    c = make(T, H, BF16, F32, "channel", seed=T)
    check_forward(lib, c)
    check_backward(lib, c)


@pytest.mark.parametrize("x_pad,y_pad", [(8, 16), (3, 0), (0, 5)])
def test_row_strides(lib, x_pad, y_pad):
    c = make(6, 520, BF16, BF16, "full", seed=4, x_pad=x_pad, y_pad=y_pad)
    assert (c["x"].stride(0), c["y"].stride(0)) == (520 + x_pad, 520 + y_pad)
    check_forward(lib, c)
    check_backward(lib, c)


def test_unaligned_start(lib):
    c = make(3, 640, seed=5)
    base = torch.empty(3 * 640 + 1, dtype=BF16, device="cuda")
    base[1:] = c["y"].reshape(-1)
    c["y"] = base[1:].view(3, 640)
    check_forward(lib, c)
    check_backward(lib, c)


def test_same_bits_for_any_batch(lib):
    """A row's results do not depend on the rows beside it, nor on its stride."""
    c = make(33, 2048, BF16, BF16, "channel", seed=6)
    out, n = check_forward(lib, c)
    for t in (0, 17, 32):
        o1, n1 = lib.block_norm(c["x"][t:t + 1], c["y"][t:t + 1], res_scale=0.875, eps=EPS, **args(c))
        assert torch.equal(o1[0], out[t]) and torch.equal(n1[0], n[t])
    a = check_backward(lib, c)
    b = check_backward(lib, c)
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("H", [512, 4096, 1001])
def test_in_place(lib, H):
    c = make(21, H, seed=7)
    out, n = check_forward(lib, c)
    x = c["x"].clone()
    got, n2 = lib.block_norm(x, c["y"], res_scale=0.875, eps=EPS, out=x, **args(c))
    assert got is x and torch.equal(x, out) and torch.equal(n2, n)


def test_zero_rows_and_large_values(lib):
    c = make(5, 768, BF16, BF16, "none", seed=8)
    c["y"][1] = 0
    c["x"][2] = 0
    c["y"][2] = 0
    c["y"][3] = (c["y"][3].float() * 1e15).to(BF16)
    c["x"][4] = (c["x"][4].float() * 1e-15).to(BF16)
    check_forward(lib, c)
    out, n = lib.block_norm(c["x"], c["y"], res_scale=0.875, eps=EPS, **args(c))
    assert not out[2].any() and not n[2].any()


def test_nan_and_inf_stay_in_their_row(lib):
    c = make(4, 1024, seed=9)
    c["x"][1, 5] = float("nan")
    c["y"][2, 7] = float("inf")
    out, n = lib.block_norm(c["x"], c["y"], res_scale=0.875, eps=EPS, **args(c))
    ok = make(4, 1024, seed=9)
    ref, refn = lib.block_norm(ok["x"], ok["y"], res_scale=0.875, eps=EPS, **args(ok))
    for t in (0, 3):
        assert torch.equal(out[t], ref[t]) and torch.equal(n[t], refn[t])
    assert bool(torch.isnan(out[1, 5])) and bool(torch.isnan(n[1]).all())
    assert bool(torch.isnan(out[2, 7])) and bool(torch.isnan(n[2]).all())


def test_missing_gradients_count_as_zero(lib):
    c = make(9, 520, BF16, BF16, "channel", seed=10)
    full = lib.block_norm_backward(c["grad_out"], torch.zeros_like(c["grad_n"]), c["x"], c["y"], **args(c))
    part = lib.block_norm_backward(c["grad_out"], None, c["x"], c["y"], **args(c))
    assert all(torch.equal(full[k], part[k]) for k in full)
    c["grad_out"] = None
    check_backward(lib, c)


@pytest.mark.parametrize("gate", ["channel", "token", "full"])
def test_gradient_against_differences(lib, gate):
    """<gradient, v> of the library against a central difference of the float64
    forward formula along v, for each input; the difference itself is exact to
    about h^2 = 1e-8 and 2^-52 / h = 2e-12 of the sum's magnitude."""
    c = make(6, 136, F32, F32, gate, seed=11)
    a, h = 0.875, 1e-4
    out = reference(c, a)[0]
    got = lib.block_norm_backward(c["grad_out"], c["grad_n"], out.float(), c["y"], res_scale=a, eps=EPS,
                                  **args(c))
    go, gn = c["grad_out"].double(), c["grad_n"].double()

    def loss(p):
        o, _, n, _ = reference(p, a)
        return float((o * go).sum() + (n * gn).sum())

    gen = torch.Generator(device="cuda").manual_seed(3)
    for k in ("x", "y", "gate", "w_post", "w_next"):
        v = torch.randn(c[k].shape, generator=gen, device="cuda", dtype=torch.float64)
        ends = [loss({**{q: f64(t) for q, t in c.items()}, k: c[k].double() + s * h * v}) for s in (1, -1)]
        want = (ends[0] - ends[1]) / (2 * h)
        have = float((got[k].double() * v).sum())
        size = float((got[k].double() * v).abs().sum())
        assert abs(have - want) <= 2e-6 * size + 1e-6, (k, have, want)


def test_no_tokens(lib):
    c = make(0, 256, BF16, BF16, "channel", seed=12)
    out, n = lib.block_norm(c["x"], c["y"], **args(c))
    assert out.shape == n.shape == (0, 256)
    g = lib.block_norm_backward(c["grad_out"], c["grad_n"], c["x"], c["y"], **args(c))
    for k in ("gate", "w_post", "w_next"):
        assert g[k].shape == (256,) and not g[k].any()


def test_past_32_bit_offsets(lib):
    """More than 2^31 elements: the first and last rows against the formula."""
    T, H = 262144 + 3, 8192
    x = torch.zeros((T, H), dtype=BF16, device="cuda")
    c = make(6, H, seed=13, y=None)
    w = c["w_next"]
    x[:3], x[-3:] = c["x"][:3], c["x"][3:]
    n = torch.full((T, H), 7.0, dtype=BF16, device="cuda")
    lib.block_norm(x, w_next=w, n=n)
    _, _, rn, mn = reference(c, 1.0)
    close(torch.cat((n[:3], n[-3:])), rn, mn, C_ROW, "n")
    assert not n[T // 2].any()
    del n
    g = lib.block_norm_backward(None, x, x, w_next=w)
    c["grad_out"], c["grad_n"] = None, c["x"]
    want, mag = gradients(c, 1.0)
    close(torch.cat((g["x"][:3], g["x"][-3:])), want["x"], mag["x"], 2 * C_ROW, "x")
    close(g["w_next"], want["w_next"], mag["w_next"], 2 * C_ROW + 2000, "w_next")


def test_captured_and_replayed(lib):
    c = make(40, 1024, BF16, BF16, "channel", seed=14)
    out, n = (torch.empty_like(c["x"]) for _ in range(2))

    def step():
        lib.block_norm(c["x"], c["y"], out=out, n=n, **args(c))
        return lib.block_norm_backward(c["grad_out"], c["grad_n"], out, c["y"], **args(c))

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        c["x"].copy_(make(40, 1024, seed=20 + i)["x"])
        c["y"].copy_(make(40, 1024, seed=30 + i)["y"])
        graph.replay()
        torch.cuda.synchronize()
        got = {**{k: v.clone() for k, v in held.items()}, "out": out.clone(), "n": n.clone()}
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(got["out"], out) and torch.equal(got["n"], n)
        assert all(torch.equal(got[k], want[k]) for k in want), i


def test_on_another_stream(lib):
    c = make(64, 2048, seed=15)
    out, n = check_forward(lib, c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o2, n2 = lib.block_norm(c["x"], c["y"], res_scale=0.875, eps=EPS, stream=s, **args(c))
    s.synchronize()
    assert torch.equal(o2, out) and torch.equal(n2, n)


def test_refusals(lib):
    c = make(4, 64, seed=16)
    with pytest.raises(ValueError):   # another shape
        lib.block_norm(c["x"], c["y"][:3], **args(c))
    with pytest.raises(ValueError):   # weights of another dtype
        lib.block_norm(c["x"], c["y"], w_next=c["w_next"].float())
    with pytest.raises(ValueError):   # columns that are not consecutive
        lib.block_norm(c["x"].t(), w_next=c["w_next"][:4])
    with pytest.raises(ValueError):   # out without y
        lib.block_norm(c["x"], w_next=c["w_next"], out=torch.empty_like(c["x"]))
    with pytest.raises(ValueError):   # half precision is not one of the library's types
        lib.block_norm(c["x"].half(), w_next=c["w_next"])
    with pytest.raises(lib.MoeError):  # nothing to compute
        lib.block_norm(c["x"])
    with pytest.raises(lib.MoeError):  # FP32 stream with a BF16 block
        lib.block_norm(c["x"].float(), c["y"], w_next=c["w_next"].float())


@pytest.mark.parametrize("H", [4104, 5120, 8192, 8191])
@pytest.mark.parametrize("kind", range(len(KINDS)))
def test_forward_more_rows_than_cus(lib, H, kind):
    """Rows of this length take another launch shape in a batch of this size."""
    x, y, gate, post, nxt = KINDS[kind]
    check_forward(lib, make(300, H, x, y, gate, post, nxt, seed=H + kind))
