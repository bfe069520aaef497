"""The operators around the layer in one run, as a model's block uses them: the
norm before the block, the gating scores from a 4-bit matrix, the router, its
load statistics, the experts, and the join with the residual stream and the
next norm; then the gradients back through the join and the router.  Each
step is held to its formula in float64 on the inputs that it really got, so a
tolerance is that of one operator."""

import numpy as np
import pytest
import torch

import workloads as W
from oracle import layer as L
from oracle import router as R
from _helpers import assert_layer_close, device_weights, oracle_kw, to_f64

pytestmark = pytest.mark.gpu

CFG = W.QWEN3_DECODE_MXFP8.replace(num_experts=16, top_k=4, hidden=512, inter=256, tag=61)
U, BF16_STEP, EPS = 2.0 ** -24, 2.0 ** -8, 1e-6


class Block:
    def __init__(self, lib, t, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        h, e = CFG.hidden, CFG.num_experts

        def normal(*shape):
            return torch.randn(*shape, generator=g, device="cuda")

        self.lib, self.t = lib, t
        self.x = normal(t, h).to(torch.bfloat16)
        self.w_pre, self.w_post, self.w_next = ((1 + 0.1 * normal(h)).to(torch.bfloat16) for _ in range(3))
        self.gate = (0.5 + 0.1 * normal(h)).to(torch.bfloat16)
        q = torch.randint(0, 256, (e, h // 2), generator=g, device="cuda", dtype=torch.uint8)
        scale = (0.05 + 0.05 * torch.rand(e, h // 64, generator=g, device="cuda")) / 4
        self.router = lib.W4Weights(q, scale)
        self.experts = device_weights(CFG)

    def run(self, stream=None):
        lib = self.lib
        r = {}
        _, r["n"] = lib.block_norm(self.x, w_next=self.w_pre, eps=EPS, stream=stream)
        r["scores"] = lib.w4_linear(self.router, r["n"], stream=stream)
        r["ids"], r["wts"] = lib.topk_route(r["scores"], CFG.top_k, stream=stream)
        r["loss"], r["counts"], r["tokens"] = lib.balance_loss(r["scores"], r["ids"], stream=stream)
        r["y"], _ = lib.layer(self.experts, r["n"], r["ids"], r["wts"], path="decode", stream=stream)
        r["out"], r["next"] = lib.block_norm(self.x, r["y"], w_post=self.w_post, w_next=self.w_next,
                                             gate=self.gate, eps=EPS, stream=stream)
        return r


def rms(v):
    return (v.square().mean(1, keepdim=True) + EPS).sqrt()


def near(got, want, roundings, size, step=0.0):
    err = (got.double() - want).abs()
    tol = roundings * U * size + step * want.abs() + 1e-37
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.parametrize("t", [1, 7, 24])
def test_forward_step_by_step(lib, t):
    b = Block(lib, t, t)
    r = b.run()
    x = b.x.double()
    n = x / rms(x) * b.w_pre.double()
    near(r["n"], n, 64, n.abs(), BF16_STEP)
    q, s, _ = b.router.tensors
    v = torch.empty(CFG.num_experts, CFG.hidden, dtype=torch.float64, device="cuda")
    v[:, 0::2], v[:, 1::2] = (q & 15).double() - 8, (q >> 4).double() - 8
    m = v * s.double().repeat_interleave(64, 1)
    size = ((v.abs() + 16) * s.double().repeat_interleave(64, 1)) @ r["n"].double().abs().t()
    near(r["scores"], r["n"].double() @ m.t(), CFG.hidden / 32 + 32, size.t())
    scores = r["scores"].cpu().numpy()
    ids, wts = R.topk_route(scores, CFG.top_k)
    assert np.array_equal(r["ids"].cpu().numpy(), ids)
    assert np.allclose(r["wts"].cpu().numpy(), wts, rtol=2e-6, atol=1e-8)
    assert np.array_equal(r["counts"][0].cpu().numpy(), np.bincount(ids.reshape(-1), minlength=CFG.num_experts))
    p = torch.softmax(r["scores"].double(), 1)
    f = r["counts"][0].double() * CFG.num_experts / (CFG.top_k * t)
    near(r["loss"][0, 0], (f * p.mean(0)).sum(), 192, (f * p.mean(0)).sum())
    ref = L.moe_layer(to_f64(r["n"]), ids, r["wts"].cpu().numpy(), act_quant="none", **oracle_kw(CFG))
    assert_layer_close(to_f64(r["y"]), ref, t)
    y = r["y"].double()
    join = y / rms(y) * b.w_post.double() * b.gate.double()
    out = x + join
    mag = x.abs() + join.abs()
    near(r["out"], out, 64, mag, BF16_STEP)
    spread = mag.norm(dim=1, keepdim=True) / out.norm(dim=1, keepdim=True)
    nxt = out / rms(out) * b.w_next.double()
    near(r["next"], nxt, 64, nxt.abs() * (1 + spread) + mag / rms(out) * b.w_next.double().abs(), BF16_STEP)


def test_backward_reaches_every_parameter(lib):
    """The join's gradients and, through the routing weights and the balance
    loss, the scores': one directional difference of the float64 formulas."""
    t = 20
    b = Block(lib, t, 5)
    r = b.run()
    g = torch.Generator(device="cuda").manual_seed(9)
    go, gn = (torch.randn(t, CFG.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    d = lib.block_norm_backward(go, gn, r["out"], r["y"], w_post=b.w_post, w_next=b.w_next, gate=b.gate, eps=EPS)
    assert all(bool(torch.isfinite(d[k]).all()) and bool(d[k].any()) for k in d)
    dw = torch.randn(t, CFG.top_k, generator=g, device="cuda")
    gl = torch.tensor([[0.3, 0.01]], device="cuda")
    ds = lib.router_backward(r["scores"], r["ids"], grad_loss=gl, counts=r["counts"], tokens=r["tokens"],
                             weights=r["wts"], grad_weights=dw)

    def value(s):
        f = r["counts"][0].double() * CFG.num_experts / (CFG.top_k * t)
        w = torch.softmax(torch.gather(s, 1, r["ids"].long()), 1)
        return float((w * dw.double()).sum() + 0.3 * (f * torch.softmax(s, 1).mean(0)).sum()
                     + 0.01 * torch.logsumexp(s, 1).square().mean())

    v = torch.randn(t, CFG.num_experts, generator=g, device="cuda", dtype=torch.float64)
    s = r["scores"].double()
    want = (value(s + 1e-4 * v) - value(s - 1e-4 * v)) / 2e-4
    have = float((ds.double() * v).sum())
    assert abs(have - want) <= 2e-6 * float((ds.double() * v).abs().sum()) + 1e-6


def test_captured_on_its_own_stream_and_replayed(lib):
    b = Block(lib, 12, 3)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.run(stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = b.run()
    for i in range(4):
        b.x.copy_(Block(lib, 12, 10 + i).x)
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in held.items()}
        want = b.run()
        torch.cuda.synchronize()
        assert all(torch.equal(got[k], want[k]) for k in want), i
