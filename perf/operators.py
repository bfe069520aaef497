"""Cases of the operators that stand around the routed experts of a layer.

block_norm / block_norm_backward   norms before and after a block, fused with
                                   its gate and residual scale
balance_loss / router_backward     per-expert counts, balance and z loss of the
                                   router, and the router's gradient
w4_linear                          products with 4-bit weights and group
                                   scales: one dense matrix, or the experts'

`own` chooses between the operators written out in elementary torch operations
and the library's calls.  `exact` is the definition in 64 bits.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    """The listed cases.  Hidden sizes, expert counts and top-k are those of
    this repository's workloads where a model shape is meant."""
    return [
        # one token of a decode step between two blocks: latency alone
        _norm("norm_one_token", 1, 2048, "bf16", "f32", "none", True, True),
        # prompt of 16384 tokens, learned gate for each channel: HBM
        _norm("norm_prompt", 16384, 4096, "bf16", "bf16", "channel", True, True),
        # a ragged batch of a small odd model in FP32, gate for each token
        _norm("norm_ragged_f32", 777, 1001, "f32", "f32", "token", True, True),
        # training step of the prompt's shape: every gradient
        _norm("norm_back_prompt", 16384, 4096, "bf16", "bf16", "channel", True, True, back=True),
        # a short ragged training batch of a wide model, gate of its own for each value
        _norm("norm_back_ragged", 515, 7168, "bf16", "f32", "full", True, True, back=True),
        # load statistics of one decode batch: latency
        _balance("balance_decode", 32, 128, 8, 1, False),
        # packed training batch: ragged sequences, padding tokens masked
        _balance("balance_packed", 65536, 256, 8, 24, True),
        # router gradient of a small batch
        _balance("router_back_small", 333, 128, 8, 3, False, back=True),
        # router gradient of the packed training batch, through the routing weights too
        _balance("router_back_packed", 65536, 256, 8, 24, True, back=True),
        # one token through a dense projection
        _w4("w4_one_token", 1, 4096, 2048, 128, "bf16", False),
        # an output head: odd number of rows, few tokens
        _w4("w4_head", 5, 40961, 7168, 64, "f32", True, y="f32"),
        # gate and up products of a decode batch with 4-bit experts
        _w4("w4_experts_gate_up", 32, 1536, 2048, 128, "bf16", True, E=128, k=8, swiglu=True),
    ]


def _norm(name, T, H, x, y, gate, post, nxt, back=False):
    return {"name": name, "op": "norm_back" if back else "norm", "T": T, "H": H, "x": x, "y": y,
            "gate": gate, "post": post, "next": nxt}


def _balance(name, T, E, k, S, mask, back=False):
    return {"name": name, "op": "router_back" if back else "balance", "T": T, "E": E, "k": k,
            "S": S, "mask": mask}


def _w4(name, T, N, K, group, scale, zero, E=1, k=0, swiglu=False, slots=False, y="bf16"):
    return {"name": name, "op": "w4", "T": T, "N": N, "K": K, "group": group, "scale": scale,
            "zero": zero, "E": E, "k": k, "swiglu": swiglu, "slots": slots, "y": y}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "norm_back", "balance", "router_back", "w4", "w4_experts"))
    if op in ("norm", "norm_back"):
        H = _log_int(rng, 64, 8192)
        T = _log_int(rng, 1, min(16384, 16384 * 4096 // H))
        x = rng.choice(("bf16", "bf16", "f32"))
        y = "f32" if x == "f32" else rng.choice(("bf16", "f32"))
        if x == "f32" or y == "f32":
            T = max(1, T // 3)
        c = _norm("", T, H, x, y, rng.choice(("none", "channel", "token", "full")),
                  rng.random() < 0.8, True, back=op == "norm_back")
    elif op in ("balance", "router_back"):
        E = _log_int(rng, 4, 512)
        T = _log_int(rng, 1, min(65536, 65536 * 256 // E))
        c = _balance("", T, E, rng.randint(1, min(8, E)), _log_int(rng, 1, 24), rng.random() < 0.5,
                     back=op == "router_back")
    elif op == "w4":
        group = rng.choice((32, 64, 128))
        K = group * _log_int(rng, 1, 7168 // group)
        N = _log_int(rng, 16, min(40961, 40961 * 7168 // K))
        c = _w4("", _log_int(rng, 1, 64), N, K, group, rng.choice(("bf16", "f32")),
                rng.random() < 0.5, y=rng.choice(("bf16", "f32")))
    else:
        group = rng.choice((32, 64, 128))
        K = group * _log_int(rng, 2, 4096 // group)
        E, k = rng.choice(((8, 2), (64, 4), (128, 8)))
        T = _log_int(rng, 1, 32)
        N = 2 * _log_int(rng, 32, max(32, min(1024, 1536 * 2048 // (2 * K))))
        swiglu = rng.random() < 0.5
        c = _w4("", T, N, K, group, rng.choice(("bf16", "f32")), rng.random() < 0.5, E=E, k=k,
                swiglu=swiglu, slots=not swiglu, y=rng.choice(("bf16", "f32")))
    del c["name"]
    return c


def work(c):
    size = {"bf16": 2, "f32": 4}
    if c["op"] in ("norm", "norm_back"):
        n, x, y = c["T"] * c["H"], size[c["x"]], size[c["y"]]
        full = n * x if c["gate"] == "full" else 0
        small = 4 * c["T"] if c["gate"] == "token" else 0
        vec = c["H"] * x * (int(c["post"]) + int(c["next"]) + int(c["gate"] == "channel"))
        if c["op"] == "norm":   # x, y -> out, n
            return {"bytes": n * (2 * x + y) + full + small + vec + (n * x if c["next"] else 0),
                    "flops": 12 * n}
        # grad_out, grad_n, out, y -> dx, dy, and the gate's and weights' gradients
        vec += 4 * c["H"] * (int(c["post"]) + int(c["next"]) + int(c["gate"] == "channel"))
        return {"bytes": n * (2 * x + 2 * y) + (2 * n * x if c["next"] else 0) + 2 * full + 2 * small + vec,
                "flops": 30 * n}
    if c["op"] in ("balance", "router_back"):
        rows, ids = 4 * c["T"] * c["E"], 4 * c["T"] * c["k"]
        mask, seqs = c["T"] if c["mask"] else 0, 4 * c["S"] * (c["E"] + 4)
        if c["op"] == "balance":
            return {"bytes": rows + ids + mask + seqs, "flops": 6 * c["T"] * c["E"]}
        return {"bytes": 2 * rows + 3 * ids + mask + seqs, "flops": 10 * c["T"] * c["E"]}
    groups = c["K"] // c["group"]
    matrix = c["N"] * (c["K"] // 2 + groups * (size[c["scale"]] + int(c["zero"])))
    entries = c["T"] * max(1, c["k"])
    mats = c["E"] * (1 - (1 - c["k"] / c["E"]) ** c["T"]) if c["k"] else 1
    x = 2 * c["K"] * (entries if c["slots"] else c["T"])
    y = entries * (c["N"] // 2 if c["swiglu"] else c["N"]) * size[c["y"]]
    return {"bytes": int(mats * matrix) + x + y, "flops": 2 * entries * c["N"] * c["K"]}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    s = {"case": c}
    if c["op"] in ("norm", "norm_back"):
        T, H, xd, yd = c["T"], c["H"], DTYPES[c["x"]], DTYPES[c["y"]]
        # a residual stream with a few large channels, a block's output below it
        loud = 1 + 8 * (uniform(H) < 0.01).float()
        s["x"] = (normal(T, H) * loud).to(xd)
        s["y"] = (0.3 * normal(T, H)).to(yd)
        s["w_post"] = (1 + 0.1 * normal(H)).to(xd) if c["post"] else None
        s["w_next"] = (1 + 0.1 * normal(H)).to(xd) if c["next"] else None
        s["gate"] = None
        if c["gate"] == "channel":
            s["gate"] = (0.5 + 0.2 * normal(H)).to(xd)
        elif c["gate"] == "token":
            s["gate"] = uniform(T, 1)
        elif c["gate"] == "full":
            s["gate"] = uniform(T, H).to(xd)
        s["scale"] = 0.875
        if c["op"] == "norm_back":
            s["grad_out"] = normal(T, H).to(xd)
            s["grad_n"] = normal(T, H).to(xd) if c["next"] else None
        return s
    if c["op"] in ("balance", "router_back"):
        T, E, k, S = c["T"], c["E"], c["k"], c["S"]
        scores = 1.5 * normal(T, E)
        s["ids"] = torch.topk(scores + 0.5 * normal(E), k, dim=1).indices.to(torch.int32)
        s["weights"] = torch.softmax(torch.gather(scores, 1, s["ids"].long()), 1)
        s["mask"] = None
        if c["mask"]:
            # padding tokens: what stands in their rows is of no account
            s["mask"] = uniform(T) < 0.9
            scores = torch.where(s["mask"][:, None], scores, float("nan"))
        s["scores"] = scores
        # ragged sequences, some of them empty; a tail behind the last one
        s["offsets"] = None
        if S > 1:
            cuts = torch.sort((uniform(S + 1) * (T + 1)).to(torch.int32)).values
            cuts[0] = 0
            s["offsets"] = cuts
        if c["op"] == "router_back":
            s["grad_weights"] = normal(T, k)
            s["grad_loss"] = torch.stack((0.01 + 0.01 * uniform(S), 0.001 + 0.001 * uniform(S)), 1)
            s["counts"], s["tokens"] = _plain_counts(s)
        return s
    N, K, E, T, k = c["N"], c["K"], c["E"], c["T"], c["k"]
    groups = K // c["group"]
    s["q"] = torch.randint(0, 256, (E, N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    s["scale"] = ((0.5 + uniform(E, N, groups)) / (4.6 * math.sqrt(K))).to(DTYPES[c["scale"]])
    s["zero"] = None
    if c["zero"]:
        s["zero"] = torch.randint(4, 12, (E, N, groups), generator=g, device="cuda", dtype=torch.uint8)
    s["ids"] = s["weights"] = None
    if k:
        logits = normal(T, E)
        s["ids"] = torch.topk(logits, k, dim=1).indices.to(torch.int32)
        if c["slots"]:   # the products that are joined by the routing weights
            s["weights"] = torch.softmax(torch.gather(logits, 1, s["ids"].long()), 1)
    s["x"] = normal(*((T, k, K) if c["slots"] else (T, K))).to(torch.bfloat16)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if own:
        return _own(op, s)
    return {"norm": _plain_norm, "norm_back": _plain_norm_back, "balance": _plain_balance,
            "router_back": _plain_router_back, "w4": _plain_w4}[op](s)


def _own(op, s):
    import mixture_experts_decode_amd as moe
    c = s["case"]
    if op == "norm":
        out, n = moe.block_norm(s["x"], s["y"], w_post=s["w_post"], w_next=s["w_next"],
                                gate=s["gate"], res_scale=s["scale"], eps=EPS)
        return {"out": out, "n": n}
    if op == "norm_back":
        return moe.block_norm_backward(s["grad_out"], s["grad_n"], s["x"], s["y"],
                                       w_post=s["w_post"], w_next=s["w_next"], gate=s["gate"],
                                       res_scale=s["scale"], eps=EPS)
    if op == "balance":
        loss, counts, tokens = moe.balance_loss(s["scores"], s["ids"], mask=s["mask"],
                                                seq_offsets=s["offsets"])
        return {"loss": loss, "counts": counts, "tokens": tokens}
    if op == "router_back":
        return moe.router_backward(s["scores"], s["ids"], grad_loss=s["grad_loss"],
                                   counts=s["counts"], tokens=s["tokens"], mask=s["mask"],
                                   seq_offsets=s["offsets"], weights=s["weights"],
                                   grad_weights=s["grad_weights"])
    W = moe.W4Weights(s["q"], s["scale"], s["zero"])
    return moe.w4_linear(W, s["x"], ids=s["ids"], weights=s["weights"], swiglu=c["swiglu"],
                         y_dtype=c["y"])


def _inv_rms(v):
    return torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)


def _plain_norm(s):
    x, y = s["x"].float(), s["y"].float()
    if s["w_post"] is not None:
        y = y * _inv_rms(y) * s["w_post"].float()
    if s["gate"] is not None:
        y = y * s["gate"].float()
    out = s["scale"] * x + y
    n = None
    if s["w_next"] is not None:
        n = (out * _inv_rms(out) * s["w_next"].float()).to(s["x"].dtype)
    return {"out": out.to(s["x"].dtype), "n": n}


def _plain_norm_back(s):
    """s["x"] stands for the joined stream that the forward pass stored."""
    out, y, d = s["x"].float(), s["y"].float(), s["grad_out"].float()
    H = out.shape[1]
    grads = {"w_post": None, "w_next": None, "gate": None}
    if s["w_next"] is not None:
        r, dn = _inv_rms(out), s["grad_n"].float()
        grads["w_next"] = (dn * out * r).sum(0)
        q = dn * s["w_next"].float()
        d = d + r * q - out * (r * r * r * (q * out).sum(-1, keepdim=True) / H)
    b, r = y, None
    if s["w_post"] is not None:
        r = _inv_rms(y)
        b = y * r * s["w_post"].float()
    q = d
    if s["gate"] is not None:
        q = d * s["gate"].float()
        dg = d * b
        if s["gate"].dim() == 1:
            grads["gate"] = dg.sum(0)
        elif s["gate"].shape[1] == 1 and H > 1:
            grads["gate"] = dg.sum(-1, keepdim=True)
        else:
            grads["gate"] = dg.to(s["gate"].dtype)
    if s["w_post"] is not None:
        grads["w_post"] = (q * y * r).sum(0)
        q = q * s["w_post"].float()
        q = r * q - y * (r * r * r * (q * y).sum(-1, keepdim=True) / H)
    grads["x"] = (s["scale"] * d).to(s["x"].dtype)
    grads["y"] = q.to(s["y"].dtype)
    return grads


def _plain_segments(s):
    """Sequence of each token (S where it is in none), and whether it counts."""
    T, S = s["scores"].shape[0], s["case"]["S"]
    dev = s["scores"].device
    if s["offsets"] is None:
        seq = torch.zeros(T, dtype=torch.int64, device=dev)
    else:
        seq = torch.searchsorted(s["offsets"][1:].contiguous(),
                                 torch.arange(T, dtype=torch.int32, device=dev), right=True)
    return (seq, seq < S) if s["mask"] is None else (seq, (seq < S) & s["mask"])


def _plain_counts(s):
    E, S = s["scores"].shape[1], s["case"]["S"]
    seq, valid = _plain_segments(s)
    seq = torch.where(valid, seq, S)
    counts = torch.zeros((S + 1) * E, dtype=torch.int32, device=seq.device)
    place = (seq[:, None] * E + s["ids"]).reshape(-1)
    counts.scatter_add_(0, place, torch.ones_like(place, dtype=torch.int32))
    tokens = torch.zeros(S + 1, dtype=torch.int32, device=seq.device)
    tokens.scatter_add_(0, seq, torch.ones_like(seq, dtype=torch.int32))
    return counts.view(S + 1, E)[:S].contiguous(), tokens[:S].contiguous()


def _plain_softmax(scores):
    m = scores.amax(1, keepdim=True)
    e = torch.exp(scores - m)
    z = e.sum(1, keepdim=True)
    return e / z, (m + torch.log(z))[:, 0]


def _plain_balance(s):
    E, S, k = s["scores"].shape[1], s["case"]["S"], s["ids"].shape[1]
    seq, valid = _plain_segments(s)
    counts, tokens = _plain_counts(s)
    p, lse = _plain_softmax(torch.where(valid[:, None], s["scores"], 0.0))
    member = ((seq[None, :] == torch.arange(S, device=seq.device)[:, None]) & valid[None, :]).float()
    n = tokens.clamp(min=1).float()
    mean_p = member @ p / n[:, None]
    f = counts.float() * (E / k) / n[:, None]
    return {"loss": torch.stack(((f * mean_p).sum(1), member @ lse.square() / n), 1),
            "counts": counts, "tokens": tokens}


def _plain_router_back(s):
    E, k = s["scores"].shape[1], s["ids"].shape[1]
    seq, valid = _plain_segments(s)
    p, lse = _plain_softmax(torch.where(valid[:, None], s["scores"], 0.0))
    at = torch.where(valid, seq, 0)
    n = s["tokens"].clamp(min=1).float()
    f = (s["counts"].float() * (E / k) / n[:, None])[at]
    g = s["grad_loss"][at] / n[at][:, None]
    d = p * (g[:, :1] * (f - (f * p).sum(1, keepdim=True)) + 2 * g[:, 1:] * lse[:, None])
    d = torch.where(valid[:, None], d, 0.0)
    w, dw = s["weights"], s["grad_weights"]
    return d.scatter_add_(1, s["ids"].long(), w * (dw - (w * dw).sum(1, keepdim=True)))


def _plain_matrix(s, q, scale, zero):
    v = torch.stack((q & 15, q >> 4), -1).flatten(-2).float()
    v = v.view(*scale.shape, -1)
    v = v - (8.0 if zero is None else zero.float()[..., None])
    return (v * scale.float()[..., None]).flatten(-2)


def _plain_w4(s):
    c, x = s["case"], s["x"].float()
    if not c["k"]:
        y = x @ _plain_matrix(s, s["q"][0], s["scale"][0], None if s["zero"] is None else s["zero"][0]).t()
        return y.to(DTYPES[c["y"]])
    ids = s["ids"].long().reshape(-1)
    W = _plain_matrix(s, s["q"][ids], s["scale"][ids], None if s["zero"] is None else s["zero"][ids])
    rows = x.reshape(-1, c["K"]) if c["slots"] else x.repeat_interleave(c["k"], 0)
    y = torch.matmul(W, rows[:, :, None])[:, :, 0]
    if c["swiglu"]:
        gate, up = y.chunk(2, 1)
        y = gate / (1 + torch.exp(-gate)) * up
    if s["weights"] is not None:
        y = y * s["weights"].reshape(-1, 1)
    return y.view(c["T"], c["k"], -1).to(DTYPES[c["y"]])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in ("norm", "norm_back"):
        return _exact_norm(s)
    if c["op"] in ("balance", "router_back"):
        return _exact_router(s)
    return _exact_w4(s)


def _exact_rms(v, w):
    length = torch.linalg.vector_norm(v, dim=1, keepdim=True)
    return v / torch.sqrt(length ** 2 / v.shape[1] + EPS) * w


def _exact_norm(s):
    c = s["case"]
    back = c["op"] == "norm_back"
    var = {k: None if s[k] is None else s[k].double().requires_grad_(back)
           for k in ("x", "y", "w_post", "w_next", "gate")}
    with torch.set_grad_enabled(back):
        block = var["y"] if var["w_post"] is None else _exact_rms(var["y"], var["w_post"])
        block = block if var["gate"] is None else block * var["gate"]
        if not back:
            out = s["scale"] * var["x"] + block
            return {"out": out, "n": None if var["w_next"] is None else _exact_rms(out, var["w_next"])}
        # the gradient at the stored stream, then through the join
        d, got = s["grad_out"].double(), {}
        if var["w_next"] is not None:
            dx, got["w_next"] = torch.autograd.grad(_exact_rms(var["x"], var["w_next"]),
                                                    (var["x"], var["w_next"]), s["grad_n"].double())
            d = d + dx
        wrt = [k for k in ("y", "w_post", "gate") if var[k] is not None]
        got.update(zip(wrt, torch.autograd.grad(block, [var[k] for k in wrt], d)))
        got["x"] = s["scale"] * d
    return {k: got.get(k) for k in ("x", "y", "gate", "w_post", "w_next")}


def _exact_router(s):
    c = s["case"]
    T, E, k, S = c["T"], c["E"], c["k"], c["S"]
    back = c["op"] == "router_back"
    cuts = [0, T] if s["offsets"] is None else s["offsets"].tolist()
    loss, counts, tokens, terms = [], [], [], []
    scores = s["scores"].double().requires_grad_(back)
    with torch.set_grad_enabled(back):
        for a, b in zip(cuts[:-1], cuts[1:]):
            rows, ids = scores[a:b], s["ids"][a:b].long()
            if s["mask"] is not None:
                rows, ids = rows[s["mask"][a:b]], ids[s["mask"][a:b]]
            n = rows.shape[0]
            share = torch.bincount(ids.reshape(-1), minlength=E)
            counts.append(share)
            tokens.append(n)
            if n == 0:
                loss.append(torch.zeros(2, dtype=torch.float64, device=rows.device))
                continue
            p = torch.softmax(rows, 1).mean(0)
            z = torch.logsumexp(rows, 1).square().mean()
            loss.append(torch.stack(((share.double() * E / (k * n) * p).sum(), z)))
        loss = torch.stack(loss)
        if not back:
            return {"loss": loss, "counts": torch.stack(counts).to(torch.int32),
                    "tokens": torch.tensor(tokens, dtype=torch.int32, device=loss.device)}
        grad = torch.zeros_like(s["scores"], dtype=torch.float64)
        if loss.requires_grad:
            grad = torch.autograd.grad(loss, scores, s["grad_loss"].double())[0]
    w, dw = s["weights"].double(), s["grad_weights"].double()
    through = w * dw - w * (w * dw).sum(1, keepdim=True)
    return grad.scatter_add(1, s["ids"].long(), through)


def _exact_w4(s):
    c = s["case"]
    q = s["q"].to(torch.int16)
    ids = [0] if not c["k"] else s["ids"].reshape(-1).tolist()
    out, known = [], {}
    for i, e in enumerate(ids):
        if e not in known:
            w = torch.empty(c["N"], c["K"], dtype=torch.float64, device=q.device)
            w[:, 0::2] = (q[e] % 16).double()
            w[:, 1::2] = (q[e] // 16).double()
            zero = 8.0 if s["zero"] is None else s["zero"][e].double().repeat_interleave(c["group"], 1)
            known[e] = (w - zero) * s["scale"][e].double().repeat_interleave(c["group"], 1)
        if not c["k"]:
            return s["x"].double() @ known[e].t()
        t, j = divmod(i, c["k"])
        y = known[e] @ (s["x"][t, j] if c["slots"] else s["x"][t]).double()
        if c["swiglu"]:
            half = c["N"] // 2
            y = y[:half] * torch.sigmoid(y[:half]) * y[half:]
        out.append(y if s["weights"] is None else y * s["weights"][t, j].double())
    return torch.stack(out).view(c["T"], c["k"], -1)
