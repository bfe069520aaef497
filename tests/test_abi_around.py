"""Host-side checks of the operators around the layer: every refusal comes
before any launch (no GPU needed; the pointers are never followed)."""

import ctypes
import os

import pytest

P = ctypes.c_void_p
DUMMY = P(4096)


@pytest.fixture(scope="module")
def moe():
    import mixture_experts_decode_amd as m
    if not os.path.exists(m.LIB_PATH):
        pytest.fail("libmoe_mi355x.so is not built (run python -m mixture_experts_decode_amd.build)")
    m.load()
    return m


def balance(moe, T=4, E=16, k=2, S=1, scores=DUMMY, ids=DUMMY, mask=None, off=None, counts=DUMMY,
            tokens=DUMMY, loss=DUMMY, ws=DUMMY, wsb=1 << 30):
    return moe.load().moe_balance_loss(scores, ids, mask, off, T, E, k, S, counts, tokens, loss, ws, wsb,
                                       None)


def test_balance_refusals(moe):
    bad = moe.ERR_INVALID_ARG
    for kw in (dict(T=-1), dict(E=0), dict(E=1025), dict(k=0), dict(k=17), dict(E=128, k=65), dict(S=0),
               dict(scores=None), dict(ids=None), dict(counts=None), dict(tokens=None), dict(loss=None),
               dict(S=2), dict(T=5000, ws=None), dict(T=5000, ws=P(4100))):
        assert balance(moe, **kw) == bad, kw
    assert balance(moe, T=(1 << 30) + 1) == moe.ERR_UNSUPPORTED
    assert balance(moe, T=1 << 29, k=16) == moe.ERR_UNSUPPORTED
    assert balance(moe, S=(1 << 20) + 1, off=DUMMY) == moe.ERR_UNSUPPORTED
    need = moe.load().moe_balance_workspace_bytes(5000, 16, 1)
    assert need > 0 and balance(moe, T=5000, wsb=need - 1) == moe.ERR_WORKSPACE_TOO_SMALL
    assert moe.load().moe_balance_workspace_bytes(4, 16, 1) == 0
    assert moe.load().moe_balance_workspace_bytes(-1, 16, 1) == 0


def test_balance_workspace_grows_with_the_sizes(moe):
    ws = moe.load().moe_balance_workspace_bytes
    for E in (8, 64, 256, 257, 1024):
        last = 0
        for T in (100, 1000, 10000, 100000, 1000000):
            b = ws(T, E, 1)
            assert b >= last
            last = b
        # a few MB whatever the batch: about one partial row of sums per CU
        assert last <= 16 * (1 << 20)


def router(moe, T=4, E=16, k=2, S=1, scores=DUMMY, ids=DUMMY, w=DUMMY, dw=DUMMY, off=None, counts=DUMMY,
           tokens=DUMMY, gl=DUMMY, out=DUMMY):
    return moe.load().moe_router_backward(scores, ids, w, dw, None, off, counts, tokens, gl, T, E, k, S,
                                          out, None)


def test_router_backward_refusals(moe):
    for kw in (dict(T=-1), dict(E=0), dict(k=17), dict(w=None), dict(dw=None),
               dict(gl=None, w=None, dw=None), dict(out=None), dict(scores=None), dict(counts=None),
               dict(tokens=None), dict(ids=None), dict(S=3)):
        assert router(moe, **kw) == moe.ERR_INVALID_ARG, kw
    assert router(moe, T=0, out=None) == moe.OK
    assert router(moe, T=1 << 29, k=16) == moe.ERR_UNSUPPORTED


def block(moe, **kw):
    d = dict(T=4, H=64, x_dtype=1, y_dtype=1, gate_kind=0, res_scale=1.0, eps=1e-6, x_stride=64,
             y_stride=64, x=4096, y=8192, w_post=4096, w_next=4096, gate=None)
    d.update(kw)
    return moe._Block(**d)


def test_block_norm_refusals(moe):
    f = moe.load().moe_block_norm
    bad = moe.ERR_INVALID_ARG
    assert f(None, DUMMY, DUMMY, None) == bad
    for kw in (dict(T=-1), dict(H=0), dict(x_dtype=2), dict(y_dtype=-1), dict(gate_kind=4),
               dict(gate_kind=1), dict(gate=4096), dict(eps=-1.0), dict(eps=float("nan")),
               dict(res_scale=float("inf")), dict(x_stride=63), dict(y_stride=1), dict(x=None)):
        assert f(block(moe, **kw), P(1 << 16), DUMMY, None) == bad, kw
    assert f(block(moe), None, DUMMY, None) == bad            # out goes with y
    assert f(block(moe), P(1 << 16), None, None) == bad       # n goes with w_next
    assert f(block(moe, w_next=None), P(1 << 16), DUMMY, None) == bad
    assert f(block(moe, y=None), None, DUMMY, None) == bad    # w_post without y
    assert f(block(moe, y=None, w_post=None, w_next=None), None, None, None) == bad
    assert f(block(moe, x_stride=72), DUMMY, P(1 << 16), None) == bad   # in place with another stride
    assert f(block(moe), P(1 << 16), P(1 << 16), None) == bad                 # out and n are two buffers
    assert f(block(moe, H=16385, x_stride=16385, y_stride=16385), P(1 << 16), DUMMY,
             None) == moe.ERR_UNSUPPORTED
    assert f(block(moe, x_dtype=0, y_dtype=1), P(1 << 16), DUMMY, None) == moe.ERR_UNSUPPORTED
    assert f(block(moe, T=0), None, None, None) == moe.OK


def test_block_norm_backward_refusals(moe):
    lib = moe.load()
    need = lib.moe_block_norm_backward_workspace_bytes(4, 64)
    assert need >= 3 * 64 * 4

    def f(b=None, go=DUMMY, gn=DUMMY, dx=DUMMY, dy=DUMMY, dg=None, dwp=DUMMY, dwn=DUMMY, ws=DUMMY, wsb=need):
        return lib.moe_block_norm_backward(block(moe) if b is None else b, go, gn, dx, dy, dg, dwp, dwn, ws,
                                           wsb, None)

    for kw in (dict(gn=None), dict(dx=None), dict(dy=None), dict(dg=DUMMY), dict(dwp=None), dict(dwn=None),
               dict(ws=None), dict(ws=P(4104)), dict(b=block(moe, y=None)), dict(b=block(moe, x=None)),
               dict(b=block(moe, y=None, w_post=None, w_next=None), gn=None, dy=None, dwp=None, dwn=None),
               dict(b=block(moe, w_next=None), go=None, gn=None, dwn=None),
               dict(b=block(moe, gate_kind=1, gate=4096))):
        assert f(**kw) == moe.ERR_INVALID_ARG, kw
    assert f(wsb=need - 1) == moe.ERR_WORKSPACE_TOO_SMALL
    assert lib.moe_block_norm_backward_workspace_bytes(4, 20000) == 0
    assert lib.moe_block_norm_backward_workspace_bytes(0, 64) == 0


def test_binding_refuses_host_tensors(moe):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.block_norm(x, w_next=torch.ones(64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        moe.block_norm_backward(x, None, x, x)
    with pytest.raises(ValueError):
        moe.block_norm_backward(None, None, x, x)
    with pytest.raises(ValueError):
        moe.balance_loss(torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32))
    with pytest.raises(ValueError):
        moe.router_backward(torch.zeros(4, 16), torch.zeros(4, 2, dtype=torch.int32))


def w4(moe, T=4, k=1, ids=None, wts=None, x=DUMMY, slots=0, swiglu=0, y=DUMMY, ydt=0, **kw):
    d = dict(rows=32, cols=128, num_mats=1, group=64, scale_dtype=1, q=4096, scale=4096, zero=None)
    d.update(kw)
    return moe.load().moe_w4_linear(moe._W4(**d), x, ids, wts, T, k, slots, swiglu, y, ydt, None)


def test_w4_linear_refusals(moe):
    assert moe.load().moe_w4_linear(None, DUMMY, None, None, 1, 1, 0, 0, DUMMY, 0, None) == moe.ERR_INVALID_ARG
    for kw in (dict(rows=0), dict(cols=0), dict(num_mats=0), dict(group=0), dict(T=-1), dict(k=0),
               dict(scale_dtype=3), dict(ydt=2), dict(slots=2), dict(swiglu=-1), dict(rows=31, swiglu=1),
               dict(num_mats=2), dict(k=2), dict(slots=1), dict(wts=DUMMY), dict(q=None), dict(q=4104),
               dict(scale=None), dict(x=None), dict(x=P(4100)), dict(y=None), dict(scale=4097),
               dict(scale=4098, scale_dtype=0), dict(y=P(4098)), dict(y=P(4097), ydt=1)):
        assert w4(moe, **kw) == moe.ERR_INVALID_ARG, kw
    for kw in (dict(group=16), dict(group=48, cols=96), dict(cols=96), dict(rows=(1 << 24) + 1),
               dict(cols=1 << 21), dict(num_mats=1025, ids=DUMMY), dict(T=(1 << 21) + 1),
               dict(T=(1 << 20) + 1), dict(rows=1 << 17, cols=1 << 20, group=64),
               dict(T=1025, k=2, ids=DUMMY, num_mats=4)):
        assert w4(moe, **kw) == moe.ERR_UNSUPPORTED, kw
    assert w4(moe, T=0, x=None, y=None) == moe.OK


def test_block_norm_in_place_with_a_stride(moe):
    """Row t of out or n would be written where other rows of x still stand."""
    f = moe.load().moe_block_norm
    strided = dict(x_stride=72)
    assert f(block(moe, **strided), P(1 << 16), DUMMY, None) == moe.ERR_INVALID_ARG
    assert f(block(moe, y=None, w_post=None, **strided), None, DUMMY, None) == moe.ERR_INVALID_ARG
    assert f(block(moe, w_next=None, **strided), DUMMY, None, None) == moe.ERR_INVALID_ARG


def test_balance_misaligned_pointers(moe):
    """Elements of four bytes at addresses of four (bytes of the mask anywhere)."""
    odd = P(4098)
    for name in ("scores", "ids", "off", "counts", "tokens", "loss"):
        assert balance(moe, **{name: odd}) == moe.ERR_INVALID_ARG, name
    for name in ("scores", "ids", "w", "dw", "off", "counts", "tokens", "gl", "out"):
        assert router(moe, **{name: odd}) == moe.ERR_INVALID_ARG, name


def test_block_norm_misaligned_pointers(moe):
    """Elements of their own type's size."""
    lib, bad = moe.load(), moe.ERR_INVALID_ARG
    byte, half = 4097, 4098
    a, b = P(1 << 16), P(1 << 17)
    for kw in (dict(x=byte), dict(y=byte), dict(w_post=byte), dict(w_next=byte), dict(y=half, y_dtype=0),
               dict(gate=byte, gate_kind=1), dict(gate=byte, gate_kind=3), dict(gate=half, gate_kind=2)):
        assert lib.moe_block_norm(block(moe, **kw), a, b, None) == bad, kw
        g = a if "gate" in kw else None
        assert lib.moe_block_norm_backward(block(moe, **kw), a, a, b, b, g, a, a, a, 1 << 30, None) == bad, kw
    assert lib.moe_block_norm(block(moe), P(byte), b, None) == bad
    assert lib.moe_block_norm(block(moe), a, P(byte), None) == bad
    good = dict(go=a, gn=a, dx=b, dy=b, dg=a, dwp=a, dwn=a)
    for name, at, gate in (("go", byte, 1), ("gn", byte, 1), ("dx", byte, 1), ("dy", byte, 1), ("dg", half, 1),
                           ("dg", half, 2), ("dg", byte, 3), ("dwp", half, 1), ("dwn", half, 1)):
        p = {**good, name: P(at)}
        assert lib.moe_block_norm_backward(block(moe, gate=4096, gate_kind=gate), p["go"], p["gn"], p["dx"], p["dy"],
                                           p["dg"], p["dwp"], p["dwn"], a, 1 << 30, None) == bad, (name, gate)


def test_w4_misaligned_routing(moe):
    for kw in (dict(ids=P(4098)), dict(ids=DUMMY, wts=P(4098))):
        assert w4(moe, num_mats=4, k=2, **kw) == moe.ERR_INVALID_ARG, kw
