"""Python binding of libmoe_mi355x.so (the routed-expert MoE FFN for gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels of the library.  torch supplies device memory and the current stream;
nothing else of torch is used here.  The library must be built
(``python -m mixture_experts_decode_amd.build``); without it every call raises.
"""

import contextlib
import ctypes
import functools
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_mi355x.so")

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE_TOO_SMALL, ERR_HIP = range(5)
DT = {"f32": 0, "bf16": 1}
FMT = {"f32": 0, "mxfp8": 1, "mxfp4": 2, "fp8_blk128": 3}
PATH = {"auto": 0, "decode": 1, "grouped": 2}
PATH_NAME = {v: k for k, v in PATH.items()}
DOWN_VARIANT = {"auto": 0, "token": 1, "expert": 2}
GATE = {"none": 0, "channel": 1, "token": 2, "full": 3}

_lib = None


class MoeError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: {_lib.moe_status_string(status).decode() if _lib else status}")


class _Weights(ctypes.Structure):
    _fields_ = [("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("num_experts", ctypes.c_int32), ("num_shared", ctypes.c_int32),
                ("format", ctypes.c_int32),
                ("w13", ctypes.c_void_p), ("w13_scale", ctypes.c_void_p),
                ("w2", ctypes.c_void_p), ("w2_scale", ctypes.c_void_p)]


class _Block(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32),
                ("x_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32),
                ("gate_kind", ctypes.c_int32),
                ("res_scale", ctypes.c_float), ("eps", ctypes.c_float),
                ("x_stride", ctypes.c_int64), ("y_stride", ctypes.c_int64),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p),
                ("w_post", ctypes.c_void_p), ("w_next", ctypes.c_void_p),
                ("gate", ctypes.c_void_p)]


class _W4(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int32), ("cols", ctypes.c_int32),
                ("num_mats", ctypes.c_int32), ("group", ctypes.c_int32),
                ("scale_dtype", ctypes.c_int32),
                ("q", ctypes.c_void_p), ("scale", ctypes.c_void_p), ("zero", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I = ctypes.c_int32
_Z = ctypes.c_size_t
_WP = ctypes.POINTER(_Weights)
_BP = ctypes.POINTER(_Block)

_SIGS = {
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_abi_version": (_I, []),
    "moe_decode_max_entries": (_I, []),
    "moe_gate_up": (_I, [_WP, _P, _I, _P, _I, _I, _P, _I, _P]),
    "moe_down_workspace_bytes": (_Z, [_WP, _I, _I]),
    "moe_down": (_I, [_WP, _P, _I, _P, _P, _I, _I, _P, _I, _I, _P, _Z, _P]),
    "moe_align_sort_capacity": (_Z, [_I, _I, _I, _I, _I]),
    "moe_align_sort_workspace_bytes": (_Z, [_I, _I, _I, _I, _I]),
    "moe_align_sort": (_I, [_P, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_quant_rows": (_I, [_P, _I, _I, _I, _P, _P, _P]),
    "moe_grouped_gate_up": (_I, [_WP, _P, _P, _I, _I, _P, _P, _P, _I, _I, _P, _P, _P]),
    "moe_grouped_down": (_I, [_WP, _P, _P, _P, _P, _P, _I, _I, _P, _I, _I, _P, _P]),
    "moe_combine": (_I, [_P, _I, _I, _I, _P, _I, _P]),
    "moe_topk_route": (_I, [_P, _P, _I, _I, _I, _P, _P, _P]),
    "moe_check_routing": (_I, [_P, _I, _I, _I, _P, _P]),
    "moe_balance_workspace_bytes": (_Z, [_I, _I, _I]),
    "moe_balance_loss": (_I, [_P, _P, _P, _P, _I, _I, _I, _I, _P, _P, _P, _P, _Z, _P]),
    "moe_router_backward": (_I, [_P] * 9 + [_I, _I, _I, _I, _P, _P]),
    "moe_block_norm": (_I, [_BP, _P, _P, _P]),
    "moe_block_norm_backward_workspace_bytes": (_Z, [_I, _I]),
    "moe_block_norm_backward": (_I, [_BP, _P, _P, _P, _P, _P, _P, _P, _P, _Z, _P]),
    "moe_w4_linear": (_I, [ctypes.POINTER(_W4), _P, _P, _P, _I, _I, _I, _I, _P, _I, _P]),
    "moe_choose_path": (_I, [_WP, _I, _I]),
    "moe_layer_workspace_bytes": (_Z, [_WP, _I, _I, _I, _I]),
    "moe_layer": (_I, [_WP, _P, _I, _P, _P, _I, _I, _P, _I, _I, _I, _P, _Z,
                       ctypes.POINTER(_I), _P]),
    "moe_layer_noalloc_max_bytes": (_Z, []),
    "moe_layer_noalloc": (_I, [_WP, _P, _I, _P, _P, _I, _I, _P, _I, _I, _I,
                               ctypes.POINTER(_I), _P]),
    "moe_util_copy": (_I, [_P, _P, _Z, _P]),
    "moe_util_read": (_I, [_P, _Z, _P, _P]),
    "moe_util_read_sink_len": (_I, []),
    "moe_util_fill": (_I, [_P, _Z, ctypes.c_uint32, _P]),
    "moe_util_num_cus": (_I, []),
}

EXPORTS = tuple(_SIGS)


def load(path=LIB_PATH):
    """Load the HIP library (idempotent).  Raises if it is not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is not built: run python -m mixture_experts_decode_amd.build")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib


def _check(status, where):
    if status != OK:
        raise MoeError(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _on_stream(fn):
    """Run a binding call with its `stream` argument made torch's current
    stream, so every tensor the call allocates (outputs, scratch) belongs to
    the stream its kernels are enqueued on and the caching allocator does not
    hand that memory to other work while they run."""
    @functools.wraps(fn)
    def wrapped(*args, stream=None, **kwargs):
        ctx = torch.cuda.stream(stream) if stream is not None else contextlib.nullcontext()
        with ctx:
            return fn(*args, stream=stream, **kwargs)
    return wrapped


class Weights:
    """One layer's expert weights resident on the device.

    Tensors as stored (see include/moe_mi355x.h): w13 [E+S][2][I][H*],
    w2 [E+S][H][I*] and their scales (None for "f32")."""

    def __init__(self, fmt, hidden, inter, num_experts, num_shared, w13, w13_scale, w2, w2_scale):
        self.fmt = fmt
        self.hidden, self.inter = hidden, inter
        self.num_experts, self.num_shared = num_experts, num_shared
        self.tensors = (w13, w13_scale, w2, w2_scale)
        self._s = _Weights(hidden, inter, num_experts, num_shared, FMT[fmt],
                           w13.data_ptr(), None if w13_scale is None else w13_scale.data_ptr(),
                           w2.data_ptr(), None if w2_scale is None else w2_scale.data_ptr())

    @classmethod
    def from_arrays(cls, cfg, arrays, device="cuda"):
        """Upload stacked numpy arrays (as made by the workload generators)."""
        def up(a):
            return None if a is None else torch.from_numpy(a).to(device)
        return cls(cfg.fmt, cfg.hidden, cfg.inter, cfg.num_experts, cfg.num_shared,
                   up(arrays["w13"]), up(arrays.get("w13_scale")), up(arrays["w2"]),
                   up(arrays.get("w2_scale")))

    @property
    def ref(self):
        return ctypes.byref(self._s)

    @property
    def slots_extra(self):
        return self.num_shared

    def nbytes(self):
        return sum(t.numel() * t.element_size() for t in self.tensors if t is not None)


def _dt(t):
    if t.dtype == torch.float32:
        return DT["f32"]
    if t.dtype in (torch.bfloat16, torch.int16, torch.uint16):
        return DT["bf16"]
    raise ValueError(f"unsupported activation dtype {t.dtype}")


def _alloc(shape, dtype, device):
    tdt = torch.float32 if dtype == "f32" else torch.bfloat16
    return torch.empty(shape, dtype=tdt, device=device)


@_on_stream
def gate_up(W, x, topk_ids, h=None, h_dtype="f32", stream=None):
    """h [T][k+S][I] for the decode path."""
    load()
    t, k = topk_ids.shape
    if h is None:
        h = _alloc((t, k + W.num_shared, W.inter), h_dtype, x.device)
    st = _lib.moe_gate_up(W.ref, _ptr(x), _dt(x), _ptr(topk_ids), t, k, _ptr(h), _dt(h),
                          _stream(stream))
    _check(st, "moe_gate_up")
    return h


@_on_stream
def down(W, h, topk_ids, topk_weights, y=None, y_dtype="f32", variant="auto", workspace=None,
         stream=None):
    """y [T][H] for the decode path.  variant: "token" (token-major), "expert"
    (expert-major with a slot buffer in `workspace`) or "auto" (as moe_layer
    does; it may pick either, so a slot buffer is passed)."""
    load()
    t, k = topk_ids.shape
    if y is None:
        y = _alloc((t, W.hidden), y_dtype, h.device)
    ws, wsb = None, 0
    if variant in ("expert", "auto"):
        wsb = _lib.moe_down_workspace_bytes(W.ref, t, k)
        if workspace is None:
            workspace = torch.empty(max(wsb, 16), dtype=torch.uint8, device=h.device)
        ws, wsb = _ptr(workspace), workspace.numel() * workspace.element_size()
    st = _lib.moe_down(W.ref, _ptr(h), _dt(h), _ptr(topk_ids), _ptr(topk_weights), t, k, _ptr(y),
                       _dt(y), DOWN_VARIANT[variant], ws, wsb, _stream(stream))
    _check(st, "moe_down")
    return y


def align_sort_capacity(t, k, num_experts, num_shared, block):
    load()
    return _lib.moe_align_sort_capacity(t, k, num_experts, num_shared, block)


@_on_stream
def align_sort(topk_ids, num_experts, num_shared, block, stream=None):
    """Returns dict of device tensors: sorted_token_ids [cap], expert_ids
    [cap/bs], expert_offsets [E+S+1], num_tokens_post_padded [1]."""
    load()
    t, k = topk_ids.shape
    dev = topk_ids.device
    cap = _lib.moe_align_sort_capacity(t, k, num_experts, num_shared, block)
    wsb = _lib.moe_align_sort_workspace_bytes(t, k, num_experts, num_shared, block)
    out = {
        "sorted_token_ids": torch.empty(cap, dtype=torch.int32, device=dev),
        "expert_ids": torch.empty(max(cap // block, 1), dtype=torch.int32, device=dev),
        "expert_offsets": torch.empty(num_experts + num_shared + 1, dtype=torch.int32, device=dev),
        "num_tokens_post_padded": torch.empty(1, dtype=torch.int32, device=dev),
    }
    ws = torch.empty(max(wsb, 4), dtype=torch.uint8, device=dev)
    st = _lib.moe_align_sort(_ptr(topk_ids), t, k, num_experts, num_shared, block,
                             _ptr(out["sorted_token_ids"]), _ptr(out["expert_ids"]),
                             _ptr(out["expert_offsets"]), _ptr(out["num_tokens_post_padded"]),
                             _ptr(ws), ws.numel(), _stream(stream))
    _check(st, "moe_align_sort")
    out["capacity"] = cap
    out["_ws"] = ws
    return out


@_on_stream
def quant_rows(x, stream=None):
    """Each token row of x [T][H] quantised once to MXFP8: (xq [T][H] u8,
    xs [T][H/32] u8)."""
    load()
    t, h = x.shape
    xq = torch.empty((t, h), dtype=torch.uint8, device=x.device)
    xs = torch.empty((t, h // 32), dtype=torch.uint8, device=x.device)
    st = _lib.moe_quant_rows(_ptr(x), _dt(x), t, h, _ptr(xq), _ptr(xs), _stream(stream))
    _check(st, "moe_quant_rows")
    return xq, xs


@_on_stream
def grouped_gate_up(W, xq, xs, t, k, sorted_ids, expert_ids, npp, capacity, block, stream=None):
    """Grouped gate_up GEMM over the sorted rows; row r reads token row
    sorted_ids[r] // (k + S) of xq / xs.  Returns (hq [2][cap][I], hs [2][cap][I/32])."""
    load()
    hq = torch.empty((2, capacity, W.inter), dtype=torch.uint8, device=xq.device)
    hs = torch.empty((2, capacity, W.inter // 32), dtype=torch.uint8, device=xq.device)
    st = _lib.moe_grouped_gate_up(W.ref, _ptr(xq), _ptr(xs), t, k, _ptr(sorted_ids),
                                  _ptr(expert_ids), _ptr(npp), capacity, block, _ptr(hq), _ptr(hs),
                                  _stream(stream))
    _check(st, "moe_grouped_gate_up")
    return hq, hs


@_on_stream
def grouped_down(W, hq, hs, sorted_ids, expert_ids, npp, capacity, block, topk_weights, t, k,
                 slot_out=None, stream=None):
    load()
    if slot_out is None:
        slot_out = torch.empty((t * (k + W.num_shared), W.hidden), dtype=torch.bfloat16,
                               device=hq.device)
    if slot_out.dtype != torch.bfloat16:
        raise TypeError("slot_out holds BF16 values")
    st = _lib.moe_grouped_down(W.ref, _ptr(hq), _ptr(hs), _ptr(sorted_ids), _ptr(expert_ids),
                               _ptr(npp), capacity, block, _ptr(topk_weights), t, k,
                               _ptr(slot_out), _stream(stream))
    _check(st, "moe_grouped_down")
    return slot_out


@_on_stream
def combine(slot_out, t, slots, y=None, y_dtype="f32", stream=None):
    load()
    if slot_out.dtype != torch.bfloat16:
        raise TypeError("slot_out holds BF16 values (as grouped_down writes them)")
    h = slot_out.shape[1]
    if y is None:
        y = _alloc((t, h), y_dtype, slot_out.device)
    st = _lib.moe_combine(_ptr(slot_out), t, slots, h, _ptr(y), _dt(y), _stream(stream))
    _check(st, "moe_combine")
    return y


@_on_stream
def topk_route(scores, k, bias=None, ids=None, wts=None, stream=None):
    """Router front-end: scores [T][E] float32 (device), bias [E] or None ->
    (topk_ids int32 [T][k], topk_weights float32 [T][k]), written into ids /
    wts when given."""
    load()
    t, e = scores.shape
    if ids is None:
        ids = torch.empty((t, k), dtype=torch.int32, device=scores.device)
    if wts is None:
        wts = torch.empty((t, k), dtype=torch.float32, device=scores.device)
    st = _lib.moe_topk_route(_ptr(scores), None if bias is None else _ptr(bias), t, e, k, _ptr(ids),
                             _ptr(wts), _stream(stream))
    _check(st, "moe_topk_route")
    return ids, wts


@_on_stream
def check_routing(ids, num_experts, result=None, stream=None):
    """Device check of topk_ids [T][k] int32: returns (or fills) an int32 [2]
    device tensor (number of ids outside [0, num_experts), first such entry
    t*k + j or -1)."""
    load()
    t, k = ids.shape
    if result is None:
        result = torch.empty(2, dtype=torch.int32, device=ids.device)
    st = _lib.moe_check_routing(_ptr(ids) if ids.numel() else None, t, k, num_experts,
                                _ptr(result), _stream(stream))
    _check(st, "moe_check_routing")
    return result


# ---- operators around the layer ------------------------------------------
#
# As everywhere in this binding no call records an autograd graph: a result is
# a constant to torch, whatever its inputs require, and the gradients are calls
# of their own (router_backward, block_norm_backward), which a caller's
# torch.autograd.Function can make.

def _on_device(fn):
    """Run a binding call on its first tensor's device and, with `stream`,
    with that stream made torch's current one (as _on_stream)."""
    name = fn.__code__.co_varnames[0]

    @functools.wraps(fn)
    def wrapped(*args, stream=None, **kwargs):
        first = args[0] if args else kwargs[name]
        dev = first.get_device()
        if dev < 0:
            raise ValueError(f"{fn.__name__}: tensors must be on a GPU, not on {first.device}")
        if stream is None and dev == torch.cuda.current_device():
            return fn(*args, **kwargs)
        if stream is not None and stream.device != first.device:
            raise ValueError(f"{fn.__name__}: the stream belongs to {stream.device}, the tensors to "
                             f"{first.device}")
        with torch.cuda.device(dev), torch.cuda.stream(stream):
            return fn(*args, **kwargs)
    return wrapped


def _current(t):
    """Handle of torch's current stream on t's device (a stream object costs
    a small call more than its launch)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _need(cond, what):
    if not cond:
        raise ValueError(what)


def _tensor(t, name, like, shape, dtypes):
    """Data pointer of t (None for None) after its checks: on `like`'s device,
    contiguous, of that shape and one of those dtypes."""
    if t is None:
        return None
    if t.device != like.device or t.dtype not in dtypes or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous tensor {list(shape)} of {dtypes} on {like.device} is "
                         f"needed, not {list(t.shape)} {t.dtype} on {t.device}"
                         f"{'' if t.is_contiguous() else ', strided'}")
    return t.data_ptr()


_F32, _I32 = (torch.float32,), (torch.int32,)
_BYTES = (torch.uint8, torch.bool)


def _sequences(seq_offsets, scores):
    if seq_offsets is None:
        return 1, None
    _need(seq_offsets.dim() == 1 and seq_offsets.shape[0] >= 2, "seq_offsets: [S + 1] with S >= 1")
    return seq_offsets.shape[0] - 1, _tensor(seq_offsets, "seq_offsets", scores, seq_offsets.shape, _I32)


@_on_device
def balance_loss(scores, ids, mask=None, seq_offsets=None):
    """Router statistics of scores [T][E] float32 and the routed ids [T][k]:
    (loss [S][2] float32 -- balance and z loss, counts [S][E] int32, tokens [S]
    int32).  mask [T] bool: tokens that count; seq_offsets [S+1] int32: the
    sequences' bounds in T (default: one sequence of all tokens).  The loss has
    no autograd graph: its gradient is router_backward's."""
    load()
    _need(scores.dim() == 2 and ids.dim() == 2, "scores [T][E] and ids [T][k] are needed")
    t, e = scores.shape
    k = ids.shape[1]
    s, offs = _sequences(seq_offsets, scores)
    args = (_tensor(scores, "scores", scores, (t, e), _F32), _tensor(ids, "ids", scores, (t, k), _I32),
            _tensor(mask, "mask", scores, (t,), _BYTES), offs)
    loss, counts, tokens = scores.new_empty((s, 2)), ids.new_empty((s, e)), ids.new_empty((s,))
    wsb = _lib.moe_balance_workspace_bytes(t, e, s)
    ws = torch.empty(wsb, dtype=torch.uint8, device=scores.device) if wsb else None
    st = _lib.moe_balance_loss(*args, t, e, k, s, counts.data_ptr(), tokens.data_ptr(),
                               loss.data_ptr(), None if ws is None else ws.data_ptr(), wsb,
                               _current(scores))
    _check(st, "moe_balance_loss")
    return loss, counts, tokens


@_on_device
def router_backward(scores, ids, grad_loss=None, counts=None, tokens=None, mask=None,
                    seq_offsets=None, weights=None, grad_weights=None, out=None):
    """Gradient [T][E] float32 of the scores: from grad_loss [S][2] with counts
    and tokens of balance_loss on the same inputs, and / or from grad_weights
    [T][k] through the routing weights of topk_route."""
    load()
    _need(scores.dim() == 2 and ids.dim() == 2, "scores [T][E] and ids [T][k] are needed")
    t, e = scores.shape
    k = ids.shape[1]
    s, offs = _sequences(seq_offsets, scores)
    po = _tensor(out, "out", scores, (t, e), _F32)
    if out is None:
        out = torch.empty_like(scores)
        po = out.data_ptr()
    st = _lib.moe_router_backward(
        _tensor(scores, "scores", scores, (t, e), _F32), _tensor(ids, "ids", scores, (t, k), _I32),
        _tensor(weights, "weights", scores, (t, k), _F32),
        _tensor(grad_weights, "grad_weights", scores, (t, k), _F32),
        _tensor(mask, "mask", scores, (t,), _BYTES), offs,
        _tensor(counts, "counts", scores, (s, e), _I32), _tensor(tokens, "tokens", scores, (s,), _I32),
        _tensor(grad_loss, "grad_loss", scores, (s, 2), _F32), t, e, k, s, po,
        _current(scores))
    _check(st, "moe_router_backward")
    return out


_ROWS = {torch.bfloat16: DT["bf16"], torch.float32: DT["f32"]}


def _row_stride(x, name):
    """Elements from a row of x [T][H] to the next, after its checks."""
    if x.dtype not in _ROWS:
        raise ValueError(f"{name}: bfloat16 or float32 rows are needed, not {x.dtype}")
    if x.dim() != 2:
        raise ValueError(f"{name}: rows [T][H] are needed")
    t, h = x.shape
    if x.is_contiguous():
        return h
    row, col = x.stride()
    if (h > 1 and col != 1) or (t > 1 and row < h):
        raise ValueError(f"{name}: rows [T][H] with consecutive elements are needed")
    return row if t > 1 else h


def _block(like, x, y, w_post, w_next, gate, res_scale, eps):
    t, h = like.shape
    dt = like.dtype
    dts, code = (dt,), _ROWS[dt]
    px = py = pg = None
    xs = ys = h
    ycode, kind = code, "none"
    if x is not None:
        px, xs = x.data_ptr(), _row_stride(x, "x")
    if y is not None:
        ys = _row_stride(y, "y")
        _need(y.shape == like.shape and y.device == like.device, "y: of x's shape and device")
        py, ycode = y.data_ptr(), _ROWS[y.dtype]
    if gate is not None:
        if gate.dim() == 1:
            kind, shape, gdt = "channel", (h,), dts
        elif gate.dim() == 2 and gate.shape[1] == 1 and (h > 1 or gate.dtype == torch.float32):
            kind, shape, gdt = "token", (t, 1), _F32
        else:
            kind, shape, gdt = "full", (t, h), dts
        pg = _tensor(gate, "gate", like, shape, gdt)
    return _Block(t, h, code, ycode, GATE[kind], res_scale, eps, xs, ys, px, py,
                  _tensor(w_post, "w_post", like, (h,), dts), _tensor(w_next, "w_next", like, (h,), dts),
                  pg), kind


@_on_device
def block_norm(x, y=None, w_post=None, w_next=None, gate=None, res_scale=1.0, eps=1e-6, out=None,
               n=None):
    """The norm after a block, its gate and residual join, and the norm before
    the next block: (out, n) with out = res_scale x + gate (.) norm(y) w_post and
    n = norm(out) w_next.  Without y: (None, norm(x) w_next).  x, y [T][H] with
    any row stride; weights [H] and gate [H] (channels) or [T][H] in x's dtype,
    or gate [T][1] float32 (tokens).  out may be x (in place).  The results have
    no autograd graph: their gradient is block_norm_backward's."""
    load()
    _need(x.dim() == 2 and x.dtype in _ROWS, "x: bfloat16 or float32 rows [T][H] are needed")
    b, _ = _block(x, x, y, w_post, w_next, gate, res_scale, eps)
    po = pn = None
    if y is None:
        _need(out is None, "out goes with y")
    elif out is None:
        out = torch.empty_like(x, memory_format=torch.contiguous_format)
        po = out.data_ptr()
    else:
        po = _tensor(out, "out", x, x.shape, (x.dtype,))
    if w_next is None:
        _need(n is None, "n goes with w_next")
    elif n is None:
        n = torch.empty_like(x, memory_format=torch.contiguous_format)
        pn = n.data_ptr()
    else:
        pn = _tensor(n, "n", x, x.shape, (x.dtype,))
    st = _lib.moe_block_norm(b, po, pn, _current(x))
    _check(st, "moe_block_norm")
    return out, n


def block_norm_backward(grad_out, grad_n, out, y=None, w_post=None, w_next=None, gate=None,
                        res_scale=1.0, eps=1e-6, stream=None):
    """Gradients of block_norm's inputs, a dict of "x", "y", "gate", "w_post"
    and "w_next" (None where the input was), from grad_out and grad_n (either
    may be None where it does not reach the loss or does not exist).  out: what
    block_norm returned (without y: its x)."""
    like = grad_out if grad_out is not None else grad_n
    _need(like is not None, "grad_out or grad_n is needed")
    return _block_norm_backward(like, grad_out, grad_n, out, y, w_post, w_next, gate, res_scale, eps,
                                stream=stream)


@_on_device
def _block_norm_backward(like, grad_out, grad_n, out, y, w_post, w_next, gate, res_scale, eps):
    load()
    _need(like.dtype in _ROWS and like.dim() == 2, "gradients: bfloat16 or float32 rows [T][H]")
    t, h = like.shape
    dev, dts = like.device, (like.dtype,)
    if w_next is not None:
        _need(out is not None and out.shape == like.shape and out.dtype == like.dtype and
              out.device == dev, "out: of the gradients' shape, dtype and device")
        if grad_n is None:
            grad_n = torch.zeros_like(like)
    b, kind = _block(like, out if w_next is not None else None, y, w_post, w_next, gate, res_scale, eps)
    g = {"x": torch.empty_like(like, memory_format=torch.contiguous_format), "y": None, "gate": None,
         "w_post": None, "w_next": None}
    if y is not None:
        g["y"] = torch.empty((t, h), dtype=y.dtype, device=dev)
    if gate is not None:
        g["gate"] = torch.empty(gate.shape, dtype=like.dtype if kind == "full" else torch.float32,
                                device=dev)
    for name, w in (("w_post", w_post), ("w_next", w_next)):
        if w is not None:
            g[name] = torch.empty((h,), dtype=torch.float32, device=dev)
    wsb = _lib.moe_block_norm_backward_workspace_bytes(t, h)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=dev)
    st = _lib.moe_block_norm_backward(
        b, _tensor(grad_out, "grad_out", like, (t, h), dts), _tensor(grad_n, "grad_n", like, (t, h), dts),
        g["x"].data_ptr(), _ptr(g["y"]), _ptr(g["gate"]), _ptr(g["w_post"]), _ptr(g["w_next"]),
        ws.data_ptr(), wsb, _current(like))
    _check(st, "moe_block_norm_backward")
    return g


class W4Weights:
    """Matrices of 4-bit codes resident on the device (see moe_w4_linear): q
    [N][K/2] or [E][N][K/2] uint8, two codes a byte, the even input in the low
    nibble; scale [..][N][K/G] float32 or bfloat16; zero uint8 of scale's shape,
    or None (8)."""

    def __init__(self, q, scale, zero=None):
        _need(q.dim() in (2, 3) and scale.dim() == q.dim() and scale.dtype in _ROWS,
              "q [E][N][K/2] and scale [E][N][K/G] float32 or bfloat16 are needed")
        (*mats, rows, half), (*smats, srows, groups) = q.shape, scale.shape
        cols = 2 * half
        _need(groups > 0 and cols % groups == 0 and (mats, rows) == (smats, srows),
              "scale: q's shape with one value for every G inputs")
        self.mats, self.rows, self.cols = mats[0] if mats else 1, rows, cols
        self.device = q.device
        self.tensors = (q, scale, zero)
        self._s = _W4(self.rows, cols, self.mats, cols // groups, _ROWS[scale.dtype],
                      _tensor(q, "q", q, q.shape, (torch.uint8,)),
                      _tensor(scale, "scale", q, scale.shape, (scale.dtype,)),
                      _tensor(zero, "zero", q, scale.shape, (torch.uint8,)))

    def nbytes(self):
        return sum(t.numel() * t.element_size() for t in self.tensors if t is not None)


def w4_linear(W, x, ids=None, weights=None, swiglu=False, y=None, y_dtype="f32", stream=None):
    """y [T][N] = x [T][K] times the transpose of W4Weights W's one matrix; with ids
    [T][k]: y [T][k][N] of the routed matrices, x [T][K] or [T][k][K].  swiglu:
    SiLU(first half) * second half of the outputs; weights [T][k] float32: slot
    (t, j)'s outputs times its weight.  y has no autograd graph, and there is no
    backward pass."""
    return _w4_linear(x, W, ids, weights, swiglu, y, y_dtype, stream=stream)


@_on_device
def _w4_linear(x, W, ids, weights, swiglu, y, y_dtype):
    load()
    _need(W.device == x.device, "W and x: on one device")
    t = x.shape[0]
    outs = W.rows // 2 if swiglu else W.rows
    slots = x.dim() == 3
    if ids is None:
        _need(W.mats == 1, "ids are needed to choose among several matrices")
        k, shape = 1, (t, outs)
        _need(not slots, "x [T][K] is needed without ids")
    else:
        _need(ids.dim() == 2, "ids [T][k] are needed")
        k = ids.shape[1]
        shape = (t, k, outs)
    if y is None:
        _need(y_dtype in DT, f"y_dtype: one of {list(DT)}")
        y = x.new_empty(shape, dtype=torch.float32 if y_dtype == "f32" else torch.bfloat16)
    else:
        _tensor(y, "y", x, shape, tuple(_ROWS))
    st = _lib.moe_w4_linear(
        W._s, _tensor(x, "x", x, (t, k, W.cols) if slots else (t, W.cols), (torch.bfloat16,)),
        _tensor(ids, "ids", x, (t, k), _I32), _tensor(weights, "weights", x, (t, k), _F32), t, k,
        int(slots), int(swiglu), y.data_ptr(), _ROWS[y.dtype],
        _current(x))
    _check(st, "moe_w4_linear")
    return y


def choose_path(W, t, k):
    load()
    return PATH_NAME[_lib.moe_choose_path(W.ref, t, k)]


def layer_workspace_bytes(W, t, k, path="auto", block=0):
    load()
    return _lib.moe_layer_workspace_bytes(W.ref, t, k, PATH[path], block)


@_on_stream
def layer(W, x, topk_ids, topk_weights, path="auto", block=0, y=None, y_dtype="f32",
          workspace=None, stream=None):
    """y [T][H] for the whole layer; returns (y, path that ran)."""
    load()
    t, k = topk_ids.shape
    if y is None:
        y = _alloc((t, W.hidden), y_dtype, x.device)
    need = _lib.moe_layer_workspace_bytes(W.ref, t, k, PATH[path], block)
    if workspace is None:
        workspace = torch.empty(max(need, 256), dtype=torch.uint8, device=x.device)
    chosen = ctypes.c_int32(-1)
    st = _lib.moe_layer(W.ref, _ptr(x), _dt(x), _ptr(topk_ids), _ptr(topk_weights), t, k, _ptr(y),
                        _dt(y), PATH[path], block, _ptr(workspace),
                        workspace.numel() * workspace.element_size(), ctypes.byref(chosen),
                        _stream(stream))
    _check(st, "moe_layer")
    return y, PATH_NAME.get(chosen.value, "?")


def layer_noalloc_max_bytes():
    load()
    return _lib.moe_layer_noalloc_max_bytes()


def layer_noalloc(W, x, topk_ids, topk_weights, y, path="auto", block=0, stream=None):
    """moe_layer_noalloc: y [T][H] (caller-allocated, written in place) with
    the library's own device array as workspace; nothing is allocated here.
    Returns the path that ran."""
    load()
    t, k = topk_ids.shape
    chosen = ctypes.c_int32(-1)
    st = _lib.moe_layer_noalloc(W.ref, _ptr(x), _dt(x), _ptr(topk_ids), _ptr(topk_weights), t, k,
                                _ptr(y), _dt(y), PATH[path], block, ctypes.byref(chosen),
                                _stream(stream))
    _check(st, "moe_layer_noalloc")
    return PATH_NAME.get(chosen.value, "?")


# ---- measurement kernels ------------------------------------------------

def util_copy(src, dst, nbytes, stream=None):
    load()
    _check(_lib.moe_util_copy(_ptr(src), _ptr(dst), nbytes, _stream(stream)), "moe_util_copy")


def util_read(src, nbytes, sink, stream=None):
    load()
    _check(_lib.moe_util_read(_ptr(src), nbytes, _ptr(sink), _stream(stream)), "moe_util_read")


def util_fill(dst, nbytes, value=0, stream=None):
    load()
    _check(_lib.moe_util_fill(_ptr(dst), nbytes, value, _stream(stream)), "moe_util_fill")


def num_cus():
    load()
    return _lib.moe_util_num_cus()
