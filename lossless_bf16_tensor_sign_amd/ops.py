"""Python binding of libzc_ops (the C ABI in include/zc_ops.h): the operators of
a training step before a buffer is compressed and after it is decoded.

The calls check shapes, types and devices, allocate their outputs on the
stream and queue the kernels; nothing is copied, cast or synchronised.  Each
takes stream= (a torch stream; by default the current one); its work is ordered
after what was queued on that stream alone, and its arguments may be freed at
once (but a TensorList or AdamWTensors, and with the current stream tensors of
another, are the caller's to keep until the work has ended).  Small calls are
bound by this host code, so it passes plain integers to the library and asks
torch for the stream's handle alone.  There is no fallback: if libzc_ops.so is
missing, every call raises.

route, dispatch and combine take part in autograd, with the gradient calls as
their backward: for logits, x, rows, weights and base that require a gradient
while gradients are recorded.  (Experts, slots and the router's bias have
none.)  The gradient calls, grad_norm and adamw are not differentiable.
"""
from __future__ import annotations

import ctypes as ct
import os

import torch
from torch.autograd.function import once_differentiable

from .zc import ZC_OK, ZcError, _HERE, _on

OPS_LIB_PATH = os.path.join(_HERE, "libzc_ops.so")

ZC_BF16, ZC_F16, ZC_F32, ZC_E4M3 = 0, 1, 2, 3
ZC_MAX_EXPERTS, ZC_MAX_TOPK, ZC_STATE_BLOCK = 1024, 32, 256
SCORES = {"softmax": 0, "sigmoid": 1}
GROUP_SCORES = {"max": 0, "top2": 1}


class Router(ct.Structure):
    _fields_ = [("experts", ct.c_int32), ("k", ct.c_int32), ("score", ct.c_int32),
                ("groups", ct.c_int32), ("top_groups", ct.c_int32), ("group_score", ct.c_int32),
                ("renorm", ct.c_int32), ("scale", ct.c_float)]


class Tensor(ct.Structure):
    _fields_ = [("data", ct.c_void_p), ("n", ct.c_int64)]


class AdamWTensor(ct.Structure):
    _fields_ = [("param", ct.c_void_p), ("master", ct.c_void_p), ("grad", ct.c_void_p),
                ("avg", ct.c_void_p), ("sq", ct.c_void_p), ("avg_scale", ct.c_void_p),
                ("sq_scale", ct.c_void_p), ("n", ct.c_int64)]


class AdamWConfig(ct.Structure):
    _fields_ = [("param_dtype", ct.c_int32), ("grad_dtype", ct.c_int32),
                ("state_dtype", ct.c_int32), ("pad", ct.c_int32), ("step", ct.c_int64),
                ("lr", ct.c_double), ("beta1", ct.c_double), ("beta2", ct.c_double),
                ("eps", ct.c_double), ("weight_decay", ct.c_double)]

_DTYPES = {torch.bfloat16: ZC_BF16, torch.float16: ZC_F16, torch.float32: ZC_F32}

# Handle of the current stream of a device, by its index:
# torch.cuda.current_stream() builds a stream object for the same number, 2.7
# us against 0.1 us.
_current_stream = torch._C._cuda_getCurrentRawStream
# torch's number of the current GPU; torch.cuda.current_device() first sees that
# there is a GPU at all, which a tensor on one shows.
_current_gpu = torch._C._cuda_getDevice

# Counts up the versions of a list of tensors, by which autograd sees that what
# it saved was written since (torch.autograd.graph.increment_version).
_count_version = torch._C._increment_version

_ops = None


def ops_lib():
    """The loaded libzc_ops.so (raises if it has not been built)."""
    global _ops
    if _ops is None:
        if not os.path.exists(OPS_LIB_PATH):
            raise RuntimeError(
                "libzc_ops.so is not built (run __graft_entry__.build() or "
                "python lossless_bf16_tensor_sign_amd/build_ops.py)")
        L = ct.CDLL(OPS_LIB_PATH)
        V, I32, I64 = ct.c_void_p, ct.c_int32, ct.c_int64
        L.zc_route.argtypes = [V, I32, I64, I64, ct.POINTER(Router), V, V, V, V, V]
        L.zc_route_grad.argtypes = [V, I32, I64, I64, ct.POINTER(Router), V, V, V, V]
        L.zc_slots_workspace_bytes.argtypes = [I64, I32]
        L.zc_slots_workspace_bytes.restype = ct.c_size_t
        L.zc_expert_slots.argtypes = [V, I64, I32, I64, V, V, V, ct.c_size_t, V]
        L.zc_dispatch.argtypes = [V, I32, I64, I64, I64, V, I32, V, V]
        L.zc_combine.argtypes = [V, I32, I64, I64, V, I32, V, V, I64, V, V]
        L.zc_combine_grad.argtypes = [V, I32, I64, I64, I64, V, V, I32, V, V, V, V]
        L.zc_grad_norm_workspace_bytes.argtypes = [ct.POINTER(Tensor), I32, I32]
        L.zc_grad_norm_workspace_bytes.restype = ct.c_size_t
        L.zc_grad_norm.argtypes = [ct.POINTER(Tensor), I32, I32, ct.c_float, V, V, ct.c_size_t, V]
        L.zc_adamw.argtypes = [ct.POINTER(AdamWTensor), I32, ct.POINTER(AdamWConfig), V, V]
        for name in ("route", "route_grad", "expert_slots", "dispatch", "combine", "combine_grad",
                     "grad_norm", "adamw"):
            getattr(L, "zc_" + name).restype = ct.c_int
        _ops = L
    return _ops


def _lend(stream, *tensors):
    """Context that makes `stream` current.  The tensors, which the call reads
    there, may be of another: torch's allocator is told, so that one that is
    freed when the call returns is not given out before the work has ended."""
    for t in tensors:
        if t is not None and t.is_cuda:
            t.record_stream(stream)
    return _on(stream)


def _dtype(t, name):
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError("%s must be bfloat16, float16 or float32, not %s" % (name, t.dtype))
    return code


def _current_device(dev, name="tensors"):
    """dev, which must be the current GPU: kernels are queued there."""
    if dev.type != "cuda" or dev.index != _current_gpu():
        raise ValueError("%s must be on the current GPU, not on %s" % (name, dev))
    return dev


def _device(t, name):
    return _current_device(t.device, name)


def _row_stride(t, name):
    """Elements from one row of a 2-D tensor to the next; a row has no gaps."""
    if t.dim() != 2:
        raise ValueError("%s must have 2 dimensions, not %d" % (name, t.dim()))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have rows without gaps (stride(1) == 1)" % name)
    return t.stride(0)


def _plain(t, name, dtype, device, shape=None):
    """A contiguous tensor of this type, device and shape."""
    if t.dtype is not dtype or t.device != device or not t.is_contiguous():
        raise ValueError("%s must be a contiguous %s tensor on %s" % (name, dtype, device))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, not %s" % (name, tuple(shape), tuple(t.shape)))
    return t.data_ptr()


def _router(experts, k, score, groups, top_groups, group_score, renorm, scale):
    if score not in SCORES or group_score not in GROUP_SCORES:
        raise ValueError("score is one of %s, group_score one of %s"
                         % (sorted(SCORES), sorted(GROUP_SCORES)))
    return Router(experts, k, SCORES[score], groups, groups if top_groups is None else top_groups,
                  GROUP_SCORES[group_score], 1 if renorm else 0, scale)


def _wants_grad(*tensors):
    """Whether autograd has to know of a call with these arguments."""
    for t in tensors:
        if t is not None and t.requires_grad:
            return torch.is_grad_enabled()
    return False


def _without_gaps(t):
    """t, or a copy of it where a row's values do not follow one another."""
    return t if t.shape[1] <= 1 or t.stride(1) == 1 else t.contiguous()


# In a Function's forward gradients are not recorded, so that the calls in it
# take the plain way.

class _Route(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, k, score, bias, groups, top_groups, group_score, renorm, scale, valid):
        experts, weights = route(logits, k, score, bias, groups, top_groups, group_score, renorm,
                                 scale, valid)
        ctx.save_for_backward(logits, experts)
        ctx.options = score, renorm, scale
        ctx.mark_non_differentiable(experts)
        return experts, weights

    @staticmethod
    @once_differentiable
    def backward(ctx, _, d_weights):
        logits, experts = ctx.saved_tensors
        return (route_grad(logits, experts, d_weights.contiguous(), *ctx.options),) + (None,) * 9


class _Dispatch(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, slots):
        ctx.save_for_backward(slots)
        return dispatch(x, slots)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_rows):
        return combine(d_rows.contiguous(), *ctx.saved_tensors), None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, slots, weights, base):
        ctx.save_for_backward(slots, weights, None if weights is None else rows)
        return combine(rows, slots, weights, base)

    @staticmethod
    @once_differentiable
    def backward(ctx, d_out):
        slots, weights, rows = ctx.saved_tensors
        for_rows, _, for_weights, for_base = ctx.needs_input_grad
        d_rows = d_weights = None
        if weights is None:
            if for_rows:
                d_rows = dispatch(_without_gaps(d_out), slots)
        elif for_rows or for_weights:
            d_rows, d_weights = combine_grad(_without_gaps(d_out), rows, slots, weights)
        return (d_rows if for_rows else None, None, d_weights if for_weights else None,
                d_out if for_base else None)


def route(logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_score="max",
          renorm=True, scale=1.0, valid=None, stream=None):
    """Experts and weights of every token, from logits [tokens, experts].

    score "softmax" or "sigmoid"; bias float32 [experts] takes part in the
    choice alone; groups of neighbouring experts, of which the top_groups best
    (by their largest key, or with group_score "top2" the sum of their two
    largest) take part; renorm divides the k weights by their sum; valid bool
    [tokens] marks the tokens to route.  Ties go to the lowest index.
    Returns (int32 [tokens, k], float32 [tokens, k]); a choice without an
    expert is -1 with weight 0."""
    if stream is not None:
        with _lend(stream, logits, bias, valid):
            return route(logits, k, score, bias, groups, top_groups, group_score, renorm, scale,
                         valid)
    if _wants_grad(logits):
        return _Route.apply(logits, k, score, bias, groups, top_groups, group_score, renorm, scale,
                            valid)
    dev = _device(logits, "logits")
    stride = _row_stride(logits, "logits")
    T, E = logits.shape
    r = _router(E, k, score, groups, top_groups, group_score, renorm, scale)
    bp = None if bias is None else _plain(bias, "bias", torch.float32, dev, (E,))
    vp = None if valid is None else _plain(valid, "valid", torch.bool, dev, (T,))
    experts = logits.new_empty((T, max(k, 0)), dtype=torch.int32)
    weights = logits.new_empty((T, max(k, 0)), dtype=torch.float32)
    st = ops_lib().zc_route(logits.data_ptr(), _dtype(logits, "logits"), T, stride, ct.byref(r), bp,
                            vp, experts.data_ptr(), weights.data_ptr(), _current_stream(dev.index))
    if st != ZC_OK:
        raise ZcError(st, "zc_route")
    return experts, weights


def route_grad(logits, experts, d_weights, score="softmax", renorm=True, scale=1.0, stream=None):
    """Gradient of route's weights with respect to the logits (logits' type),
    for experts and d_weights [tokens, k]."""
    if stream is not None:
        with _lend(stream, logits, experts, d_weights):
            return route_grad(logits, experts, d_weights, score, renorm, scale)
    dev = _device(logits, "logits")
    stride = _row_stride(logits, "logits")
    T, E = logits.shape
    if experts.dim() != 2 or experts.shape[0] != T:
        raise ValueError("experts must have shape [tokens, k]")
    r = _router(E, experts.shape[1], score, 1, 1, "max", renorm, scale)
    ep = _plain(experts, "experts", torch.int32, dev)
    gp = _plain(d_weights, "d_weights", torch.float32, dev, experts.shape)
    out = logits.new_empty((T, E))
    st = ops_lib().zc_route_grad(logits.data_ptr(), _dtype(logits, "logits"), T, stride,
                                 ct.byref(r), ep, gp, out.data_ptr(), _current_stream(dev.index))
    if st != ZC_OK:
        raise ZcError(st, "zc_route_grad")
    return out


def expert_slots(experts, num_experts, row_values=1, stream=None):
    """Slots of the (token, choice) pairs in per-expert chunks.

    experts int32, any shape.  Returns (int32 slots of that shape: the pair's
    row, or ~row for one without an expert; int64 counts [num_experts + 1]:
    row_values times each chunk's rows, the last for the rows of pairs
    without an expert).  counts is what compress_dev takes for the dispatched
    rows."""
    if stream is not None:
        with _lend(stream, experts):
            return expert_slots(experts, num_experts, row_values)
    dev = _device(experts, "experts")
    ep = _plain(experts, "experts", torch.int32, dev)
    n = experts.numel()
    L = ops_lib()
    slots = torch.empty_like(experts)
    counts = experts.new_empty(max(num_experts, 0) + 1, dtype=torch.int64)
    need = int(L.zc_slots_workspace_bytes(n, num_experts))
    ws = experts.new_empty(need, dtype=torch.uint8) if need else None
    st = L.zc_expert_slots(ep, n, num_experts, row_values, slots.data_ptr(), counts.data_ptr(),
                           None if ws is None else ws.data_ptr(), need, _current_stream(dev.index))
    if st != ZC_OK:
        raise ZcError(st, "zc_expert_slots")
    return slots, counts


def _slots(slots, tokens, dev):
    if slots.dim() != 2 or slots.shape[0] != tokens:
        raise ValueError("slots must have shape [tokens, k]")
    return _plain(slots, "slots", torch.int32, dev)


def dispatch(x, slots, stream=None):
    """Rows of x [tokens, values] at their slots [tokens, k]: [tokens k,
    values]; the rows of pairs without an expert are zeros."""
    if stream is not None:
        with _lend(stream, x, slots):
            return dispatch(x, slots)
    if _wants_grad(x):
        return _Dispatch.apply(x, slots)
    dev = _device(x, "x")
    stride = _row_stride(x, "x")
    T, H = x.shape
    sp = _slots(slots, T, dev)
    k = slots.shape[1]
    rows = x.new_empty((T * k, H))
    st = ops_lib().zc_dispatch(x.data_ptr(), _dtype(x, "x"), T, H, stride, sp, k, rows.data_ptr(),
                               _current_stream(dev.index))
    if st != ZC_OK:
        raise ZcError(st, "zc_dispatch")
    return rows


def combine(rows, slots, weights=None, base=None, stream=None):
    """base + the weighted sum of each token's rows: [tokens, values] in
    rows' type.  Without weights and base it is the gradient of dispatch."""
    if stream is not None:
        with _lend(stream, rows, slots, weights, base):
            return combine(rows, slots, weights, base)
    if _wants_grad(rows, weights, base):
        return _Combine.apply(rows, slots, weights, base)
    dev = _device(rows, "rows")
    T, k = slots.shape if slots.dim() == 2 else (-1, 0)
    sp = _slots(slots, T, dev)
    rp = _plain(rows, "rows", rows.dtype, dev)
    if rows.dim() != 2 or rows.shape[0] != T * k:
        raise ValueError("rows must have shape [tokens k, values]")
    H = rows.shape[1]
    wp = None if weights is None else _plain(weights, "weights", torch.float32, dev, slots.shape)
    bp, bs = None, 0
    if base is not None:
        bs = _row_stride(base, "base")
        if base.dtype is not rows.dtype or base.device != dev or base.shape != (T, H):
            raise ValueError("base must be [tokens, values] of rows' type and device")
        bp = base.data_ptr()
    out = rows.new_empty((T, H))
    st = ops_lib().zc_combine(rp, _dtype(rows, "rows"), T, H, sp, k, wp, bp, bs, out.data_ptr(),
                              _current_stream(dev.index))
    if st != ZC_OK:
        raise ZcError(st, "zc_combine")
    return out


def combine_grad(d_out, rows, slots, weights, stream=None):
    """Gradients of combine: (rows' [tokens k, values], weights' float32
    [tokens, k]) for d_out [tokens, values]."""
    if stream is not None:
        with _lend(stream, d_out, rows, slots, weights):
            return combine_grad(d_out, rows, slots, weights)
    dev = _device(d_out, "d_out")
    stride = _row_stride(d_out, "d_out")
    T, H = d_out.shape
    sp = _slots(slots, T, dev)
    k = slots.shape[1]
    rp = _plain(rows, "rows", d_out.dtype, dev, (T * k, H))
    wp = _plain(weights, "weights", torch.float32, dev, slots.shape)
    d_rows = d_out.new_empty((T * k, H))
    d_weights = weights.new_empty((T, k))
    st = ops_lib().zc_combine_grad(d_out.data_ptr(), _dtype(d_out, "d_out"), T, H, stride, rp, sp,
                                   k, wp, d_rows.data_ptr(), d_weights.data_ptr(),
                                   _current_stream(dev.index))
    if st != ZC_OK:
        raise ZcError(st, "zc_combine_grad")
    return d_rows, d_weights


def _list_of(tensors, name, types, count=None):
    """Checks a list of contiguous tensors of one type on one GPU.  The list
    returned holds the memory they have now: where a tensor's .data is given
    other memory later, the address that the library has been given stays
    good.  (Detached tensors share their version counters.)"""
    ts = [t.detach() for t in tensors]
    if count is not None and len(ts) != count:
        raise ValueError("%s has %d tensors for %d parameters" % (name, len(ts), count))
    for t in ts:
        if t.dtype is not ts[0].dtype or t.dtype not in types:
            raise ValueError("%s must all be of one type of %s" % (name, [str(d) for d in types]))
        if t.device != ts[0].device or not t.is_contiguous():
            raise ValueError("%s must be contiguous and on one device" % name)
    if ts:
        _device(ts[0], name)
    return ts


class TensorList:
    """Gradients whose norm is taken: contiguous tensors of one type (bfloat16
    or float32), checked and laid out for the library once.  The memory they
    have then is kept alive and is what every call reads: where a step makes
    its gradients anew (zero_grad's default), so is the list (2 us and 0.9 us a
    tensor)."""

    def __init__(self, tensors):
        self.tensors = _list_of(tensors, "tensors", (torch.bfloat16, torch.float32))
        self.count = len(self.tensors)
        self.dtype = _DTYPES[self.tensors[0].dtype] if self.tensors else ZC_F32
        self.device = (self.tensors[0].device if self.tensors
                       else torch.device("cuda", torch.cuda.current_device()))
        entries = [(t.data_ptr(), t.numel()) for t in self.tensors]
        self.array = (Tensor * max(self.count, 1))(*entries)
        self.ws_bytes = int(ops_lib().zc_grad_norm_workspace_bytes(self.array, self.count,
                                                                   self.dtype))


def grad_norm(grads, max_norm=0.0, stream=None):
    """float32 [2] on the GPU: the norm of all values of grads (a TensorList,
    or tensors), and the factor that clips it to max_norm (1 if that is not
    positive; NaN, which makes adamw skip the step, if the norm is not
    finite)."""
    if stream is not None:
        kept = isinstance(grads, TensorList)
        grads = grads if kept else list(grads)
        with _lend(stream, *(() if kept else grads)):
            return grad_norm(grads, max_norm)
    g = grads if isinstance(grads, TensorList) else TensorList(grads)
    dev = _current_device(g.device)
    out = torch.empty(2, dtype=torch.float32, device=dev)
    ws = torch.empty(g.ws_bytes, dtype=torch.uint8, device=dev) if g.ws_bytes else None
    st = ops_lib().zc_grad_norm(g.array, g.count, g.dtype, max_norm, out.data_ptr(),
                                None if ws is None else ws.data_ptr(), g.ws_bytes,
                                _current_stream(dev.index))
    if st != ZC_OK:
        raise ZcError(st, "zc_grad_norm")
    return out


class AdamWTensors:
    """The tensors of an AdamW step, checked and laid out for the library once:
    params (bfloat16 or float32), grads (bfloat16 or float32), the states avg
    and sq (float32; or float8_e4m3fn with float32 scales per 256 values, sq
    holding square roots), and for bfloat16 params optionally float32 masters.
    The memory they have then is kept alive and is what every step reads and
    writes: keep gradients in place (zero_grad(set_to_none=False), or decode
    the summed gradient into them), or make the list anew each step (5 us and 4
    to 5 us a tensor)."""

    def __init__(self, params, grads, avg, sq, masters=None, avg_scales=None, sq_scales=None):
        two = (torch.bfloat16, torch.float32)
        params, masters = list(params), None if masters is None else list(masters)
        p = _list_of(params, "params", two)
        n = len(p)
        state = (torch.float32, torch.float8_e4m3fn)
        lists = [p, _list_of(grads, "grads", two, n), _list_of(avg, "avg", state, n),
                 _list_of(sq, "sq", state, n)]
        eight = n > 0 and lists[2][0].dtype is torch.float8_e4m3fn
        if n and lists[3][0].dtype is not lists[2][0].dtype:
            raise ValueError("avg and sq must be of one type")
        if masters is not None:
            if n and p[0].dtype is not torch.bfloat16:
                raise ValueError("masters go with bfloat16 params")
            lists.append(_list_of(masters, "masters", (torch.float32,), n))
        for ts in lists[1:]:
            for a, b in zip(p, ts):
                if a.numel() != b.numel() or a.device != b.device:
                    raise ValueError("a parameter's tensors must be of its size and on its device")
        if n and (eight != (avg_scales is not None) or eight != (sq_scales is not None)):
            raise ValueError("avg_scales and sq_scales go with float8_e4m3fn states")
        scales = []
        if eight:
            scales = [_list_of(avg_scales, "avg_scales", (torch.float32,), n),
                      _list_of(sq_scales, "sq_scales", (torch.float32,), n)]
            for ts in scales:
                for a, b in zip(p, ts):
                    if b.numel() != -(-a.numel() // ZC_STATE_BLOCK) or a.device != b.device:
                        raise ValueError("a tensor needs one scale per 256 values")
        self.tensors = lists + scales
        # the tensors whose version a step counts up: what autograd may have
        # saved, one of those that share a counter as views of one tensor
        counted = {id(t if t._base is None else t._base): t for t in params + (masters or [])}
        self.counted = list(counted.values())
        self.count = n
        self.array = (AdamWTensor * max(n, 1))()
        for i in range(n):
            at = [ts[i].data_ptr() for ts in lists]
            sc = [ts[i].data_ptr() for ts in scales] or [None, None]
            self.array[i] = AdamWTensor(at[0], at[4] if masters is not None else None, at[1], at[2],
                                        at[3], sc[0], sc[1], p[i].numel())
        code = _DTYPES
        self.param_dtype = code[p[0].dtype] if n else ZC_F32
        self.grad_dtype = code[lists[1][0].dtype] if n else ZC_F32
        self.state_dtype = ZC_E4M3 if eight else ZC_F32
        self.device = p[0].device if n else None


def adamw(tensors, step, lr, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, grad_scale=None,
          stream=None):
    """One AdamW step (number `step`, from 1) over an AdamWTensors, in place.
    grad_scale: float32 tensor of one value on the GPU, a factor on every
    gradient (grad_norm(...)[1:]); one that is not finite skips the step."""
    if stream is not None:
        with _lend(stream, grad_scale):
            return adamw(tensors, step, lr, betas, eps, weight_decay, grad_scale)
    if not tensors.count:
        return
    dev = _current_device(tensors.device)
    gp = None
    if grad_scale is not None:
        if grad_scale.numel() != 1:
            raise ValueError("grad_scale must be one value")
        gp = _plain(grad_scale, "grad_scale", torch.float32, dev)
    c = AdamWConfig(tensors.param_dtype, tensors.grad_dtype, tensors.state_dtype, 0, step, lr,
                    betas[0], betas[1], eps, weight_decay)
    st = ops_lib().zc_adamw(tensors.array, tensors.count, ct.byref(c), gp,
                            _current_stream(dev.index))
    if st != ZC_OK:
        raise ZcError(st, "zc_adamw")
    _count_version(tensors.counted)
