"""The hard selections beside the soft top-k: Python binding.

Routing of tokens to experts and back, with gradients:

    weights, chosen = route_forward(logits, k, bias, score="sigmoid", groups=8, top_groups=4)
    offsets, slot, order = dispatch_plan(chosen, experts)
    xs = dispatch_forward(x, slot, offsets)          # expert e's rows: xs[offsets[e]:offsets[e + 1]]
    y = combine_forward(ys, slot, weights)           # ys: the experts' outputs, in the rows of xs
    route / dispatch / combine                       # the same, differentiable

A cache that keeps the entries which received the most attention:

    out = cache_attend(q, k, v, lengths, account)    # adds each entry's weight to account
    kept, lengths = cache_evict(k, v, account, positions, lengths, keep, next_position=n, recent=256)

As in the rest of the package this only marshals arguments; the formulas and
what happens to masked, infinite and missing values stand in
``include/lapsum.h``.  Calls run on torch's current stream.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os

from . import EXPORTED, LapsumError, _check, _workspace, load_library

F32, BF16, F16 = 0, 1, 2
# bound by the first call: the package can be imported without torch
torch = None
_TYPES, _FUNCTIONS = {}, {}
_raw_stream = _current_device = None
# the native front (csrc/binding.cpp): it takes the calls whose arguments need no conversion and returns None for all
# others, which then go the way written out below.  Without the built file every call does.
_native = None
_NATIVE_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_binding.so")
_NATIVE_CALLS = ["route_forward", "route_backward", "dispatch_plan_workspace_bytes", "dispatch_plan",
                 "dispatch_forward", "dispatch_backward", "combine_forward", "combine_backward",
                 "cache_attend_workspace_bytes", "cache_attend", "cache_evict_workspace_bytes", "cache_evict"]
SCORES = {"softmax": 0, "sigmoid": 1}
MAX_EXPERTS, MAX_CHOICES, MAX_GROUPS = 1024, 32, 64


class RouteOptions(ctypes.Structure):
    _fields_ = [("k", ctypes.c_int32), ("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("top_groups", ctypes.c_int32), ("renormalise", ctypes.c_int32), ("scale", ctypes.c_float)]


class Cache(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32), ("width", ctypes.c_int32),
                ("batch", ctypes.c_int64), ("heads", ctypes.c_int64), ("capacity", ctypes.c_int64),
                ("k_stride_batch", ctypes.c_int64), ("k_stride_head", ctypes.c_int64),
                ("k_stride_entry", ctypes.c_int64), ("v_stride_batch", ctypes.c_int64),
                ("v_stride_head", ctypes.c_int64), ("v_stride_entry", ctypes.c_int64)]


def declare(lib):
    i32, i64, vp, size = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
    opt, cache = ctypes.POINTER(RouteOptions), ctypes.POINTER(Cache)
    for name, res, args in [
        ("route_forward", ctypes.c_int, [vp, i32, i64, i64, i64, vp, opt, vp, vp, vp]),
        ("route_backward", ctypes.c_int, [vp, vp, i32, i64, i64, i64, vp, opt, vp, vp]),
        ("dispatch_plan_workspace_bytes", size, [i64, i64, i64]),
        ("dispatch_plan", ctypes.c_int, [vp, i64, i64, i64, vp, vp, vp, vp, size, vp]),
        ("dispatch_forward", ctypes.c_int, [vp, i32, i64, i64, i64, i64, vp, vp, i64, vp, vp]),
        ("dispatch_backward", ctypes.c_int, [vp, i32, i64, i64, i64, vp, vp, vp]),
        ("combine_forward", ctypes.c_int, [vp, i32, i64, i64, i64, vp, vp, vp, vp]),
        ("combine_backward", ctypes.c_int, [vp, i64, vp, i32, i64, i64, i64, vp, vp, vp, i64, vp, vp, vp]),
        ("cache_attend_workspace_bytes", size, [cache, i64, i64, i32]),
        ("cache_attend", ctypes.c_int, [vp, cache, vp, i64, i64, ctypes.c_float, vp, vp, vp, vp, size, vp]),
        ("cache_evict_workspace_bytes", size, [cache, i64]),
        ("cache_evict", ctypes.c_int, [cache, vp, vp, vp, i64, vp, i32, i32, vp, vp, vp, vp, vp, size, vp]),
    ]:
        f = getattr(lib, "lapsum_" + name)
        f.restype, f.argtypes = res, args


def _bind():
    global torch, _raw_stream, _current_device, _native
    import torch as t
    lib = load_library()
    _FUNCTIONS.update({name: getattr(lib, name) for name in EXPORTED})
    _TYPES.update({t.float32: F32, t.bfloat16: BF16, t.float16: F16})
    # torch's raw reader of the current stream takes 0.1 us, its stream object 1.9 us
    raw = getattr(t._C, "_cuda_getCurrentRawStream", None)
    _raw_stream = raw if raw is not None else (lambda index: t.cuda.current_stream(index).cuda_stream)
    _current_device = getattr(t._C, "_cuda_getDevice", None) or t.cuda.current_device
    torch = t
    if os.path.exists(_NATIVE_PATH):
        spec = importlib.util.spec_from_file_location(__package__ + "._binding", _NATIVE_PATH)
        native = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(native)
        native.bind(*[ctypes.cast(getattr(lib, "lapsum_" + name), ctypes.c_void_p).value for name in _NATIVE_CALLS])
        native.on_failure(_check)
        _native = native


# ----------------------------------------------------------------- checks
def _int32(x, name):
    x = int(x)
    if not -2 ** 31 <= x < 2 ** 31:
        raise LapsumError(f"{name} must be a 32-bit integer")
    return x


def _size(x, name, most):
    """A size that arrays are made by: checked before they are."""
    x = int(x)
    if not 1 <= x <= most:
        raise LapsumError(f"{name} must be 1 to {most}")
    return x


def _dtype(x, name, only=None):
    code = _TYPES.get(x.dtype)
    if code is None or (only is not None and code not in only):
        kinds = "bfloat16 or float16" if only else "float32, bfloat16 or float16"
        raise LapsumError(f"{name} must be {kinds}")
    return code


def _gpu(x, name, dim=None, dev=None):
    """A GPU tensor (of `dim` dimensions, on `dev`).  The first check of every entry point."""
    if torch is None:
        _bind()
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise LapsumError(f"{name} must be a GPU tensor (no CPU path exists)")
    if dim is not None and x.dim() != dim:
        raise LapsumError(f"{name} must have {dim} dimensions")
    if dev is not None and x.device != dev:
        raise LapsumError(f"{name} must be on {dev}")
    return x


def _array(x, name, dtype, shape, dev):
    """A contiguous device tensor of exactly this type and shape."""
    if not isinstance(x, torch.Tensor) or x.device != dev:
        _gpu(x, name, None, dev)
    if x.dtype != dtype or x.shape != shape:
        raise LapsumError(f"{name} must be {dtype} {list(shape)}")
    return x if x.is_contiguous() else x.contiguous()


def _out(x, name, dtype, shape, dev):
    """An output: the caller's tensor (used as it is, so it must be contiguous), or a new one."""
    if x is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    if not isinstance(x, torch.Tensor) or x.device != dev:
        _gpu(x, name, None, dev)
    if x.dtype != dtype or x.shape != shape or not x.is_contiguous():
        raise LapsumError(f"{name} must be contiguous {dtype} {list(shape)}")
    return x


def _written(*tensors):
    """Tensors of the caller that a call has written: autograd learns of it, as of any change in place."""
    for x in tensors:
        if x is not None and not x.is_inference():
            torch.autograd.graph.increment_version(x)


def _rows(x, name):
    """[tokens, n] with contiguous rows (any distance between them): (x, tokens, n, stride)."""
    tokens, n = x.shape
    stride, inner = x.stride()
    if (inner != 1 and n > 1) or (stride < n and tokens > 1):
        x, stride = x.contiguous(), n
    return x, tokens, n, (stride if tokens > 1 else n)


def _call(dev, name, *args):
    """A library call on a device's current stream (every entry point takes the stream last)."""
    f = _FUNCTIONS[name]
    index = dev.index
    if index == _current_device():
        rc = f(*args, _raw_stream(index))
    else:
        with torch.cuda.device(dev):
            rc = f(*args, _raw_stream(index))
    if rc:
        _check(rc, name)


# ---------------------------------------------------------------- routing
@functools.lru_cache(maxsize=256)
def _route_options(k, score, groups, top_groups, renormalise, scale):
    if score not in SCORES:
        raise LapsumError(f"score must be one of {sorted(SCORES)}")
    return RouteOptions(_int32(k, "k"), SCORES[score], _int32(groups, "groups"),
                        _int32(groups if top_groups is None else top_groups, "top_groups"), int(bool(renormalise)),
                        scale)


def route_forward(logits, k, bias=None, *, score="softmax", groups=1, top_groups=None, renormalise=True, scale=1.0,
                  out=None):
    """weights fp32 [tokens, k] and chosen int32 [tokens, k] for a router's logits [tokens, experts].

    The k largest of score + bias are chosen, in descending order (ties to the
    lowest index), among the experts of the top_groups best groups (all groups
    by default); the weights are the chosen scores (without the bias), divided
    by their sum if renormalise, times scale.  A slot without an available
    expert holds -1 and weight 0.  out: (weights, chosen) to write into."""
    if _native is not None and out is None:
        done = _native.route_forward(logits, bias, k, SCORES.get(score, -1), groups, top_groups, renormalise, scale)
        if done is not None:
            return done
    code = _dtype(_gpu(logits, "logits", 2), "logits")
    x, tokens, experts, stride = _rows(logits, "logits")
    dev = x.device
    opt = _route_options(_size(k, "k", min(experts, MAX_CHOICES)), score, int(groups), top_groups, renormalise, float(scale))
    if bias is not None:
        bias = _array(bias, "bias", torch.float32, (experts,), dev)
    weights = _out(None if out is None else out[0], "weights", torch.float32, (tokens, opt.k), dev)
    chosen = _out(None if out is None else out[1], "chosen", torch.int32, (tokens, opt.k), dev)
    if tokens == 0:
        return weights, chosen
    _call(dev, "lapsum_route_forward", x.data_ptr(), code, tokens, experts, stride,
          None if bias is None else bias.data_ptr(), opt, weights.data_ptr(), chosen.data_ptr())
    if out is not None:
        _written(*out)
    return weights, chosen


def route_backward(dweights, logits, chosen, *, score="softmax", renormalise=True, scale=1.0, out=None):
    """dlogits [tokens, experts], of the logits' type: the gradient of the weights, the choice held fixed
    (score, renormalise and scale as in the forward)."""
    if _native is not None and out is None:
        done = _native.route_backward(dweights, logits, chosen, SCORES.get(score, -1), renormalise, scale)
        if done is not None:
            return done
    code = _dtype(_gpu(logits, "logits", 2), "logits")
    x, tokens, experts, stride = _rows(logits, "logits")
    dev = x.device
    chosen = _array(_gpu(chosen, "chosen", 2), "chosen", torch.int32, (tokens, chosen.shape[1]), dev)
    dweights = _array(dweights, "dweights", torch.float32, chosen.shape, dev)
    opt = _route_options(chosen.shape[1], score, 1, 1, renormalise, float(scale))
    dlogits = _out(out, "dlogits", logits.dtype, (tokens, experts), dev)
    if tokens == 0:
        return dlogits
    _call(dev, "lapsum_route_backward", dweights.data_ptr(), x.data_ptr(), code, tokens, experts, stride,
          chosen.data_ptr(), opt, dlogits.data_ptr())
    _written(out)
    return dlogits


def route(logits, k, bias=None, *, score="softmax", groups=1, top_groups=None, renormalise=True, scale=1.0):
    """Differentiable route_forward: the weights' gradient reaches the logits.  The choice is not differentiable, so
    the bias, which takes part in nothing else, gets no gradient."""
    _gpu(logits, "logits", 2)
    if bias is not None and getattr(bias, "requires_grad", False):
        bias = bias.detach()  # or weights that cannot have a gradient would ask for one
    return _differentiable()[0].apply(logits, k, bias, score, groups, top_groups, renormalise, scale)


# --------------------------------------------------------------- dispatch
@functools.lru_cache(maxsize=1024)
def _plan_bytes(tokens, k, experts):
    return int(load_library().lapsum_dispatch_plan_workspace_bytes(tokens, k, experts))


def dispatch_plan(chosen, experts):
    """The expert order of the (token, choice) pairs of chosen [tokens, k]:
    offsets int32 [experts + 1] (expert e's rows are offsets[e]:offsets[e + 1]), slot int32 [tokens, k] (a pair's row,
    -1 for entries that name no expert) and order int32 [tokens * k] (the pair t * k + j of a row, -1 behind the last)."""
    if _native is not None:
        done = _native.dispatch_plan(chosen, experts)
        if done is not None:
            return done
    _gpu(chosen, "chosen", 2)
    (tokens, k), dev, experts = chosen.shape, chosen.device, _size(experts, "experts", MAX_EXPERTS)
    chosen = _array(chosen, "chosen", torch.int32, (tokens, k), dev)
    if tokens * k == 0:
        return (torch.zeros(experts + 1, dtype=torch.int32, device=dev), torch.empty_like(chosen),
                torch.empty(0, dtype=torch.int32, device=dev))
    slot = torch.empty_like(chosen)
    order = torch.empty(tokens * k, dtype=torch.int32, device=dev)
    offsets = torch.empty(experts + 1, dtype=torch.int32, device=dev)
    ws, wptr, wlen = _workspace(_plan_bytes(tokens, k, experts), dev)
    _call(dev, "lapsum_dispatch_plan", chosen.data_ptr(), tokens, k, experts, offsets.data_ptr(), slot.data_ptr(),
          order.data_ptr(), wptr, wlen)
    del ws  # back to the pool, ordered after this call on its stream
    return offsets, slot, order


def _slot_of(slot, dev, tokens=None):
    """slot as a contiguous int32 [tokens, k] on dev: (slot, tokens, k)."""
    if not isinstance(slot, torch.Tensor) or slot.device != dev or slot.dim() != 2 or slot.dtype != torch.int32:
        _gpu(slot, "slot", 2, dev)
        raise LapsumError("slot must be torch.int32")
    n, k = slot.shape
    if tokens is not None and n != tokens:
        raise LapsumError(f"slot must have {tokens} rows")
    return (slot if slot.is_contiguous() else slot.contiguous()), n, k


def _offsets_of(offsets, dev):
    if not isinstance(offsets, torch.Tensor) or offsets.device != dev or offsets.dim() != 1 or \
            offsets.dtype != torch.int32:
        _gpu(offsets, "offsets", 1, dev)
        raise LapsumError("offsets must be torch.int32")
    return offsets if offsets.is_contiguous() else offsets.contiguous()


def dispatch_forward(x, slot, offsets, *, out=None):
    """xs [tokens * k, width]: token rows in expert order, xs[slot[t, j]] = x[t] (rows behind the last pair zero)."""
    if _native is not None and out is None:
        done = _native.dispatch_forward(x, slot, offsets)
        if done is not None:
            return done
    code = _dtype(_gpu(x, "x", 2), "x")
    x, tokens, width, stride = _rows(x, "x")
    dev = x.device
    slot, _, k = _slot_of(slot, dev, tokens)
    offsets = _offsets_of(offsets, dev)
    xs = _out(out, "xs", x.dtype, (tokens * k, width), dev)
    if xs.numel() == 0:
        return xs
    _call(dev, "lapsum_dispatch_forward", x.data_ptr(), code, tokens, k, width, stride, slot.data_ptr(),
          offsets.data_ptr(), offsets.numel() - 1, xs.data_ptr())
    _written(out)
    return xs


def dispatch_backward(dxs, slot, *, out=None):
    """dx [tokens, width]: the sum of each token's rows of dxs."""
    if _native is not None and out is None:
        done = _native.dispatch_backward(dxs, slot)
        if done is not None:
            return done
    code = _dtype(_gpu(dxs, "dxs", 2), "dxs")
    dev = dxs.device
    slot, tokens, k = _slot_of(slot, dev)
    width = dxs.shape[1]
    dxs = _array(dxs, "dxs", dxs.dtype, (tokens * k, width), dev)
    dx = _out(out, "dx", dxs.dtype, (tokens, width), dev)
    if dxs.numel() == 0:
        return dx.zero_()
    _call(dev, "lapsum_dispatch_backward", dxs.data_ptr(), code, tokens, k, width, slot.data_ptr(), dx.data_ptr())
    _written(out)
    return dx


def combine_forward(ys, slot, weights, *, out=None):
    """y [tokens, width]: y[t] = sum_j weights[t, j] ys[slot[t, j]]."""
    if _native is not None and out is None:
        done = _native.combine_forward(ys, slot, weights)
        if done is not None:
            return done
    code = _dtype(_gpu(ys, "ys", 2), "ys")
    dev = ys.device
    slot, tokens, k = _slot_of(slot, dev)
    width = ys.shape[1]
    ys = _array(ys, "ys", ys.dtype, (tokens * k, width), dev)
    weights = _array(weights, "weights", torch.float32, (tokens, k), dev)
    y = _out(out, "y", ys.dtype, (tokens, width), dev)
    if ys.numel() == 0:
        return y.zero_()
    _call(dev, "lapsum_combine_forward", ys.data_ptr(), code, tokens, k, width, slot.data_ptr(), weights.data_ptr(),
          y.data_ptr())
    _written(out)
    return y


def combine_backward(dy, ys, slot, weights, offsets, *, out=None):
    """dys [tokens * k, width] and dweights fp32 [tokens, k]: dys[slot] = w dy[t], dweights = <dy[t], ys[slot]>."""
    if _native is not None and out is None:
        done = _native.combine_backward(dy, ys, slot, weights, offsets)
        if done is not None:
            return done
    code = _dtype(_gpu(dy, "dy", 2), "dy")
    dy, tokens, width, stride = _rows(dy, "dy")
    dev = dy.device
    slot, _, k = _slot_of(slot, dev, tokens)
    offsets = _offsets_of(offsets, dev)
    ys = _array(ys, "ys", dy.dtype, (tokens * k, width), dev)
    weights = _array(weights, "weights", torch.float32, (tokens, k), dev)
    dys = _out(None if out is None else out[0], "dys", dy.dtype, (tokens * k, width), dev)
    dweights = _out(None if out is None else out[1], "dweights", torch.float32, (tokens, k), dev)
    if ys.numel() == 0:
        return dys, dweights.zero_()
    _call(dev, "lapsum_combine_backward", dy.data_ptr(), stride, ys.data_ptr(), code, tokens, k, width,
          slot.data_ptr(), weights.data_ptr(), offsets.data_ptr(), offsets.numel() - 1, dys.data_ptr(),
          dweights.data_ptr())
    if out is not None:
        _written(*out)
    return dys, dweights


def dispatch(x, slot, offsets):
    """Differentiable dispatch_forward."""
    _gpu(x, "x", 2)
    return _differentiable()[1].apply(x, slot, offsets)


def combine(ys, weights, slot, offsets):
    """Differentiable combine_forward: gradients reach the experts' outputs and the weights."""
    _gpu(ys, "ys", 2)
    return _differentiable()[2].apply(ys, weights, slot, offsets)


# ---------------------------------------------------------- differentiable
@functools.lru_cache(maxsize=None)
def _differentiable():
    """The autograd functions of route, dispatch and combine, made once torch is bound (a class made by each call takes
    longer than the call, and as a cycle keeps what it closes over until the collector runs)."""
    once = torch.autograd.function.once_differentiable

    class Route(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, k, bias, score, groups, top_groups, renormalise, scale):
            weights, chosen = route_forward(x, k, bias, score=score, groups=groups, top_groups=top_groups,
                                            renormalise=renormalise, scale=scale)
            ctx.save_for_backward(x, chosen)
            ctx.options = dict(score=score, renormalise=renormalise, scale=scale)
            ctx.mark_non_differentiable(chosen)
            return weights, chosen

        @staticmethod
        @once
        def backward(ctx, dweights, _):
            x, chosen = ctx.saved_tensors
            return (route_backward(dweights.contiguous(), x, chosen, **ctx.options), *[None] * 7)

    # slots and offsets are saved, so autograd notices if they are written again before the backward
    class Dispatch(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, slot, offsets):
            xs = dispatch_forward(x, slot, offsets)
            ctx.save_for_backward(slot)
            return xs

        @staticmethod
        @once
        def backward(ctx, dxs):
            slot, = ctx.saved_tensors
            return dispatch_backward(dxs.contiguous(), slot), None, None

    class Combine(torch.autograd.Function):
        @staticmethod
        def forward(ctx, ys, weights, slot, offsets):
            y = combine_forward(ys, slot, weights)
            ctx.save_for_backward(ys, weights, slot, offsets)
            return y

        @staticmethod
        @once
        def backward(ctx, dy):
            ys, weights, slot, offsets = ctx.saved_tensors
            return (*combine_backward(dy, ys, slot, weights, offsets), None, None)

    return Route, Dispatch, Combine


# ------------------------------------------------------------------ cache
@functools.lru_cache(maxsize=1024)
def _cache_shape(code, k_shape, k_strides, v_strides):
    """The layout of a cache (everything but its pointers)."""
    if k_strides[3] != 1 or v_strides[3] != 1:
        raise LapsumError("the entries of k and v must be contiguous (last stride 1)")
    batch, heads, capacity, width = k_shape
    return Cache(None, None, code, width, batch, heads, capacity, *k_strides[:3], *v_strides[:3])


def _cache_of(k, v):
    code = _dtype(_gpu(k, "k", 4), "k", (BF16, F16))
    _gpu(v, "v", 4, k.device)
    if v.dtype != k.dtype or v.shape != k.shape:
        raise LapsumError("k and v must have the same type and shape")
    cache = Cache.from_buffer_copy(_cache_shape(code, k.shape, k.stride(), v.stride()))
    cache.k, cache.v = k.data_ptr(), v.data_ptr()
    return cache


@functools.lru_cache(maxsize=1024)
def _attend_bytes(code, k_shape, news, q_heads, accounts):
    batch, heads, capacity, width = k_shape
    cache = Cache(None, None, code, width, batch, heads, capacity, 0, 0, 0, 0, 0, 0)
    return int(load_library().lapsum_cache_attend_workspace_bytes(cache, news, q_heads, accounts))


def cache_attend(q, k, v, lengths, account=None, *, scale=None, account_out=None, out=None):
    """out [batch, news, q_heads, width]: attention of the newest tokens q over a cache k, v
    [batch, heads, capacity, width] whose first lengths[b] entries are filled, the new tokens' own last (token i sees
    the entries up to lengths[b] - news + i).  account fp32 [batch, heads, capacity]: each entry's weight, summed over
    the new tokens and the query heads of its key head, is added to it, in place or into account_out.
    scale: 1/sqrt(width) by default.  No gradient: the results do not require one, whatever the arguments do."""
    if _native is not None and out is None:
        done = _native.cache_attend(q, k, v, lengths, account, scale, account_out)
        if done is not None:
            return done
    cache = _cache_of(k, v)
    dev = k.device
    _gpu(q, "q", 4, dev)
    batch, news, q_heads, width = q.shape
    if q.dtype != k.dtype or batch != k.shape[0] or width != k.shape[3]:
        raise LapsumError("q must be [batch, news, q_heads, width] of the cache's type")
    q = q.contiguous()
    lengths = _array(lengths, "lengths", torch.int32, (batch,), dev)
    given, out = out, _out(out, "out", q.dtype, q.shape, dev)
    if account is not None:
        if account_out is None:
            account_out = account  # written in place: not a copy of it
        else:
            account = _array(account, "account", torch.float32, k.shape[:3], dev)
        account_out = _out(account_out, "account", torch.float32, k.shape[:3], dev)
    elif account_out is not None:
        raise LapsumError("account_out needs an account")
    if q.numel() == 0:
        if account is not None and account_out is not account:  # nothing is added to what the entries have
            there = torch.arange(k.shape[2], device=dev) < lengths[:, None, None]
            account_out.copy_(torch.where(there, account, account_out))
        return out
    nbytes = _attend_bytes(cache.dtype, k.shape, news, q_heads, int(account is not None))
    ws, wptr, wlen = _workspace(nbytes, dev)
    _call(dev, "lapsum_cache_attend", q.data_ptr(), cache, lengths.data_ptr(), news, q_heads,
          width ** -0.5 if scale is None else float(scale), None if account is None else account.data_ptr(),
          None if account is None else account_out.data_ptr(), out.data_ptr(), wptr, wlen)
    _written(account_out, given)
    del ws
    return out


@functools.lru_cache(maxsize=1024)
def _evict_bytes(code, k_shape, keep):
    batch, heads, capacity, width = k_shape
    cache = Cache(None, None, code, width, batch, heads, capacity, 0, 0, 0, 0, 0, 0)
    return int(load_library().lapsum_cache_evict_workspace_bytes(cache, keep))


def cache_evict(k, v, account, positions, lengths, keep, *, next_position=None, sinks=0, recent=0, account_out=None,
                positions_out=None):
    """Brings every cache row down to `keep` entries: protected entries (position below sinks, or at least
    next_position[b] - recent where recent is not 0) stay first, then those of the highest account (ties: the lowest slot).  Survivors
    behind slot keep move into the holes before it, keys, values, accounts and positions; k and v are changed in
    place, account and positions too unless account_out and positions_out are given.

    Returns kept int32 [batch, heads, keep] (the slot each entry came from, -1 behind the last) and the new lengths
    (a new tensor)."""
    if _native is not None:
        done = _native.cache_evict(k, v, account, positions, lengths, keep, next_position, sinks, recent, account_out,
                                   positions_out)
        if done is not None:
            return done
    cache = _cache_of(k, v)
    dev, batch, keep = k.device, k.shape[0], _size(keep, "keep", k.shape[2])
    shape = k.shape[:3]
    # arrays that are written in place have to be usable as they are
    account = _out(account, "account", torch.float32, shape, dev) if account_out is None else _array(
        account, "account", torch.float32, shape, dev)
    positions = _out(positions, "positions", torch.int32, shape, dev) if positions_out is None else _array(
        positions, "positions", torch.int32, shape, dev)
    account_out = _out(account if account_out is None else account_out, "account_out", torch.float32, shape, dev)
    positions_out = _out(positions if positions_out is None else positions_out, "positions_out", torch.int32, shape,
                         dev)
    lengths = _array(lengths, "lengths", torch.int32, (batch,), dev)
    if next_position is not None:
        next_position = _array(next_position, "next_position", torch.int32, (batch,), dev)
    kept = torch.empty((*shape[:2], keep), dtype=torch.int32, device=dev)
    lengths_out = torch.empty_like(lengths)
    if shape[0] * shape[1] == 0:  # no cache
        return kept, lengths.clamp(0, keep)
    ws, wptr, wlen = _workspace(_evict_bytes(cache.dtype, k.shape, keep), dev)
    _call(dev, "lapsum_cache_evict", cache, account.data_ptr(), positions.data_ptr(), lengths.data_ptr(), keep,
          None if next_position is None else next_position.data_ptr(), _int32(sinks, "sinks"),
          _int32(recent, "recent"),
          account_out.data_ptr(), positions_out.data_ptr(), kept.data_ptr(), lengths_out.data_ptr(), wptr, wlen)
    _written(k, v, account_out, positions_out)
    del ws
    return kept, lengths_out
