"""Binding of the library's ordered selections: routing to experts with its
gradient, stable grouping by expert, accumulated attention weights and
eviction from a cache.

Like the rest of the package this is argument marshalling only: tensors'
pointers, strides and the current stream go to the C ABI (declared in
``include/ordmerge.h``), which validates and launches.  Outputs may be passed
in; those not passed are allocated.  om_route_topk's weights carry their
gradient; the other calls stand outside autograd: what they give has none.
"""
from __future__ import annotations

import functools
import struct

import torch
from torch.autograd import forward_ad

from . import CacheArray, _check, _lib, _stream

VALUE_TYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
SCORES = {"softmax": 0, "sigmoid": 1}


# The current stream's handle without building a Stream object, the device without a
# look whether CUDA is up (a tensor there says so) and the versions of several tensors
# at once, where this torch has the calls (3 us, and a few tenths each, less a call on
# the measured host).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raise_versions = getattr(torch._C, "_increment_version", torch.autograd.graph.increment_version)
_grad_enabled = torch.is_grad_enabled
_current_device, _cuda_ready = torch.cuda.current_device, torch.cuda.is_initialized


def _ptr(t):
    return t.data_ptr()  # NULL where there are no elements


def _empty(shape, dtype, device, stream):
    """New output, allocated for the stream that will write it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _no_tangents(names, tensors):
    """Refuses tensors that carry a forward-mode tangent: the library reads their values alone."""
    for i, t in enumerate(tensors):
        if t is not None and forward_ad.unpack_dual(t).tangent is not None:
            name = names.split()[min(i, names.count(" "))]
            raise ValueError(f"{name} carries a forward-mode tangent, for which the library has no derivative")


def _elsewhere(names, tensors):
    """Refuses the first of the tensors that is not on the current device."""
    device = _current_device() if _cuda_ready() else -2
    for i, t in enumerate(tensors):
        if t is not None and t.get_device() != device:
            name = names.split()[min(i, names.count(" "))]
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            raise ValueError(f"{name} is on {t.device}, but the current device is cuda:{torch.cuda.current_device()}")


def _launch_stream(stream, names, *tensors):
    """The handle of `stream`, or of the current one, on the current device,
    where every tensor (None: not given; the first is) has to be."""
    if forward_ad._current_level >= 0:  # in a dual_level, where tensors may have tangents
        _no_tangents(names, tensors)
    device = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            _elsewhere(names, tensors)
    if device < 0 or device != _get_device():
        _elsewhere(names, tensors)
    if stream is None and _raw_stream is not None:
        return _raw_stream(device)
    return _stream(stream)


def _written(*tensors):
    """Tells autograd that the library has written into these tensors (None: not given), which were handed in: a
    backward pass that saved one of them before refuses it then, as after any other operation in place."""
    given = [t for t in tensors if t is not None]
    if given:
        _raise_versions(given)


def _dense(t, name: str, shape, dtype):
    if t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} "
                         f"(got {t.dtype}, {tuple(t.shape)})")


def _value_type(t, name: str) -> int:
    if t.dtype not in VALUE_TYPES:
        raise ValueError(f"{name} must be float32, bfloat16 or float16 (got {t.dtype})")
    return VALUE_TYPES[t.dtype]


def _rows(t, name: str, dims: int):
    """Strides of a tensor of `dims` dimensions whose last one is contiguous."""
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions (got {t.dim()})")
    strides = t.stride()
    if t.shape[-1] > 1 and strides[-1] != 1:
        raise ValueError(f"the last dimension of {name} must be contiguous")
    return strides


def _score_code(score: str) -> int:
    if score not in SCORES:
        raise ValueError(f"score must be 'softmax' or 'sigmoid' (got {score!r})")
    return SCORES[score]


def _lengths(lengths, batch: int, name: str = "lengths"):
    if lengths is None:
        return None
    if lengths.dtype != torch.int32 or lengths.shape != (batch,) or not lengths.is_contiguous():
        _dense(lengths, name, (batch,), torch.int32)
    return lengths.data_ptr()


class _RouteWithGradient(torch.autograd.Function):
    """om_route_topk with om_route_topk_backward behind it.  The backward pass
    runs on the stream that autograd runs it on, the caller's at the forward
    call: who gives another `stream` joins the two before using the weights."""

    @staticmethod
    def forward(ctx, logits, top_k, options):
        # outputs handed in come as options: what an earlier call wrote into them is no part of this one
        ids, weights = om_route_topk(logits, top_k, **options)
        ctx.mark_non_differentiable(ids)
        ctx.save_for_backward(logits, ids)
        ctx.options = {name: options[name] for name in ("score", "renorm", "scale")}
        return ids, weights

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, _, grad_weights):
        logits, ids = ctx.saved_tensors
        return om_route_topk_backward(logits, ids, grad_weights.contiguous(), **ctx.options), None, None


def om_route_topk(logits, top_k: int, score: str = "softmax", bias=None, groups: int = 1, group_picks: int = 1,
                  group_best: int = 1, renorm: bool = False, scale: float = 1.0, ids=None, weights=None, stream=None):
    """(ids, weights) of the top_k experts of each row of logits [tokens,
    experts]: greatest score + bias first, ties to the lower index, from the
    group_picks groups whose group_best greatest sum highest; weights are the
    scores without the bias (divided by their sum with renorm) times scale.
    Masked experts (-inf or NaN) are never chosen; id -1, weight 0 fill up.
    Where logits require a gradient the weights carry it to them (the choice
    is constant, the bias has none)."""
    if logits.requires_grad and torch.is_grad_enabled():
        options = dict(score=score, bias=bias, groups=groups, group_picks=group_picks, group_best=group_best,
                       renorm=renorm, scale=scale, ids=ids, weights=weights, stream=stream)
        return _RouteWithGradient.apply(logits, top_k, options)
    row_stride = _rows(logits, "logits", 2)[0]
    tokens, experts = logits.shape
    given = ids, weights
    if bias is not None:
        _dense(bias, "bias", (experts,), torch.float32)
    if ids is None:
        ids = _empty((tokens, top_k), torch.int32, logits.device, stream)
    if weights is None:
        weights = _empty((tokens, top_k), torch.float32, logits.device, stream)
    _dense(ids, "ids", (tokens, top_k), torch.int32)
    _dense(weights, "weights", (tokens, top_k), torch.float32)
    handle = _launch_stream(stream, "logits bias ids weights", logits, bias, ids, weights)
    _check(
        _lib.om_route_topk(_value_type(logits, "logits"), _ptr(logits), tokens, experts, row_stride,
                           None if bias is None else bias.data_ptr(), _score_code(score), groups, group_picks,
                           group_best, top_k, 1 if renorm else 0, scale, _ptr(ids), _ptr(weights), handle),
        "om_route_topk",
    )
    _written(*given)
    return ids, weights


def om_route_topk_backward(logits, ids, grad_weights, score: str = "softmax", renorm: bool = False,
                           scale: float = 1.0, grad_logits=None, stream=None):
    """Gradient of om_route_topk's weights by the logits (contiguous, in
    their dtype), from its ids and the weights' gradient (float32)."""
    row_stride = _rows(logits, "logits", 2)[0]
    tokens, experts = logits.shape
    if ids.dim() != 2:
        raise ValueError("ids must have 2 dimensions")
    top_k = ids.shape[1]
    _dense(ids, "ids", (tokens, top_k), torch.int32)
    _dense(grad_weights, "grad_weights", (tokens, top_k), torch.float32)
    given = grad_logits
    if grad_logits is None:
        grad_logits = _empty((tokens, experts), logits.dtype, logits.device, stream)
    _dense(grad_logits, "grad_logits", (tokens, experts), logits.dtype)
    handle = _launch_stream(stream, "logits ids grad_weights grad_logits", logits, ids, grad_weights, grad_logits)
    _check(
        _lib.om_route_topk_backward(_value_type(logits, "logits"), _ptr(logits), tokens, experts, row_stride,
                                    _ptr(ids), _ptr(grad_weights), _score_code(score), top_k, 1 if renorm else 0,
                                    scale, _ptr(grad_logits), handle),
        "om_route_topk_backward",
    )
    _written(given)
    return grad_logits


def om_group_by_id(ids, groups: int, offsets=None, order=None, place=None, stream=None):
    """(offsets, order, place) of the stable grouping of ids (int32, any
    shape, contiguous; taken flat): order[offsets[g]:offsets[g + 1]] are the
    slots with id g in rising order, slots with an id outside [0, groups)
    come last, and order[place[i]] == i."""
    if ids.dtype != torch.int32 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int32 tensor")
    n = ids.numel()
    given = offsets, order, place
    if offsets is None:
        offsets = _empty((groups + 1,), torch.int32, ids.device, stream)
    if order is None:
        order = _empty((n,), torch.int32, ids.device, stream)
    if place is None:
        place = _empty((n,), torch.int32, ids.device, stream)
    _dense(offsets, "offsets", (groups + 1,), torch.int32)
    _dense(order, "order", (n,), torch.int32)
    _dense(place, "place", (n,), torch.int32)
    handle = _launch_stream(stream, "ids offsets order place", ids, offsets, order, place)
    _check(_lib.om_group_by_id(_ptr(ids), n, groups, _ptr(offsets), _ptr(order), _ptr(place), handle),
           "om_group_by_id")
    _written(*given)
    return offsets, order, place


def om_accumulate_weights(weights, score=None, lengths=None, decay: float = 1.0, kv_heads: int | None = None,
                          out=None, stream=None):
    """decay * score + the attention weights [batch, q_heads, queries, length]
    summed over the queries and the query heads of each cache head, as
    [batch, kv_heads, length] float32; zero past lengths (int32 [batch]).
    score None starts from zero (give kv_heads then); out may be score."""
    w_batch, w_head, w_query, _ = _rows(weights, "weights", 4)
    batch, q_heads, queries, length = weights.shape
    s_batch = s_head = 0
    if score is not None:
        s_batch, s_head, _ = _rows(score, "score", 3)
        kv_heads = score.shape[1] if kv_heads is None else kv_heads
        if score.dtype != torch.float32 or tuple(score.shape) != (batch, kv_heads, length):
            raise ValueError(f"score must be float32 of shape {(batch, kv_heads, length)}")
    if kv_heads is None:
        raise ValueError("kv_heads is needed without a score")
    given = out
    if out is None:
        out = _empty((batch, kv_heads, length), torch.float32, weights.device, stream)
    o_batch, o_head, _ = _rows(out, "out", 3)
    if out.dtype != torch.float32 or tuple(out.shape) != (batch, kv_heads, length):
        raise ValueError(f"out must be float32 of shape {(batch, kv_heads, length)}")
    length_ptr = _lengths(lengths, batch)
    handle = _launch_stream(stream, "weights score lengths out", weights, score, lengths, out)
    _check(
        _lib.om_accumulate_weights(_value_type(weights, "weights"), _ptr(weights), batch, q_heads, kv_heads, queries,
                                   length, w_batch, w_head, w_query, None if score is None else _ptr(score), s_batch,
                                   s_head, length_ptr, decay, _ptr(out), o_batch, o_head, handle),
        "om_accumulate_weights",
    )
    _written(given)
    return out


def om_evict_select(score, budget: int, first: int = 0, last: int = 0, lengths=None, keep=None, kept=None,
                    stream=None):
    """(keep, kept): the indices, rising and then -1, of the entries that each
    row of score [batch, heads, length] (float32) keeps when cut to budget
    (the first `first`, the last `last`, the greatest scores between, ties to
    the lower index), and min(length, budget) per sequence."""
    s_batch, s_head, _ = _rows(score, "score", 3)
    if score.dtype != torch.float32:
        raise ValueError(f"score must be float32 (got {score.dtype})")
    batch, heads, length = score.shape
    given = keep, kept
    if keep is None:
        keep = _empty((batch, heads, budget), torch.int32, score.device, stream)
    if kept is None:
        kept = _empty((batch,), torch.int32, score.device, stream)
    _dense(keep, "keep", (batch, heads, budget), torch.int32)
    _dense(kept, "kept", (batch,), torch.int32)
    length_ptr = _lengths(lengths, batch)
    handle = _launch_stream(stream, "score lengths keep kept", score, lengths, keep, kept)
    _check(
        _lib.om_evict_select(_ptr(score), batch, heads, length, s_batch, s_head, length_ptr, budget, first, last,
                             _ptr(keep), _ptr(kept), handle),
        "om_evict_select",
    )
    _written(*given)
    return keep, kept


def _cache_entry(shape, strides, name: str, batch: int, heads: int) -> int:
    """Elements of one entry of a cache array [batch, heads, entries, ...] whose entries are contiguous."""
    if len(shape) < 3 or shape[0] != batch or shape[1] != heads:
        raise ValueError(f"{name} must be [batch, heads, entries, ...] with batch {batch} and heads {heads}")
    inner = 1
    for d in range(len(shape) - 1, 2, -1):
        if shape[d] != 1 and strides[d] != inner:
            raise ValueError(f"the entries of {name} must be contiguous")
        inner *= shape[d]
    return inner


@functools.lru_cache(maxsize=256)
def _gather_geometry(keep_shape, *arrays):
    """Checks the arrays' shapes and strides (each array: element size, then
    shape and strides of source and output) and returns, as om_cache_array
    wants them, every array's bytes per entry and strides in bytes, and the
    number of entries.  Of the shapes alone, so it is kept from call to call."""
    batch, heads, budget = keep_shape
    words, length = [], None
    for size, src_shape, src_strides, dst_shape, dst_strides in zip(*[iter(arrays)] * 5):
        inner = _cache_entry(src_shape, src_strides, "array", batch, heads)
        want = (*keep_shape, *src_shape[3:])
        if dst_shape != want or _cache_entry(dst_shape, dst_strides, "out", batch, heads) != inner:
            raise ValueError(f"out must have shape {want} (got {tuple(dst_shape)})")
        if length is not None and src_shape[2] != length:
            raise ValueError("the arrays must have as many entries each")
        length = src_shape[2]
        words.append((inner * size, *(s * size for s in src_strides[:3]), *(s * size for s in dst_strides[:3])))
    return words, length, struct.Struct(f"{len(CacheArray._fields_) * len(words)}q").pack


def om_evict_gather(keep, arrays, out=None, stream=None):
    """The cache arrays (each [batch, heads, entries, ...], any element type,
    entries contiguous) gathered to keep [batch, heads, budget]: entry j
    becomes entry keep[j], zero where keep is -1.  Returns new arrays, or
    `out`, which must share no byte with the inputs, or is their first budget entries
    (out[i] = arrays[i][:, :, :budget]: in place, for rising keep).  One launch
    moves all of them."""
    arrays = tuple(arrays)
    shape = keep.shape
    if len(shape) != 3:
        raise ValueError("keep must have 3 dimensions")
    _dense(keep, "keep", shape, torch.int32)
    if not arrays:
        raise ValueError("no arrays to gather")
    handed = out is not None
    out = tuple(out) if handed else tuple(_empty((*shape, *t.shape[3:]), t.dtype, t.device, stream) for t in arrays)
    if len(out) != len(arrays):
        raise ValueError("out must hold one tensor for each array")
    handle = _launch_stream(stream, "keep array", keep, *arrays, *out)
    key = []
    for src, dst in zip(arrays, out):
        if dst.dtype != src.dtype:
            raise ValueError(f"out must be {src.dtype} (got {dst.dtype})")
        key += (src.element_size(), src.shape, src.stride(), dst.shape, dst.stride())
    words, length, pack = _gather_geometry(shape, *key)
    table = []
    for src, dst, fixed in zip(arrays, out, words):
        table += (src.data_ptr(), dst.data_ptr(), *fixed)
    # om_cache_array, whose fields are 64-bit words in this order
    _check(_lib.om_evict_gather(_ptr(keep), *shape, length, pack(*table), len(arrays), handle), "om_evict_gather")
    if handed:
        _written(*out)
    return out
