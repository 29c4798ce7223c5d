"""Binding of the calls around the ordered selections when a model decodes:
beam search with its states, embedding rows with their gradient, and the routed
experts' layer for a few tokens.

Argument marshalling only, as in ``selection.py``: tensors' pointers, strides and
the current stream go to the C ABI (declared in ``include/ordmerge.h``), which
validates and launches.  Outputs may be passed in; those not passed are allocated.
om_embed_lookup's rows carry their gradient to the table.  om_beam_select's choice
is a constant: what it gives has none.  The other calls have no gradient, and while
autograd records they refuse tensors that require one (under torch.no_grad(), or
detached, they take them).
"""
from __future__ import annotations

import functools
import struct

import torch

from . import BeamArray, _check, _lib
from .selection import (VALUE_TYPES, _dense, _empty, _grad_enabled, _launch_stream, _lengths, _rows, _value_type,
                        _written)

ACTIVATIONS = {"silu": 0, "gelu": 1, "relu": 2}
ID_BYTES = {torch.int32: 4, torch.int64: 8}


def _no_gradient(call: str, *tensors):
    """Refuses tensors whose gradient would end in `call` without a word, or be that of values it has moved."""
    if _grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                raise ValueError(f"{call} has no gradient: use torch.no_grad(), or detached tensors")


# ------------------------------------------------------------ beam search --

def om_beam_select(logits, top: int, scores=None, finished=None, end_id: int = 0, out_scores=None, parents=None,
                   tokens=None, stream=None):
    """(scores, parents, tokens), each [batch, top]: the greatest scores[b, i]
    + log_softmax(logits[b, i])[v] of each sequence of logits [batch, beams,
    vocab], greatest first, ties to the lower beam; within a beam by logit, ties
    to the lower token.
    scores (float32 [batch, beams]; None: zeros) are the beams' cumulative log
    probabilities; a finished beam (bool [batch, beams]) goes on with end_id
    alone, at its score.  Logits of -inf or NaN are never chosen; score -inf and
    -1 fill up."""
    b_stride, n_stride, _ = _rows(logits, "logits", 3)
    batch, beams, vocab = logits.shape
    if scores is not None:
        _dense(scores, "scores", (batch, beams), torch.float32)
    if finished is not None:
        _dense(finished, "finished", (batch, beams), torch.bool)
    given = out_scores, parents, tokens
    if out_scores is not None and out_scores.requires_grad:
        _no_gradient("what is written into out_scores", out_scores)
    if out_scores is None:
        out_scores = _empty((batch, top), torch.float32, logits.device, stream)
    if parents is None:
        parents = _empty((batch, top), torch.int32, logits.device, stream)
    if tokens is None:
        tokens = _empty((batch, top), torch.int32, logits.device, stream)
    _dense(out_scores, "out_scores", (batch, top), torch.float32)
    _dense(parents, "parents", (batch, top), torch.int32)
    _dense(tokens, "tokens", (batch, top), torch.int32)
    handle = _launch_stream(stream, "logits scores finished out_scores parents tokens", logits, scores, finished,
                            out_scores, parents, tokens)
    _check(
        _lib.om_beam_select(_value_type(logits, "logits"), logits.data_ptr(), batch, beams, vocab, b_stride, n_stride,
                            None if scores is None else scores.data_ptr(),
                            None if finished is None else finished.data_ptr(), end_id, top, out_scores.data_ptr(),
                            parents.data_ptr(), tokens.data_ptr(), handle),
        "om_beam_select",
    )
    _written(*given)
    return out_scores, parents, tokens


def _state_entry(shape, strides, name: str, batch: int, beams: int) -> int:
    """Elements of one entry of a state array [batch, beams, heads, entries, ...] whose entries are contiguous."""
    if len(shape) < 4 or shape[0] != batch or shape[1] != beams:
        raise ValueError(f"{name} must be [batch, beams, heads, entries, ...] with batch {batch} and beams {beams}")
    inner = 1
    for d in range(len(shape) - 1, 3, -1):
        if shape[d] != 1 and strides[d] != inner:
            raise ValueError(f"the entries of {name} must be contiguous")
        inner *= shape[d]
    return inner


@functools.lru_cache(maxsize=256)
def _state_geometry(parents_shape, in_place, *arrays):
    """Checks the arrays' shapes and strides (each array: element type, shape and
    strides, then those of the output if there is another) and returns, as
    om_beam_array wants them, every array's bytes per entry and strides in bytes,
    then heads, entries and a packer.  Of the shapes alone, so it is kept from call
    to call."""
    batch, beams = parents_shape
    words, common, step = [], None, 3 if in_place else 5
    for i in range(0, len(arrays), step):
        dtype, shape, src_strides = arrays[i:i + 3]
        size = dtype.itemsize
        dst_shape, dst_strides = (shape, src_strides) if in_place else arrays[i + 3:i + 5]
        inner = _state_entry(shape, src_strides, "array", batch, beams)
        if dst_shape != shape or _state_entry(dst_shape, dst_strides, "out", batch, beams) != inner:
            raise ValueError(f"out must have shape {tuple(shape)} (got {tuple(dst_shape)})")
        if common is not None and shape[2:4] != common:
            raise ValueError("the arrays must have as many heads and entries each")
        common = shape[2:4]
        words.append((inner * size, *(s * size for s in src_strides[:4]), *(s * size for s in dst_strides[:4])))
    return words, *common, struct.Struct(f"{len(BeamArray._fields_) * len(words)}q").pack


def om_beam_gather(parents, arrays, starts=None, lengths=None, out=None, stream=None):
    """The states (each [batch, beams, heads, entries, ...], any element type,
    entries contiguous) moved to the beams that go on: beam j's entries from
    starts[b] (int32 [batch]; None: 0) to lengths[b] (None: all) become those of
    beam parents[b, j] (int32 [batch, beams]); where parents is outside [0, beams),
    and other entries, stay as they are.  In place, or into `out` (arrays of the
    same shapes that share no byte with the states), which it returns.  One
    launch moves all of them."""
    arrays = tuple(arrays)
    shape = parents.shape
    if len(shape) != 2:
        raise ValueError("parents must have 2 dimensions")
    if parents.dtype != torch.int32 or not parents.is_contiguous():
        raise ValueError(f"parents must be a contiguous {torch.int32} tensor (got {parents.dtype})")
    if not arrays:
        raise ValueError("no arrays to move")
    in_place = out is None
    out = arrays if in_place else tuple(out)
    if len(out) != len(arrays):
        raise ValueError("out must hold one tensor for each array")
    start_ptr = _lengths(starts, shape[0], "starts")
    length_ptr = _lengths(lengths, shape[0])
    key = []
    if in_place:
        for t in arrays:
            if t.requires_grad:
                _no_gradient("om_beam_gather", t)
            key += (t.dtype, t.shape, t.stride())
    else:
        for src, dst in zip(arrays, out):
            if src.requires_grad or dst.requires_grad:
                _no_gradient("om_beam_gather", src, dst)
            dtype = src.dtype
            if dst.dtype != dtype:
                raise ValueError(f"out must be {dtype} (got {dst.dtype})")
            key += (dtype, src.shape, src.stride(), dst.shape, dst.stride())
    tensors = arrays if in_place else arrays + out
    handle = _launch_stream(stream, "parents starts lengths array", parents, starts, lengths, *tensors)
    words, heads, entries, pack = _state_geometry(shape, in_place, *key)
    table = []
    for src, dst, fixed in zip(arrays, out, words):
        table += (src.data_ptr(), dst.data_ptr(), *fixed)
    # om_beam_array, whose fields are 64-bit words in this order
    _check(_lib.om_beam_gather(parents.data_ptr(), *shape, heads, entries, start_ptr, length_ptr, pack(*table),
                               len(arrays), handle), "om_beam_gather")
    _written(*out)
    return out


# -------------------------------------------------------------- embedding --

def _ids(ids):
    if ids.dtype not in ID_BYTES or not ids.is_contiguous():
        raise ValueError(f"ids must be a contiguous int32 or int64 tensor (got {ids.dtype})")
    return ID_BYTES[ids.dtype]


class _LookupWithGradient(torch.autograd.Function):
    """om_embed_lookup with om_embed_lookup_backward behind it, on the stream that
    autograd runs it on, the caller's at the forward call."""

    @staticmethod
    def forward(ctx, ids, table, scale, stream):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale = table.shape[0], scale
        return om_embed_lookup(ids, table, scale, stream=stream)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad):
        ids, = ctx.saved_tensors
        return None, om_embed_lookup_backward(grad.contiguous(), ids, ctx.rows, ctx.scale), None, None


def om_embed_lookup(ids, table, scale: float = 1.0, out=None, stream=None):
    """scale * table[ids] for ids (int32 or int64, any shape, contiguous) and a
    table [rows, width]: [*ids.shape, width].  An id outside [0, rows) gives zeros.
    Where the table requires a gradient the rows carry it to the table (not into a
    given `out`)."""
    id_bytes = _ids(ids)
    if table.requires_grad and torch.is_grad_enabled():
        if out is not None:
            raise ValueError("out cannot be given where the table requires a gradient")
        return _LookupWithGradient.apply(ids, table, scale, stream)
    table_stride = _rows(table, "table", 2)[0]
    rows, width = table.shape
    shape = (*ids.shape, width)
    given = out
    if out is not None and out.requires_grad:
        _no_gradient("what is written into out", out)
    if out is None:
        out = _empty(shape, table.dtype, table.device, stream)
    _dense(out, "out", shape, table.dtype)
    handle = _launch_stream(stream, "ids table out", ids, table, out)
    _check(
        _lib.om_embed_lookup(_value_type(table, "table"), table.data_ptr(), rows, width, table_stride, ids.data_ptr(),
                             id_bytes, ids.numel(), scale, out.data_ptr(), width, handle),
        "om_embed_lookup",
    )
    _written(given)
    return out


def om_embed_lookup_backward(grad, ids, rows: int, scale: float = 1.0, accumulate: bool = False, grad_table=None,
                             stream=None):
    """The table's gradient [rows, width] from that of om_embed_lookup's rows
    (grad [*ids.shape, width], contiguous): scale * the sum of each row's terms in
    the order of ids, added to grad_table's values with accumulate.  grad_table
    (rows may be apart) is of grad's dtype or float32."""
    id_bytes = _ids(ids)
    if grad.dim() < 1 or grad.shape[:-1] != ids.shape or not grad.is_contiguous():
        raise ValueError(f"grad must be contiguous, of shape {(*ids.shape, 'width')} (got {tuple(grad.shape)})")
    width = grad.shape[-1]
    given = grad_table
    if grad_table is None:
        if accumulate:
            raise ValueError("accumulate needs a grad_table to add to")
        grad_table = _empty((rows, width), grad.dtype, grad.device, stream)
    _no_gradient("om_embed_lookup_backward", grad, grad_table)
    table_stride = _rows(grad_table, "grad_table", 2)[0]
    if tuple(grad_table.shape) != (rows, width) or grad_table.dtype not in (grad.dtype, torch.float32):
        raise ValueError(f"grad_table must be {grad.dtype} or float32 of shape {(rows, width)} "
                         f"(got {grad_table.dtype}, {tuple(grad_table.shape)})")
    handle = _launch_stream(stream, "grad ids grad_table", grad, ids, grad_table)
    _check(
        _lib.om_embed_lookup_backward(_value_type(grad, "grad"), grad.data_ptr(), ids.numel(), width, width,
                                      ids.data_ptr(), id_bytes, rows, scale, 1 if accumulate else 0,
                                      VALUE_TYPES[grad_table.dtype], grad_table.data_ptr(), table_stride, handle),
        "om_embed_lookup_backward",
    )
    _written(given)
    return grad_table


# ---------------------------------------------------------- routed experts --

def om_expert_mlp(x, ids, weights, up, down, gate=None, act: str = "silu", out=None, stream=None):
    """[tokens, hidden]: the sum over a token's picks of weights[t, j] * down[e] @
    (act(gate[e] @ x[t]) * (up[e] @ x[t])), e = ids[t, j], or of act(up[e] @ x[t])
    without a gate.  x [tokens, hidden], up and gate [experts, inner, hidden], down
    [experts, hidden, inner], all bfloat16 or all float16; ids int32 and weights
    float32 [tokens, picks] as om_route_topk gives them (an id outside the experts
    is an empty slot); act "silu", "gelu" or "relu".  For a few tokens: at most 64."""
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)} (got {act!r})")
    x_stride = _rows(x, "x", 2)[0]
    tokens, hidden = x.shape
    if x.dtype not in (torch.bfloat16, torch.float16):
        raise ValueError(f"x must be bfloat16 or float16 (got {x.dtype})")
    if ids.dim() != 2:
        raise ValueError("ids must have 2 dimensions")
    picks = ids.shape[1]
    _dense(ids, "ids", (tokens, picks), torch.int32)
    _dense(weights, "weights", (tokens, picks), torch.float32)
    up_strides, down_strides = _rows(up, "up", 3), _rows(down, "down", 3)
    experts, inner = up.shape[:2]
    gate_strides = (0, 0, 1) if gate is None else _rows(gate, "gate", 3)
    for t, name, shape in ((up, "up", (experts, inner, hidden)), (down, "down", (experts, hidden, inner)),
                           (gate, "gate", (experts, inner, hidden))):
        if t is not None and (t.dtype != x.dtype or tuple(t.shape) != shape):
            raise ValueError(f"{name} must be {x.dtype} of shape {shape} (got {t.dtype}, {tuple(t.shape)})")
    given = out
    _no_gradient("om_expert_mlp", x, weights, up, gate, down, out)
    if out is None:
        out = _empty((tokens, hidden), x.dtype, x.device, stream)
    out_stride = _rows(out, "out", 2)[0]
    if tuple(out.shape) != (tokens, hidden) or out.dtype != x.dtype:
        raise ValueError(f"out must be {x.dtype} of shape {(tokens, hidden)} (got {out.dtype}, {tuple(out.shape)})")
    handle = _launch_stream(stream, "x ids weights up down gate out", x, ids, weights, up, down, gate, out)
    _check(
        _lib.om_expert_mlp(VALUE_TYPES[x.dtype], x.data_ptr(), tokens, hidden, x_stride, ids.data_ptr(),
                           weights.data_ptr(), picks, experts, inner, up.data_ptr(), up_strides[0], up_strides[1],
                           None if gate is None else gate.data_ptr(), gate_strides[0], gate_strides[1], down.data_ptr(),
                           down_strides[0], down_strides[1], ACTIVATIONS[act], out.data_ptr(), out_stride, handle),
        "om_expert_mlp",
    )
    _written(given)
    return out
