"""Torch binding of decoding by beams: the best continuations over beams and
tokens (``fh_beam_select``) and the reordering of states by the beams that they
continue (``fh_beam_reorder``).

As in ``serve``, functions named like the C entry points marshal arguments, and
``beam_select`` and ``beam_reorder`` allocate and lay out on top of them.  Row
s * W + w of a batch is beam w of sequence s, for S sequences of W beams.
"""

from __future__ import annotations

import ctypes
import functools

import torch

from . import _abi
from ._abi import check
from .serve import _device, _on, _ptr, _rows, _size, _stream, _vector, _workspace_arg


def _beams(t, dtype, shape, name):
    """A dense [S x W] (or [S x keep]) tensor."""
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")


def fh_beam_workspace(sequences: int, beams: int, n: int) -> int:
    """Bytes of workspace of a beam_select call over [sequences beams x n] logits."""
    return _size(_abi.load().fh_beam_workspace(sequences, beams, n))


def _select_inputs(logits, ids, scores, lse, finished):
    if logits.dim() != 2 or scores.dim() != 2:
        raise ValueError(f"logits must be [S W x n] and scores [S x W], got shapes {tuple(logits.shape)} and "
                         f"{tuple(scores.shape)}")
    S, W = scores.shape
    shape = (S * W, logits.shape[1])
    ld_z = _rows(logits, torch.float32, shape, "logits")
    ld_ids = 0 if ids is None else _rows(ids, torch.int32, shape, "ids")
    _beams(scores, torch.float32, (S, W), "scores")
    if lse is not None:
        _vector(lse, torch.float32, S * W, "lse")
    if finished is not None:
        _beams(finished, torch.int32, (S, W), "finished")
    return S, W, ld_z, ld_ids


def fh_beam_select(logits, ids, v, lse, scores, finished, eos, keep, out_score, out_token, out_parent,
                   out_finished=None, workspace=None, stream=None) -> None:
    """Of each sequence the `keep` continuations with the largest scores + logits -
    lse, best first, with their tokens and the beams that they continue."""
    S, W, ld_z, ld_ids = _select_inputs(logits, ids, scores, lse, finished)
    outs = {"out_score": out_score, "out_token": out_token, "out_parent": out_parent, "out_finished": out_finished}
    for name, t in outs.items():
        if t is not None:
            _beams(t, torch.float32 if name == "out_score" else torch.int32, (S, keep), name)
    ws, ws_bytes = _workspace_arg(workspace)
    dev = _device(logits, ids, lse, scores, finished, *outs.values(), workspace)
    with _on(dev, stream):
        check(_abi.load().fh_beam_select(logits.data_ptr(), ld_z, _ptr(ids), ld_ids, S, W, logits.shape[1], v,
                                         _ptr(lse), scores.data_ptr(), _ptr(finished), eos, keep, out_score.data_ptr(),
                                         out_token.data_ptr(), out_parent.data_ptr(), _ptr(out_finished), ws, ws_bytes,
                                         _stream(dev)))


def beam_select(logits, scores, *, keep=None, ids=None, v=None, lse=None, finished=None, eos=-1,
                stream=None) -> dict:
    """Of each sequence the `keep` (the number of beams unless given) best
    continuations: logits [S W x n] after the rules, of all tokens or of the tokens
    ids, scores [S x W] float32 the beams' totals so far.  "score", "token" and
    "parent" [S x keep], best first; -inf, -1 and -1 where there are fewer.  lse
    [S W]: the rows' log-sum-exps where they are known, as of a retrieval head's
    candidates; else the call's own, in float32 sums (1e-7 or so, which order beams
    whose totals are that near to each other).  finished [S x W] int32: beams that offer `eos` alone, at their own
    score; then "finished" says which of the continuations are.  v: the number of
    tokens, which ids need."""
    S, W, ld_z, ld_ids = _select_inputs(logits, ids, scores, lse, finished)
    n = logits.shape[1]
    if v is None:
        if ids is not None:
            raise ValueError("ids need v, the number of tokens")
        v = n
    if keep is None:
        keep = W
    if keep < 1:
        raise ValueError("keep must be at least 1")
    dev = _device(logits, ids, scores, lse, finished)
    lib = _abi.load()
    with _on(dev, stream):
        size = _size(lib.fh_beam_workspace(S, W, n))
        out = logits.new_empty((3 if finished is None else 4, S, keep))
        score, token, parent, *done = out.unbind(0)
        token, parent = token.view(torch.int32), parent.view(torch.int32)
        got = {"score": score, "token": token, "parent": parent}
        if done:
            got["finished"] = done = done[0].view(torch.int32)
        ws = logits.new_empty(size // 4)
        at = out.data_ptr()
        step = 4 * S * keep
        check(lib.fh_beam_select(logits.data_ptr(), ld_z, _ptr(ids), ld_ids, S, W, n, v, _ptr(lse), scores.data_ptr(),
                                 _ptr(finished), eos, keep, at, at + step, at + 2 * step,
                                 None if finished is None else at + 3 * step, ws.data_ptr(), size, _stream(dev)))
    return got


def _reorder_args(states, layout, parent, lengths):
    """The GPU of a call, and its arguments but for the stream."""
    S, W = parent.shape
    _beams(parent, torch.int32, (S, W), "parent")
    if lengths is not None:
        _vector(lengths, torch.int32, S * W, "lengths")
    dev = _device(parent, lengths, *states)
    n = len(states)
    return dev, ((ctypes.c_void_p * n)(*[t.data_ptr() for t in states]), n, _abi.FhBeamLayout(*layout), S, W,
                 parent.data_ptr(), _ptr(lengths))


def fh_beam_reorder(states, layout, parent, lengths=None, stream=None) -> None:
    """Rows of states (tensors of one layout, fh_beam_layout's fields in bytes as a
    sequence) permuted in place by parent [S x W]."""
    dev, args = _reorder_args(states, layout, parent, lengths)
    with _on(dev, stream):
        check(_abi.load().fh_beam_reorder(*args, _stream(dev)))


def fh_beam_reorder_check(states, layout, parent, lengths=None) -> None:
    """Raises what fh_beam_reorder would, and moves nothing."""
    check(_abi.load().fh_beam_reorder_check(*_reorder_args(states, layout, parent, lengths)[1]))


def _joined(shape, strides):
    """[size, stride] of dimensions that are one after another in memory joined."""
    dims = []
    for size, stride in zip(shape, strides):
        if size == 1:
            continue
        if dims and dims[-1][1] == size * stride:
            dims[-1] = [dims[-1][0] * size, stride]
        else:
            dims.append([size, stride])
    return dims


def _layout(t, rows, dim, length_dim):
    """fh_beam_layout of a state, in bytes, as a tuple."""
    return _levels(t.shape, t.stride(), t.element_size(), rows, dim, length_dim)


@functools.lru_cache(maxsize=1024)
def _levels(shape, strides, e, rows, dim, length_dim):
    n = len(shape)
    if not -n <= dim < n or shape[dim] != rows:
        raise ValueError(f"a state of shape {tuple(shape)} has no {rows} rows in dimension {dim}")
    dim %= n
    outer = _joined(shape[:dim], strides[:dim])
    if length_dim is not None and (not -n <= length_dim < n or length_dim % n <= dim):
        raise ValueError("length_dim must be one of the dimensions behind dim")
    at = None if length_dim is None else length_dim % n
    behind = [i for i in range(dim + 1, n) if i != at]
    rest = _joined([shape[i] for i in behind], [strides[i] for i in behind])
    run = rest.pop()[0] if rest and rest[-1][1] == 1 else 1
    if at is None:
        mid, positions = rest[:-1], rest[-1:]
    else:
        mid, positions = rest, [[shape[at], strides[at]]]
    if len(outer) > 1 or len(mid) > 1:
        raise ValueError(f"a state of shape {tuple(shape)} and strides {strides} has more levels than a layout")
    (no, lo), (nm, lm), (np_, lp) = (d[0] if d else (1, 0) for d in (outer, mid, positions))
    return (no, nm, np_, run * e, lo * e, strides[dim] * e, lm * e, lp * e)


def beam_reorder(states, parent, *, dim=0, lengths=None, length_dim=None, stream=None) -> None:
    """Rows of states (a tensor or several, of any types and sizes: key and value
    caches, token histories, counts) permuted in place: row s W + w takes row s W +
    parent[s, w], all at once; where parent is outside [0, W) a row stays.  The
    rows are in dimension `dim`, dimensions before it are layers.  lengths [S W]
    int32 with length_dim (behind dim): only that many first positions of each row
    count; what lies behind them stays.  parent and lengths must not be part of a
    state, and states must not overlap (one listed twice is refused).  States of
    one layout go together in one launch; a call that is refused has moved none."""
    if isinstance(states, torch.Tensor):
        states = [states]
    if parent.dim() != 2:
        raise ValueError(f"parent must be [S x W], got shape {tuple(parent.shape)}")
    if (lengths is None) != (length_dim is None):
        raise ValueError("lengths and length_dim go together")
    rows = parent.shape[0] * parent.shape[1]
    groups = {}
    for t in states:
        layout = _layout(t, rows, dim, length_dim)
        if t.numel():
            groups.setdefault(layout, []).append(t)
    if len(groups) != 1:  # a call checks its own; none moves before all are checked
        at = [t.data_ptr() for same in groups.values() for t in same]
        if len(set(at)) != len(at):
            raise ValueError("a state is listed twice, in two layouts")
        _device(parent, lengths, *states)
        for layout, same in groups.items():
            fh_beam_reorder_check(same, layout, parent, lengths)
    for layout, same in groups.items():
        fh_beam_reorder(same, layout, parent, lengths, stream)
