"""Torch binding of the operators around the dense head: the final norm with
the residual's addition and an int8 output (``fh_rmsnorm``), the int8 product
and the dense head on it (``fh_w8a8_*``), the rules on logits and the choice of
the token (``fh_logits_apply``).

Functions named like the C entry points marshal arguments: they check types,
shapes and placement, pass raw pointers and the HIP stream, and raise on a
non-OK status.  ``rmsnorm``, ``W8A8Head``, ``LogitRules`` and ``logits_apply``
allocate outputs and workspaces on top of them.  Matrices may have any row
stride; their rows are dense.  All tensors of a call are on one GPU, which need
not be the current one; work goes to its current stream unless ``stream`` is
given, and what the call allocates belongs to that stream.  Inputs made on
another stream have to be ready, and alive until the call's stream has passed
it, as for any launch.
"""

from __future__ import annotations

import contextlib
import ctypes
import sys

import torch

from . import _abi
from ._abi import FH_BF16, FH_F32, check

_DTYPES = {torch.float32: FH_F32, torch.bfloat16: FH_BF16}


def _shaped(t, dtype, shape, name):
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")


def _rows(t, dtype, shape, name):
    """Row stride of a matrix [B x w] whose rows are dense."""
    _shaped(t, dtype, shape, name)
    ld, inner = t.stride()
    if inner != 1 and shape[1] != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    if shape[0] == 1:
        return max(ld, shape[1])  # one row: its stride says nothing
    if ld < shape[1]:
        raise ValueError(f"{name}: rows must not overlap (stride {ld})")
    return ld


def _vector(t, dtype, n, name):
    _shaped(t, dtype, (n,), name)
    if n > 1 and t.stride(0) != 1:
        raise ValueError(f"{name}: must be contiguous")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _device(*tensors):
    """The one GPU that every tensor is on."""
    dev = tensors[0].device
    for t in tensors:
        if t is not None and (t.device != dev or not t.is_cuda):
            raise ValueError("tensors of a libflashhead call must be on one GPU")
    return dev


_SAME = contextlib.nullcontext()


def _on(dev, stream):
    """Make `dev` current for a call, and `stream`, so that outputs allocated
    in the call belong to the stream that writes them."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError("stream is on another device than the tensors")
        return torch.cuda.stream(stream)
    return _SAME if dev.index == torch.cuda.current_device() else torch.cuda.device(dev)


def _stream(dev):
    return torch.cuda.current_stream(dev).cuda_stream


# The same without building a Stream object (1.9 us of a call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is not None:
    def _stream(dev):  # noqa: F811
        return _raw_stream(dev.index)


# ------------------------------------------------------------------ the norm

def _norm_inputs(x, residual, weight):
    if x.dim() != 2 or x.dtype not in _DTYPES:
        raise ValueError(f"x must be [B x d] float32 or bfloat16, got {x.dtype} {tuple(x.shape)}")
    ld_r = 0 if residual is None else _rows(residual, x.dtype, x.shape, "residual")
    if weight is not None:
        _vector(weight, x.dtype, x.shape[1], "weight")
    return _rows(x, x.dtype, x.shape, "x"), ld_r


def fh_rmsnorm(x, residual, weight, eps, weight_offset, out=None, out_residual=None, out_q=None,
               out_scale=None, stream=None) -> None:
    """out = rmsnorm(x + residual) * (weight_offset + weight); out_residual =
    x + residual; (out_q, out_scale) = the norm in int8 with a scale per row."""
    ld_x, ld_r = _norm_inputs(x, residual, weight)
    if (out_q is None) != (out_scale is None):
        raise ValueError("out_q and out_scale go together")
    dt, shape = x.dtype, x.shape
    ld_o = 0 if out is None else _rows(out, dt, shape, "out")
    ld_s = 0 if out_residual is None else _rows(out_residual, dt, shape, "out_residual")
    ld_q = 0
    if out_q is not None:
        ld_q = _rows(out_q, torch.int8, shape, "out_q")
        _vector(out_scale, torch.float32, shape[0], "out_scale")
    dev = _device(x, residual, weight, out, out_residual, out_q, out_scale)
    with _on(dev, stream):
        check(_abi.load().fh_rmsnorm(x.data_ptr(), ld_x, _ptr(residual), ld_r, _ptr(weight), _DTYPES[dt], shape[0],
                                     shape[1], eps, weight_offset, _ptr(out), ld_o, _ptr(out_residual), ld_s,
                                     _ptr(out_q), ld_q, _ptr(out_scale), _stream(dev)))


def rmsnorm(x, weight=None, *, residual=None, eps=1e-6, weight_offset=0.0, want_out=True, want_q=False,
            stream=None) -> dict:
    """The final norm of hidden states x [B x d] (any row stride, so the last
    positions of [B x T x d] need no copy).  Returns "out" (the head's h) with
    want_out, "residual" (x + residual) with a residual, and with want_q the
    int8 head's "q" [B x d] (rows padded to 16 bytes) and "q_scale" [B]."""
    ld_x, ld_r = _norm_inputs(x, residual, weight)
    dev = _device(x, residual, weight)
    dt, (B, d) = x.dtype, x.shape
    got = {}
    out = out_residual = q = scale = None
    with _on(dev, stream):
        if want_out:
            got["out"] = out = x.new_empty((B, d))
        if residual is not None:
            got["residual"] = out_residual = x.new_empty((B, d))
        ld_q = (d + 15) // 16 * 16
        if want_q:
            q = x.new_empty((B, ld_q), dtype=torch.int8)
            got["q"] = q if d == ld_q else q[:, :d]
            got["q_scale"] = scale = x.new_empty((B,), dtype=torch.float32)
        check(_abi.load().fh_rmsnorm(x.data_ptr(), ld_x, _ptr(residual), ld_r, _ptr(weight), _DTYPES[dt], B, d, eps,
                                     weight_offset, _ptr(out), d, _ptr(out_residual), d, _ptr(q), ld_q, _ptr(scale),
                                     _stream(dev)))
    return got


# ------------------------------------------------------- int8 product and head

# What each handle holds, keyed by its value: (n, k, device).
_WEIGHTS = {}


def _key(w):
    return w.value if isinstance(w, ctypes.c_void_p) else w


def _weight(w):
    info = _WEIGHTS.get(_key(w))
    if info is None:
        raise ValueError("unknown int8 weight (not created by fh_w8a8_create, or destroyed)")
    return info


def fh_w8a8_create(W: torch.Tensor, stream=None) -> ctypes.c_void_p:
    """Quantise W [n x k] (float32 or bfloat16, contiguous) row by row."""
    if W.dim() != 2 or W.dtype not in _DTYPES or not W.is_contiguous():
        raise ValueError("W must be a contiguous [n x k] float32 or bfloat16 matrix")
    dev = _device(W)
    w = ctypes.c_void_p()
    with _on(dev, stream):
        check(_abi.load().fh_w8a8_create(W.data_ptr(), _DTYPES[W.dtype], W.shape[0], W.shape[1], _stream(dev),
                                         ctypes.byref(w)))
    _WEIGHTS[w.value] = (W.shape[0], W.shape[1], dev)
    return w


def fh_w8a8_create_codes(codes: torch.Tensor, scales: torch.Tensor, stream=None) -> ctypes.c_void_p:
    """Take int8 codes [n x k] and float32 scales [n] as they are."""
    if codes.dim() != 2 or codes.dtype is not torch.int8 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous [n x k] int8 matrix")
    _vector(scales, torch.float32, codes.shape[0], "scales")
    dev = _device(codes, scales)
    w = ctypes.c_void_p()
    with _on(dev, stream):
        check(_abi.load().fh_w8a8_create_codes(codes.data_ptr(), scales.data_ptr(), codes.shape[0], codes.shape[1],
                                               _stream(dev), ctypes.byref(w)))
    _WEIGHTS[w.value] = (codes.shape[0], codes.shape[1], dev)
    return w


def fh_w8a8_destroy(w) -> None:
    """Release the weight (None is a no-op); a second time is refused."""
    if _key(w) is None:
        return
    if _WEIGHTS.pop(_key(w), None) is None:
        raise ValueError("unknown int8 weight (not created by fh_w8a8_create, or destroyed)")
    _abi.load().fh_w8a8_destroy(w)


def fh_w8a8_get(w, codes, scales, stream=None) -> None:
    n, k, dev = _weight(w)
    _shaped(codes, torch.int8, (n, k), "codes")
    if not codes.is_contiguous():
        raise ValueError("codes: must be contiguous")
    _vector(scales, torch.float32, n, "scales")
    if _device(codes, scales) != dev:
        raise ValueError("codes and scales must be on the weight's GPU")
    with _on(dev, stream):
        check(_abi.load().fh_w8a8_get(w, codes.data_ptr(), scales.data_ptr(), _stream(dev)))


def _product_args(w, q, q_scale):
    n, k, dev = _weight(w)
    if q.dim() != 2:
        raise ValueError(f"q must be [B x k], got shape {tuple(q.shape)}")
    B = q.shape[0]
    ld_q = _rows(q, torch.int8, (B, k), "q")
    _vector(q_scale, torch.float32, B, "q_scale")
    return n, B, ld_q, dev


def _size(status):
    if status < 0:
        check(status)
    return status


def _workspace_arg(workspace):
    if workspace is None:
        return None, 0
    _vector(workspace, torch.uint8, workspace.numel(), "workspace")
    return workspace.data_ptr(), workspace.numel()


def fh_w8a8_workspace(w, q, forward: bool) -> int:
    """Bytes of workspace of a product (or, with forward, head) call on q."""
    _, k, _ = _weight(w)
    ld_q = _rows(q, torch.int8, (q.shape[0], k), "q")
    return _size(_abi.load().fh_w8a8_workspace(w, q.data_ptr(), ld_q, q.shape[0], int(forward)))


def fh_w8a8_matmul(w, q, q_scale, out, workspace=None, stream=None) -> None:
    n, B, ld_q, dev = _product_args(w, q, q_scale)
    if out.dtype not in _DTYPES:
        raise ValueError("out must be float32 or bfloat16")
    ld_out = _rows(out, out.dtype, (B, n), "out")
    ws, ws_bytes = _workspace_arg(workspace)
    if _device(q, q_scale, out, workspace) != dev:
        raise ValueError("tensors must be on the weight's GPU")
    with _on(dev, stream):
        check(_abi.load().fh_w8a8_matmul(w, q.data_ptr(), ld_q, q_scale.data_ptr(), B, out.data_ptr(), ld_out,
                                         _DTYPES[out.dtype], ws, ws_bytes, _stream(dev)))


def fh_w8a8_forward(w, q, q_scale, mode, temperature, seed, out_token, out_token_logit=None, out_lse=None,
                    out_logits=None, workspace=None, stream=None) -> None:
    n, B, ld_q, dev = _product_args(w, q, q_scale)
    _vector(out_token, torch.int32, B, "out_token")
    if out_token_logit is not None:
        _vector(out_token_logit, torch.float32, B, "out_token_logit")
    if out_lse is not None:
        _vector(out_lse, torch.float32, B, "out_lse")
    ld_out = 0 if out_logits is None else _rows(out_logits, torch.float32, (B, n), "out_logits")
    ws, ws_bytes = _workspace_arg(workspace)
    if _device(q, q_scale, out_token, out_token_logit, out_lse, out_logits, workspace) != dev:
        raise ValueError("tensors must be on the weight's GPU")
    with _on(dev, stream):
        check(_abi.load().fh_w8a8_forward(w, q.data_ptr(), ld_q, q_scale.data_ptr(), B, mode, temperature, seed,
                                          out_token.data_ptr(), _ptr(out_token_logit), _ptr(out_lse),
                                          _ptr(out_logits), ld_out, ws, ws_bytes, _stream(dev)))


# Bytes of workspace that may share an allocation with the outputs of a choice,
# and so live as long as they do.
_SHARED = 16384


def _choice_outputs(t, B, size):
    """token [B] int32, token_logit and lse [B] float32 on t's GPU, and size
    bytes of workspace (None for none).  One allocation for all where the
    workspace is small (3.2 us of the host's time; 5.0 for two), else one for
    the outputs (a third of the time of three) and one for the workspace."""
    if size <= _SHARED:
        words = (size + 3) // 4
        ws = t.new_empty(words + 3 * B, dtype=torch.float32)
        _, token, logit, lse = ws.split_with_sizes((words, B, B, B))
    else:
        token, logit, lse = t.new_empty((3, B), dtype=torch.float32).unbind(0)
        ws = t.new_empty(size, dtype=torch.uint8)
    return token.view(torch.int32), logit, lse, ws if size else None


class _Steps:
    """What a decode step does on a dense head with quantised operands.  The head
    has `device`, `matmul`, `forward`, and `_states`: the norm in the form that
    both take."""

    def step(self, x: torch.Tensor, weight=None, *, residual=None, eps=1e-6, weight_offset=0.0, rules=None,
             mode: int = 0, temperature: float = 1.0, seed: int = 0, want_logits: bool = False,
             stream=None) -> dict:
        """One decode step after the last layer: rmsnorm(x + residual) in the
        head's operands, the head, the rules (LogitRules, or None) and the choice
        of the token."""
        with _on(self.device, stream):
            q, scale = self._states(x, weight, residual, eps, weight_offset)
            if rules is None:
                return self.forward(q, scale, mode, temperature, seed, want_logits)
            z = self.matmul(q, scale)
            out = logits_apply(z, rules, mode=mode, temperature=temperature, seed=seed, out=z)
            if not want_logits:
                del out["logits"]
            return out

    def beam_step(self, x: torch.Tensor, scores: torch.Tensor, weight=None, *, residual=None, eps=1e-6,
                  weight_offset=0.0, rules=None, keep=None, finished=None, eos: int = -1, want_logits: bool = False,
                  stream=None) -> dict:
        """step for beams: x [S W x d], scores [S x W]; after the norm, the head and
        the rules the best continuations over beams and tokens (beam_select),
        whose "parent" beam_reorder takes."""
        from .beam import beam_select
        with _on(self.device, stream):
            q, scale = self._states(x, weight, residual, eps, weight_offset)
            z = self.matmul(q, scale)
            if rules is not None:
                logits_apply(z, rules, want_token=False, out=z)
            out = beam_select(z, scores, keep=keep, finished=finished, eos=eos)
            if want_logits:
                out["logits"] = z
            return out


class W8A8Head(_Steps):
    """A dense head (or any linear layer) with int8 weights and activations:
    the rows of E quantised here, or int8 codes and scales as they are."""

    def __init__(self, E: torch.Tensor = None, *, codes: torch.Tensor = None, scales: torch.Tensor = None,
                 stream=None):
        self.w = None
        if (E is None) == (codes is None) or (codes is None) != (scales is None):
            raise ValueError("give either E, or codes and scales")
        if E is not None:
            self.w = fh_w8a8_create(E, stream)
        else:
            self.w = fh_w8a8_create_codes(codes, scales, stream)
        self.n, self.k, self.device = _weight(self.w)

    def close(self):
        w, self.w = self.w, None
        fh_w8a8_destroy(w)

    def __del__(self):
        # not while the interpreter shuts down (see FlashHead)
        if sys is None or sys.is_finalizing():
            return
        try:
            self.close()
        except Exception:
            pass

    def _inputs(self, q, q_scale, forward):
        """Row stride, workspace size of a call on q; all on the weight's GPU."""
        _, B, ld_q, dev = _product_args(self.w, q, q_scale)
        if _device(q, q_scale) != dev:
            raise ValueError("tensors must be on the weight's GPU")
        return ld_q, _size(_abi.load().fh_w8a8_workspace(self.w, q.data_ptr(), ld_q, B, forward))

    def _states(self, x, weight, residual, eps, weight_offset):
        h = rmsnorm(x, weight, residual=residual, eps=eps, weight_offset=weight_offset, want_out=False, want_q=True)
        return h["q"], h["q_scale"]

    def codes(self, stream=None):
        """The codes [n x k] and scales [n]."""
        with _on(self.device, stream):
            codes = torch.empty((self.n, self.k), dtype=torch.int8, device=self.device)
            scales = torch.empty((self.n,), dtype=torch.float32, device=self.device)
            fh_w8a8_get(self.w, codes, scales)
        return codes, scales

    def matmul(self, q: torch.Tensor, q_scale: torch.Tensor, dtype=torch.float32, stream=None) -> torch.Tensor:
        """[B x n] = (q code^T) scaled per token and channel, in float32 or
        bfloat16; q and q_scale as rmsnorm(want_q=True) gives them."""
        ld_q, size = self._inputs(q, q_scale, 0)
        if dtype not in _DTYPES:
            raise ValueError("dtype must be float32 or bfloat16")
        B = q.shape[0]
        with _on(self.device, stream):
            out = q.new_empty((B, self.n), dtype=dtype)
            ws = q.new_empty((size,), dtype=torch.uint8) if size else None
            check(_abi.load().fh_w8a8_matmul(self.w, q.data_ptr(), ld_q, q_scale.data_ptr(), B, out.data_ptr(),
                                             self.n, _DTYPES[dtype], _ptr(ws), size, _stream(self.device)))
        return out

    def forward(self, q: torch.Tensor, q_scale: torch.Tensor, mode: int = 0, temperature: float = 1.0,
                seed: int = 0, want_logits: bool = False, stream=None) -> dict:
        """FlashHead.dense on int8 operands: "token", "token_logit", "lse" and
        with want_logits "logits" [B x n]."""
        ld_q, size = self._inputs(q, q_scale, 1)
        B = q.shape[0]
        with _on(self.device, stream):
            token, logit, lse, ws = _choice_outputs(q, B, size)
            out = {"token": token, "token_logit": logit, "lse": lse}
            logits = None
            if want_logits:
                out["logits"] = logits = q.new_empty((B, self.n), dtype=torch.float32)
            check(_abi.load().fh_w8a8_forward(self.w, q.data_ptr(), ld_q, q_scale.data_ptr(), B, mode, temperature,
                                              seed, token.data_ptr(), logit.data_ptr(), lse.data_ptr(), _ptr(logits),
                                              self.n, _ptr(ws), size, _stream(self.device)))
        return out


# ------------------------------------------------------------ rules on logits

class LogitRules:
    """The rules of a batch of B rows over a vocabulary of v tokens, kept from
    step to step: the tensors are borrowed and read at every call, so a program
    (or a captured graph) updates them in place.

    history [B x L] int32 with n_prompt, n_history [B] int32; repetition,
    frequency, presence [B] float32 (without a history they do nothing);
    bias_ids [B x N] int32 with bias float32 and n_bias [B] int32; mask [R x ceil(v / 32)] int32 words (bit t % 32 of
    word t / 32 allows token t) with mask_row [B] int32 (outside [0, R): all
    allowed; without it row b takes mask row b).  Each may be None.
    """

    def __init__(self, v: int, *, history=None, n_prompt=None, n_history=None, repetition=None, frequency=None,
                 presence=None, bias_ids=None, bias=None, n_bias=None, mask=None, mask_row=None):
        vectors = {"n_prompt": (n_prompt, torch.int32), "n_history": (n_history, torch.int32),
                   "repetition": (repetition, torch.float32), "frequency": (frequency, torch.float32),
                   "presence": (presence, torch.float32), "n_bias": (n_bias, torch.int32),
                   "mask_row": (mask_row, torch.int32)}
        lists = {"history": history, "bias_ids": bias_ids, "bias": bias}
        sized = [t for t in lists.values() if t is not None] + [t for t, _ in vectors.values() if t is not None]
        for name, t in lists.items():
            if t is not None and t.dim() != 2:
                raise ValueError(f"{name} must be [B x length], got shape {tuple(t.shape)}")
        if history is None and (n_prompt is not None or n_history is not None):
            raise ValueError("n_prompt and n_history need a history")
        if (bias_ids is None) != (bias is None) or (n_bias is not None and bias is None):
            raise ValueError("bias_ids and bias go together, n_bias needs them")
        if mask is None and mask_row is not None:
            raise ValueError("mask_row needs a mask")
        self.v = v
        self.B = sized[0].shape[0] if sized else (mask.shape[0] if mask is not None else None)
        s = _abi.FhLogitRules()
        # an empty list or table has no address: what counts or picks its rows goes with it
        empty = {name for name, t, axis in (("n_prompt", history, 1), ("n_history", history, 1), ("n_bias", bias, 1),
                                            ("mask_row", mask, 0)) if t is not None and t.shape[axis] == 0}
        for name, (t, dt) in vectors.items():
            if t is not None:
                _vector(t, dt, self.B, name)
                if name not in empty:
                    setattr(s, name, t.data_ptr())
        if history is not None:
            s.ld_history = _rows(history, torch.int32, (self.B, history.shape[1]), "history")
            s.history, s.history_len = history.data_ptr(), history.shape[1]
        if bias is not None:
            shape = (self.B, bias.shape[1])
            s.ld_bias = _rows(bias, torch.float32, shape, "bias")
            if _rows(bias_ids, torch.int32, shape, "bias_ids") != s.ld_bias and self.B != 1 and shape[1]:
                raise ValueError("bias_ids and bias must have the same row stride")
            s.bias_ids, s.bias, s.bias_len = bias_ids.data_ptr(), bias.data_ptr(), bias.shape[1]
        if mask is not None:
            if mask.dim() != 2:
                raise ValueError(f"mask must be [R x words], got shape {tuple(mask.shape)}")
            s.ld_mask = _rows(mask, torch.int32, (mask.shape[0], (v + 31) // 32), "mask")
            if mask.shape[0]:
                s.mask, s.mask_rows = mask.data_ptr(), mask.shape[0]
            if mask_row is None and mask.shape[0] < (self.B or 0):
                raise ValueError("the mask has fewer rows than the batch; give mask_row")
        kept = [t for t in sized + [mask] if t is not None]
        self.device = _device(*kept) if kept else None
        self._kept = kept  # borrowed: alive as long as the struct points to them
        self._struct = s


def fh_logits_workspace(B: int, n: int) -> int:
    """Bytes of workspace of a call over [B x n] logits that chooses tokens."""
    return _size(_abi.load().fh_logits_workspace(B, n))


def _apply_inputs(logits, ids, v, rules):
    """Row strides of logits and ids, the rules' struct; all on one GPU."""
    if logits.dim() != 2:
        raise ValueError(f"logits must be [B x n], got shape {tuple(logits.shape)}")
    shape = logits.shape
    ld_z = _rows(logits, torch.float32, shape, "logits")
    ld_ids = 0 if ids is None else _rows(ids, torch.int32, shape, "ids")
    if rules is None:
        return ld_z, ld_ids, None
    if rules.v != v or (rules.B is not None and rules.B != shape[0]):
        raise ValueError(f"rules are of {rules.B} rows over {rules.v} tokens, logits of {shape[0]} rows over {v}")
    if rules.device is not None and rules.device != logits.device:
        raise ValueError("rules and logits must be on one GPU")
    return ld_z, ld_ids, rules._struct


def fh_logits_apply(logits, ids, v, rules, mode, temperature, seed, out_logits=None, out_token=None,
                    out_token_logit=None, out_lse=None, workspace=None, stream=None) -> None:
    """The rules (LogitRules or None) on logits [B x n], of all v tokens or of
    the tokens ids [B x n], then the choice of the token."""
    ld_z, ld_ids, struct = _apply_inputs(logits, ids, v, rules)
    B, n = logits.shape
    ld_out = 0 if out_logits is None else _rows(out_logits, torch.float32, logits.shape, "out_logits")
    if out_token is not None:
        _vector(out_token, torch.int32, B, "out_token")
    if out_token_logit is not None:
        _vector(out_token_logit, torch.float32, B, "out_token_logit")
    if out_lse is not None:
        _vector(out_lse, torch.float32, B, "out_lse")
    ws, ws_bytes = _workspace_arg(workspace)
    dev = _device(logits, ids, out_logits, out_token, out_token_logit, out_lse, workspace)
    with _on(dev, stream):
        check(_abi.load().fh_logits_apply(logits.data_ptr(), ld_z, _ptr(ids), ld_ids, B, n, v, struct, mode,
                                          temperature, seed, _ptr(out_logits), ld_out, _ptr(out_token),
                                          _ptr(out_token_logit), _ptr(out_lse), ws, ws_bytes, _stream(dev)))


def logits_apply(logits, rules=None, *, ids=None, v=None, mode: int = 0, temperature: float = 1.0, seed: int = 0,
                 want_token: bool = True, out=None, stream=None) -> dict:
    """The rules on logits [B x n] of all v tokens, or of the tokens ids [B x n]
    (a forward's "logits" and "ids"): "logits" (in `out`, which may be logits
    itself) and with want_token "token", "token_logit" and "lse".  v is the
    rules' or, of logits of all tokens, n; ids without rules need it."""
    if v is None:
        if rules is None and ids is not None:
            raise ValueError("ids without rules need v, the number of tokens")
        v = rules.v if rules is not None else logits.shape[-1]
    ld_z, ld_ids, struct = _apply_inputs(logits, ids, v, rules)
    dev = _device(logits, ids, out)
    B, n = logits.shape
    ld_out = n if out is None else _rows(out, torch.float32, logits.shape, "out")
    lib = _abi.load()
    token = logit = lse = ws = None
    size = 0
    with _on(dev, stream):
        if out is None:
            out = torch.empty_like(logits)
        got = {"logits": out}
        if want_token:
            size = _size(lib.fh_logits_workspace(B, n))
            token, logit, lse, ws = _choice_outputs(logits, B, size)
            got["token"], got["token_logit"], got["lse"] = token, logit, lse
        check(lib.fh_logits_apply(logits.data_ptr(), ld_z, _ptr(ids), ld_ids, B, n, v, struct, mode, temperature, seed,
                                  out.data_ptr(), ld_out, _ptr(token), _ptr(logit), _ptr(lse), _ptr(ws), size,
                                  _stream(dev)))
    return got
