"""Torch binding of the fp8 head: hidden states in 8-bit floating point
(``torch.float8_e4m3fn``) with a scale per 128 (``fh_rmsnorm_fp8``,
``fh_fp8_quant``), the product with a weight that has a scale per block of
128 x 128 and the dense head on it (``fh_fp8_*``).

As in ``serve``, functions named like the C entry points marshal arguments, and
``rmsnorm_fp8``, ``fp8_quant`` and ``FP8Head`` allocate outputs and workspaces on
top of them; matrices may have any row stride.
"""

from __future__ import annotations

import ctypes
import sys

import torch

from . import _abi
from ._abi import check
from .serve import (_DTYPES, _Steps, _choice_outputs, _device, _key, _norm_inputs, _on, _ptr, _rows, _shaped, _size,
                    _stream, _vector, _workspace_arg)

F8 = torch.float8_e4m3fn


def _groups(d: int) -> int:
    """Scales of a row of d elements."""
    return (d + 127) // 128


def _codes_out(out_q, out_scale, shape):
    return _rows(out_q, F8, shape, "out_q"), _rows(out_scale, torch.float32, (shape[0], _groups(shape[1])), "out_scale")


# -------------------------------------------------------- hidden states in fp8

def fh_rmsnorm_fp8(x, residual, weight, eps, weight_offset, out_q, out_scale, out=None, out_residual=None,
                   stream=None) -> None:
    """(out_q, out_scale) = rmsnorm(x + residual) * (weight_offset + weight) in
    fp8; out, out_residual as fh_rmsnorm's."""
    ld_x, ld_r = _norm_inputs(x, residual, weight)
    dt, shape = x.dtype, x.shape
    ld_o = 0 if out is None else _rows(out, dt, shape, "out")
    ld_s = 0 if out_residual is None else _rows(out_residual, dt, shape, "out_residual")
    ld_q, ld_g = _codes_out(out_q, out_scale, shape)
    dev = _device(x, residual, weight, out, out_residual, out_q, out_scale)
    with _on(dev, stream):
        check(_abi.load().fh_rmsnorm_fp8(x.data_ptr(), ld_x, _ptr(residual), ld_r, _ptr(weight), _DTYPES[dt], shape[0],
                                         shape[1], eps, weight_offset, _ptr(out), ld_o, _ptr(out_residual), ld_s,
                                         out_q.data_ptr(), ld_q, out_scale.data_ptr(), ld_g, _stream(dev)))


def fh_fp8_quant(x, out_q, out_scale, stream=None) -> None:
    """(out_q, out_scale) = x in fp8."""
    ld_x, _ = _norm_inputs(x, None, None)
    ld_q, ld_g = _codes_out(out_q, out_scale, x.shape)
    dev = _device(x, out_q, out_scale)
    with _on(dev, stream):
        check(_abi.load().fh_fp8_quant(x.data_ptr(), ld_x, _DTYPES[x.dtype], x.shape[0], x.shape[1], out_q.data_ptr(),
                                       ld_q, out_scale.data_ptr(), ld_g, _stream(dev)))


def _new_codes(x):
    """q [B x d] with rows padded to 16 bytes, their stride, and the scales."""
    B, d = x.shape
    ld_q = (d + 15) // 16 * 16
    q = x.new_empty((B, ld_q), dtype=F8)
    return q if d == ld_q else q[:, :d], ld_q, x.new_empty((B, _groups(d)), dtype=torch.float32)


def rmsnorm_fp8(x, weight=None, *, residual=None, eps=1e-6, weight_offset=0.0, want_out=False, stream=None) -> dict:
    """The final norm of hidden states x [B x d] for an fp8 head: "q" [B x d]
    (rows padded to 16 bytes) and "q_scale" [B x ceil(d / 128)]; "residual" (x +
    residual) with a residual, and with want_out the norm in x's type, "out"."""
    ld_x, ld_r = _norm_inputs(x, residual, weight)
    dev = _device(x, residual, weight)
    dt, (B, d) = x.dtype, x.shape
    got = {}
    out = out_residual = None
    with _on(dev, stream):
        if want_out:
            got["out"] = out = x.new_empty((B, d))
        if residual is not None:
            got["residual"] = out_residual = x.new_empty((B, d))
        q, ld_q, scale = _new_codes(x)
        got["q"], got["q_scale"] = q, scale
        check(_abi.load().fh_rmsnorm_fp8(x.data_ptr(), ld_x, _ptr(residual), ld_r, _ptr(weight), _DTYPES[dt], B, d,
                                         eps, weight_offset, _ptr(out), d, _ptr(out_residual), d, q.data_ptr(), ld_q,
                                         scale.data_ptr(), scale.shape[1], _stream(dev)))
    return got


def fp8_quant(x, stream=None) -> dict:
    """Activations x [B x d] as an fp8 product takes them: "q" and "q_scale" as
    rmsnorm_fp8's, without a norm."""
    ld_x, _ = _norm_inputs(x, None, None)
    dev = _device(x)
    with _on(dev, stream):
        q, ld_q, scale = _new_codes(x)
        check(_abi.load().fh_fp8_quant(x.data_ptr(), ld_x, _DTYPES[x.dtype], x.shape[0], x.shape[1], q.data_ptr(),
                                       ld_q, scale.data_ptr(), scale.shape[1], _stream(dev)))
    return {"q": q, "q_scale": scale}


# -------------------------------------------------------- fp8 product and head

# What each handle holds, keyed by its value: (n, k, device).
_WEIGHTS = {}


def _weight(w):
    info = _WEIGHTS.get(_key(w))
    if info is None:
        raise ValueError("unknown fp8 weight (not created by fh_fp8_create, or destroyed)")
    return info


def fh_fp8_create(W: torch.Tensor, stream=None) -> ctypes.c_void_p:
    """Quantise W [n x k] (float32 or bfloat16, contiguous) by blocks of 128 x 128."""
    if W.dim() != 2 or W.dtype not in _DTYPES or not W.is_contiguous():
        raise ValueError("W must be a contiguous [n x k] float32 or bfloat16 matrix")
    dev = _device(W)
    w = ctypes.c_void_p()
    with _on(dev, stream):
        check(_abi.load().fh_fp8_create(W.data_ptr(), _DTYPES[W.dtype], W.shape[0], W.shape[1], _stream(dev),
                                        ctypes.byref(w)))
    _WEIGHTS[w.value] = (W.shape[0], W.shape[1], dev)
    return w


def fh_fp8_create_codes(codes: torch.Tensor, scales: torch.Tensor, stream=None) -> ctypes.c_void_p:
    """Take float8_e4m3fn codes [n x k] and float32 scales [ceil(n / 128) x
    ceil(k / 128)] as they are."""
    if codes.dim() != 2 or codes.dtype is not F8 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous [n x k] float8_e4m3fn matrix")
    n, k = codes.shape
    _shaped(scales, torch.float32, (_groups(n), _groups(k)), "scales")
    if not scales.is_contiguous():
        raise ValueError("scales: must be contiguous")
    dev = _device(codes, scales)
    w = ctypes.c_void_p()
    with _on(dev, stream):
        check(_abi.load().fh_fp8_create_codes(codes.data_ptr(), scales.data_ptr(), n, k, _stream(dev), ctypes.byref(w)))
    _WEIGHTS[w.value] = (n, k, dev)
    return w


def fh_fp8_destroy(w) -> None:
    """Release the weight (None is a no-op); a second time is refused."""
    if _key(w) is None:
        return
    if _WEIGHTS.pop(_key(w), None) is None:
        raise ValueError("unknown fp8 weight (not created by fh_fp8_create, or destroyed)")
    _abi.load().fh_fp8_destroy(w)


def fh_fp8_get(w, codes, scales, stream=None) -> None:
    n, k, dev = _weight(w)
    _shaped(codes, F8, (n, k), "codes")
    _shaped(scales, torch.float32, (_groups(n), _groups(k)), "scales")
    if not codes.is_contiguous() or not scales.is_contiguous():
        raise ValueError("codes and scales must be contiguous")
    if _device(codes, scales) != dev:
        raise ValueError("codes and scales must be on the weight's GPU")
    with _on(dev, stream):
        check(_abi.load().fh_fp8_get(w, codes.data_ptr(), scales.data_ptr(), _stream(dev)))


def _product_args(w, q, q_scale):
    n, k, dev = _weight(w)
    if q.dim() != 2:
        raise ValueError(f"q must be [B x k], got shape {tuple(q.shape)}")
    B = q.shape[0]
    return n, B, _rows(q, F8, (B, k), "q"), _rows(q_scale, torch.float32, (B, _groups(k)), "q_scale"), dev


def fh_fp8_workspace(w, q, forward: bool) -> int:
    """Bytes of workspace of a product (or, with forward, head) call on q."""
    _, k, _ = _weight(w)
    ld_q = _rows(q, F8, (q.shape[0], k), "q")
    return _size(_abi.load().fh_fp8_workspace(w, q.data_ptr(), ld_q, q.shape[0], int(forward)))


def fh_fp8_matmul(w, q, q_scale, out, workspace=None, stream=None) -> None:
    n, B, ld_q, ld_g, dev = _product_args(w, q, q_scale)
    if out.dtype not in _DTYPES:
        raise ValueError("out must be float32 or bfloat16")
    ld_out = _rows(out, out.dtype, (B, n), "out")
    ws, ws_bytes = _workspace_arg(workspace)
    if _device(q, q_scale, out, workspace) != dev:
        raise ValueError("tensors must be on the weight's GPU")
    with _on(dev, stream):
        check(_abi.load().fh_fp8_matmul(w, q.data_ptr(), ld_q, q_scale.data_ptr(), ld_g, B, out.data_ptr(), ld_out,
                                        _DTYPES[out.dtype], ws, ws_bytes, _stream(dev)))


def fh_fp8_matmul_native(w, q, q_scale, out, workspace=None, stream=None) -> None:
    """fh_fp8_matmul with bfloat16 results and fewer bits in its sums (FP8Head.matmul's native)."""
    n, B, ld_q, ld_g, dev = _product_args(w, q, q_scale)
    ld_out = _rows(out, torch.bfloat16, (B, n), "out")
    ws, ws_bytes = _workspace_arg(workspace)
    if _device(q, q_scale, out, workspace) != dev:
        raise ValueError("tensors must be on the weight's GPU")
    with _on(dev, stream):
        check(_abi.load().fh_fp8_matmul_native(w, q.data_ptr(), ld_q, q_scale.data_ptr(), ld_g, B, out.data_ptr(),
                                               ld_out, ws, ws_bytes, _stream(dev)))


def fh_fp8_forward(w, q, q_scale, mode, temperature, seed, out_token, out_token_logit=None, out_lse=None,
                   out_logits=None, workspace=None, stream=None) -> None:
    n, B, ld_q, ld_g, dev = _product_args(w, q, q_scale)
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
        check(_abi.load().fh_fp8_forward(w, q.data_ptr(), ld_q, q_scale.data_ptr(), ld_g, B, mode, temperature, seed,
                                         out_token.data_ptr(), _ptr(out_token_logit), _ptr(out_lse), _ptr(out_logits),
                                         ld_out, ws, ws_bytes, _stream(dev)))


class FP8Head(_Steps):
    """A dense head (or any linear layer) with weights and activations in 8-bit
    floating point: E quantised here by blocks of 128 x 128, or float8_e4m3fn
    codes and their scales as they are."""

    def __init__(self, E: torch.Tensor = None, *, codes: torch.Tensor = None, scales: torch.Tensor = None,
                 stream=None):
        self.w = None
        if (E is None) == (codes is None) or (codes is None) != (scales is None):
            raise ValueError("give either E, or codes and scales")
        if E is not None:
            self.w = fh_fp8_create(E, stream)
        else:
            self.w = fh_fp8_create_codes(codes, scales, stream)
        self.n, self.k, self.device = _weight(self.w)

    def close(self):
        w, self.w = self.w, None
        fh_fp8_destroy(w)

    def __del__(self):
        # not while the interpreter shuts down (see FlashHead)
        if sys is None or sys.is_finalizing():
            return
        try:
            self.close()
        except Exception:
            pass

    def _inputs(self, q, q_scale, forward):
        """Row strides, workspace size of a call on q; all on the weight's GPU."""
        _, B, ld_q, ld_g, dev = _product_args(self.w, q, q_scale)
        if _device(q, q_scale) != dev:
            raise ValueError("tensors must be on the weight's GPU")
        return ld_q, ld_g, _size(_abi.load().fh_fp8_workspace(self.w, q.data_ptr(), ld_q, B, forward))

    def _states(self, x, weight, residual, eps, weight_offset):
        h = rmsnorm_fp8(x, weight, residual=residual, eps=eps, weight_offset=weight_offset)
        return h["q"], h["q_scale"]

    def codes(self, stream=None):
        """The codes [n x k] and scales [ceil(n / 128) x ceil(k / 128)]."""
        with _on(self.device, stream):
            codes = torch.empty((self.n, self.k), dtype=F8, device=self.device)
            scales = torch.empty((_groups(self.n), _groups(self.k)), dtype=torch.float32, device=self.device)
            fh_fp8_get(self.w, codes, scales)
        return codes, scales

    def matmul(self, q: torch.Tensor, q_scale: torch.Tensor, dtype=torch.float32, stream=None, *,
               native: bool = False) -> torch.Tensor:
        """[B x n] = q code^T under both scales, in float32 or bfloat16; q and
        q_scale as rmsnorm_fp8 and fp8_quant give them.  Products are exact, sums in
        float32.  native (bfloat16): large calls take the matrix cores' own fp8
        product (4096 x 10240 x 2560: 103 us for 190), whose sums of eight products keep 13 binades
        below the largest: results may be off by 2^-10 of the sum of their products'
        magnitudes, codes below 2^-6 counted as 2^-6 (1.5e-5 of normally distributed codes' results, all of one whose
        products cancel), and by as much with the batch that a token is in."""
        ld_q, ld_g, size = self._inputs(q, q_scale, 0)
        if dtype not in _DTYPES:
            raise ValueError("dtype must be float32 or bfloat16")
        if native and dtype is not torch.bfloat16:
            raise ValueError("native products are bfloat16")
        B = q.shape[0]
        with _on(self.device, stream):
            out = q.new_empty((B, self.n), dtype=dtype)
            ws = q.new_empty((size,), dtype=torch.uint8) if size else None
            if native:
                check(_abi.load().fh_fp8_matmul_native(self.w, q.data_ptr(), ld_q, q_scale.data_ptr(), ld_g, B,
                                                       out.data_ptr(), self.n, _ptr(ws), size, _stream(self.device)))
            else:
                check(_abi.load().fh_fp8_matmul(self.w, q.data_ptr(), ld_q, q_scale.data_ptr(), ld_g, B,
                                                out.data_ptr(), self.n, _DTYPES[dtype], _ptr(ws), size,
                                                _stream(self.device)))
        return out

    def forward(self, q: torch.Tensor, q_scale: torch.Tensor, mode: int = 0, temperature: float = 1.0,
                seed: int = 0, want_logits: bool = False, stream=None) -> dict:
        """FlashHead.dense on fp8 operands: "token", "token_logit", "lse" and with
        want_logits "logits" [B x n]."""
        ld_q, ld_g, size = self._inputs(q, q_scale, 1)
        B = q.shape[0]
        with _on(self.device, stream):
            token, logit, lse, ws = _choice_outputs(q, B, size)
            out = {"token": token, "token_logit": logit, "lse": lse}
            logits = None
            if want_logits:
                out["logits"] = logits = q.new_empty((B, self.n), dtype=torch.float32)
            check(_abi.load().fh_fp8_forward(self.w, q.data_ptr(), ld_q, q_scale.data_ptr(), ld_g, B, mode,
                                             temperature, seed, token.data_ptr(), logit.data_ptr(), lse.data_ptr(),
                                             _ptr(logits), self.n, _ptr(ws), size, _stream(self.device)))
        return out
