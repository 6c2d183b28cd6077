"""What the fp8 operators refuse: through the C ABI (nothing is launched: argument
errors come first) and through the binding; and the float64 definitions' own pins.
CPU only."""

import ctypes

import numpy as np
import pytest
import torch

from lm_output_head_amd import _abi, fp8
from oracle import fp8_oracle

P = ctypes.c_void_p
A = P(1 << 20)  # an address that is never read
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_abi.lib_path()):
        from lm_output_head_amd.build import build
        build()
    return _abi.load()


def _refused(lib, status, needle):
    assert status < 0 and needle in lib.fh_last_error().decode(), (status, lib.fh_last_error())


# ---------------------------------------------------------------- definitions

def test_codes_are_torchs():
    """The oracle's values and rounding against torch's conversion on the CPU."""
    codes = torch.arange(256, dtype=torch.int16).to(torch.uint8)
    want = codes.view(F8).double().numpy()
    assert np.array_equal(fp8_oracle.e4m3_values(), want, equal_nan=True)
    rng = np.random.default_rng(1)
    grid = fp8_oracle.e4m3_values()[:127]
    t = np.concatenate([grid, -grid, (grid[1:] + grid[:-1]) / 2, -(grid[1:] + grid[:-1]) / 2,
                        rng.normal(size=4000) * np.exp(rng.uniform(-12, 4, 4000))]).astype(np.float32)
    t = t[np.abs(t) <= 448]
    assert np.array_equal(fp8_oracle.e4m3_encode(t), torch.from_numpy(t).to(F8).view(torch.uint8).numpy())


def test_definitions_by_hand():
    y = np.zeros((1, 130), np.float32)
    y[0, :3] = (448, -224, 1)
    y[0, 128:] = (0.5, -0.25)
    codes, scales = fp8_oracle.quant(y)
    assert np.allclose(scales, [[1, 0.5 / 448]], rtol=1e-7)
    v = fp8_oracle.e4m3_values()[codes]
    assert v[0, :3].tolist() == [448, -224, 1] and v[0, 128:].tolist() == [448, -224]
    out, size = fp8_oracle.product(codes, scales, codes, scales[:, :])
    assert abs(out[0, 0] - (448 ** 2 + 224 ** 2 + 1 + 0.5 ** 2 + 0.25 ** 2)) < 1e-3 and size[0, 0] == out[0, 0]


# ---------------------------------------------------------------------- C ABI

NORM = dict(x=A, ld_x=200, residual=A, ld_residual=200, weight=A, dtype=1, B=4, d=200, eps=1e-6, offset=0.0, out=A,
            ld_out=200, out_residual=P(1 << 21), ld_out_residual=200, q=A, ld_q=200, scale=A, ld_scale=2, stream=None)


@pytest.mark.parametrize("kw,needle", [
    ({"x": None}, "x is NULL"),
    ({"dtype": 5}, "dtype"),
    ({"q": None}, "must not be NULL"),
    ({"scale": None}, "must not be NULL"),
    ({"B": 0}, "B outside"),
    ({"B": 1 << 31}, "B outside"),
    ({"d": 0}, "d outside"),
    ({"ld_x": 199}, "ld_x=199"),
    ({"ld_residual": 0}, "ld_residual"),
    ({"ld_out": 199}, "ld_out"),
    ({"ld_out_residual": -200}, "ld_out_residual"),
    ({"ld_q": 199}, "ld_q"),
    ({"ld_scale": 1}, "ld_scale=1"),
    ({"ld_x": 1 << 62}, "too large"),
    ({"eps": -1e-6}, "eps"),
    ({"eps": float("nan")}, "eps"),
    ({"offset": float("inf")}, "weight_offset"),
    ({"x": P((1 << 20) + 1)}, "aligned"),
    ({"weight": P((1 << 20) + 1)}, "aligned"),
    ({"scale": P((1 << 20) + 2)}, "aligned"),
    ({"out_residual": A}, "same storage"),
    ({"out": None, "x": P(1 << 21), "ld_residual": 210, "residual": P(1 << 22), "ld_out_residual": 220},
     "ld_out_residual and ld_x differ"),
])
def test_norm_refusals(lib, kw, needle):
    _refused(lib, lib.fh_rmsnorm_fp8(*dict(NORM, **kw).values()), needle)


@pytest.mark.parametrize("args,needle", [
    ((None, 64, 1, 4, 64, A, 64, A, 1), "x is NULL"),
    ((A, 64, 2, 4, 64, A, 64, A, 1), "dtype"),
    ((A, 63, 1, 4, 64, A, 64, A, 1), "ld_x=63"),
    ((A, 64, 1, 4, 64, None, 64, A, 1), "must not be NULL"),
    ((A, 64, 1, 4, 64, A, 63, A, 1), "ld_q"),
    ((A, 129, 1, 4, 129, A, 129, A, 1), "ld_scale"),
    ((A, 64, 1, 0, 64, A, 64, A, 1), "B outside"),
    ((P((1 << 20) + 2), 64, 0, 4, 64, A, 64, A, 1), "aligned"),
])
def test_quant_refusals(lib, args, needle):
    _refused(lib, lib.fh_fp8_quant(*args, None), needle)


@pytest.mark.parametrize("args,needle", [
    ((None, 1, 8, 64), "W is NULL"),
    ((A, 3, 8, 64), "dtype"),
    ((P((1 << 20) + 1), 1, 8, 64), "aligned"),
    ((A, 1, 0, 64), "n outside"),
    ((A, 1, (1 << 27) + 1, 64), "n outside"),
    ((A, 1, 8, 0), "k outside"),
    ((A, 1, 8, 1 << 17), "k outside"),
])
def test_weight_refusals(lib, args, needle):
    out = P()
    _refused(lib, lib.fh_fp8_create(*args, None, ctypes.byref(out)), needle)
    assert not out.value


def test_weight_from_codes_and_null_handles(lib):
    out = P()
    _refused(lib, lib.fh_fp8_create_codes(None, A, 8, 64, None, ctypes.byref(out)), "must not be NULL")
    _refused(lib, lib.fh_fp8_create_codes(A, None, 8, 64, None, ctypes.byref(out)), "must not be NULL")
    _refused(lib, lib.fh_fp8_create_codes(A, P((1 << 20) + 2), 8, 64, None, ctypes.byref(out)), "aligned")
    _refused(lib, lib.fh_fp8_create_codes(A, A, 8, 64, None, None), "out is NULL")
    _refused(lib, lib.fh_fp8_matmul(None, A, 64, A, 1, 1, A, 8, 0, None, 0, None), "w is NULL")
    _refused(lib, lib.fh_fp8_forward(None, A, 64, A, 1, 1, 0, 1.0, 0, A, None, None, None, 0, None, 0, None), "w is NULL")
    _refused(lib, lib.fh_fp8_workspace(None, A, 64, 1, 0), "w is NULL")
    _refused(lib, lib.fh_fp8_get(None, A, A, None), "w is NULL")
    lib.fh_fp8_destroy(None)


# -------------------------------------------------------------------- binding

def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f8(*shape):
    return torch.zeros(shape).to(F8)


@pytest.mark.parametrize("kw,needle", [
    ({"x": torch.zeros(2, 8, dtype=torch.float16)}, "x must be"),
    ({"x": bf(8)}, "x must be"),
    ({"residual": bf(2, 7)}, "residual: expected"),
    ({"weight": bf(16)[::2]}, "weight: must be contiguous"),
    ({"out": bf(3, 8)}, "out: expected"),
    ({"out_q": torch.zeros(2, 8, dtype=torch.uint8)}, "out_q: expected"),
    ({"out_q": f8(2, 9)}, "out_q: expected"),
    ({"out_scale": torch.zeros(2)}, "out_scale: expected"),
    ({"out_scale": torch.zeros(2, 2)}, "out_scale: expected"),
    ({}, "one GPU"),
])
def test_binding_norm_refusals(kw, needle):
    args = dict(dict(x=bf(2, 8), residual=None, weight=None, eps=1e-6, weight_offset=0.0, out_q=f8(2, 8),
                     out_scale=torch.zeros(2, 1)), **kw)
    with pytest.raises(ValueError, match=needle):
        fp8.fh_rmsnorm_fp8(**args)


def test_binding_quant_refusals():
    for x, q, s, needle in [(bf(2, 8).half(), f8(2, 8), torch.zeros(2, 1), "x must be"),
                            (bf(2, 8), f8(2, 7), torch.zeros(2, 1), "out_q"),
                            (bf(2, 200), f8(2, 200), torch.zeros(2, 1), "out_scale"),
                            (bf(2, 8), f8(2, 8), torch.zeros(2, 1), "one GPU")]:
        with pytest.raises(ValueError, match=needle):
            fp8.fh_fp8_quant(x, q, s)


@pytest.fixture
def weight():
    fp8._WEIGHTS[0x5EED] = (12, 200, torch.device("cpu"))
    yield 0x5EED
    fp8._WEIGHTS.pop(0x5EED, None)


def test_binding_product_refusals(weight):
    q, s = f8(2, 200), torch.zeros(2, 2)
    tok = torch.zeros(2, dtype=torch.int32)
    for args, needle in [
        ((0xBAD, q, s, torch.zeros(2, 12)), "unknown fp8 weight"),
        ((weight, q[:, :199], s, torch.zeros(2, 12)), "q: expected"),
        ((weight, q[0], s, torch.zeros(2, 12)), r"q must be \[B x k\]"),
        ((weight, torch.zeros(2, 200, dtype=torch.int8), s, torch.zeros(2, 12)), "q: expected"),
        ((weight, q, s[:, :1], torch.zeros(2, 12)), "q_scale: expected"),
        ((weight, q, s[0], torch.zeros(2, 12)), "q_scale: expected"),
        ((weight, q, s, torch.zeros(2, 11)), "out: expected"),
        ((weight, q, s, torch.zeros(2, 12, dtype=torch.float16)), "float32 or bfloat16"),
        ((weight, q, s, torch.zeros(2, 12)), "one GPU"),
    ]:
        with pytest.raises(ValueError, match=needle):
            fp8.fh_fp8_matmul(*args)
    for kw, needle in [({"out_token": tok[:1]}, "out_token"), ({"out_lse": torch.zeros(2).double()}, "out_lse"),
                       ({"out_logits": torch.zeros(2, 13)}, "out_logits"),
                       ({"workspace": torch.zeros(8)}, "workspace")]:
        with pytest.raises(ValueError, match=needle):
            fp8.fh_fp8_forward(weight, q, s, 0, 1.0, 0, **dict({"out_token": tok}, **kw))
    with pytest.raises(ValueError, match="either E"):
        fp8.FP8Head()
    with pytest.raises(ValueError, match="either E"):
        fp8.FP8Head(torch.zeros(2, 2), codes=q, scales=s)
    with pytest.raises(ValueError, match="float8_e4m3fn"):
        fp8.FP8Head(codes=torch.zeros(2, 200), scales=torch.zeros(1, 2))
    with pytest.raises(ValueError, match="scales: expected"):
        fp8.FP8Head(codes=q, scales=torch.zeros(2, 2))
    with pytest.raises(ValueError, match="scales: must be contiguous"):
        fp8.FP8Head(codes=f8(200, 200), scales=torch.zeros(2, 2).t())


def test_native_product_refusals(lib, weight):
    _refused(lib, lib.fh_fp8_matmul_native(None, A, 64, A, 1, 1, A, 8, None, 0, None), "w is NULL")
    q, s = f8(2, 200), torch.zeros(2, 2)
    for out, needle in [(torch.zeros(2, 12), "out: expected"), (bf(2, 11), "out: expected"), (bf(2, 12), "one GPU")]:
        with pytest.raises(ValueError, match=needle):
            fp8.fh_fp8_matmul_native(weight, q, s, out)
    head = fp8.FP8Head.__new__(fp8.FP8Head)
    head.w, head.n, head.k, head.device = None, 12, 200, torch.device("cpu")
    head._inputs = lambda *a: (200, 2, 0)
    with pytest.raises(ValueError, match="native products are bfloat16"):
        head.matmul(q, s, native=True)
