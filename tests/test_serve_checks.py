"""What the norm, the int8 product and the rules on logits refuse: through the
C ABI (nothing is launched: argument errors come first) and through the
binding (shapes, types and placement, before the library is called).  CPU
only; and the float64 definitions' own pins."""

import ctypes

import numpy as np
import pytest
import torch

from lm_output_head_amd import _abi, serve
from oracle import serve_oracle

P = ctypes.c_void_p
A = P(1 << 20)  # an address that is never read


@pytest.fixture(scope="module")
def lib():
    import os
    if not os.path.exists(_abi.lib_path()):
        from lm_output_head_amd.build import build
        build()
    return _abi.load()


def _refused(lib, status, needle):
    assert status < 0 and needle in lib.fh_last_error().decode(), (status, lib.fh_last_error())


NORM = dict(x=A, ld_x=64, residual=A, ld_residual=64, weight=A, dtype=1, B=4, d=64, eps=1e-6, offset=0.0, out=A,
            ld_out=64, out_residual=A, ld_out_residual=64, q=A, ld_q=64, scale=A, stream=None)


@pytest.mark.parametrize("kw,needle", [
    ({"x": None}, "x is NULL"),
    ({"dtype": 5}, "dtype"),
    ({"out": None, "out_residual": None, "q": None, "scale": None}, "no output"),
    ({"scale": None}, "go together"),
    ({"q": None}, "go together"),
    ({"B": 0}, "B outside"),
    ({"B": 1 << 31}, "B outside"),
    ({"d": 0}, "d outside"),
    ({"ld_x": 63}, "ld_x=63"),
    ({"ld_residual": 0}, "ld_residual"),
    ({"ld_out": 63}, "ld_out"),
    ({"ld_out_residual": -64}, "ld_out_residual"),
    ({"ld_q": 60}, "ld_q"),
    ({"ld_x": 1 << 62}, "too large"),
    ({"eps": -1e-6}, "eps"),
    ({"eps": float("nan")}, "eps"),
    ({"offset": float("inf")}, "weight_offset"),
    ({"x": P((1 << 20) + 1)}, "aligned"),
    ({"weight": P((1 << 20) + 1)}, "aligned"),
    ({"dtype": 0, "out": P((1 << 20) + 2)}, "aligned"),
    ({"scale": P((1 << 20) + 2)}, "aligned"),
    ({}, "out and out_residual are the same storage"),
    ({"out_residual": None, "ld_out": 65}, "ld_out and ld_x differ"),
    ({"out": None, "x": P(1 << 21), "ld_residual": 70}, "ld_out_residual and ld_residual differ"),
])
def test_norm_refusals(lib, kw, needle):
    _refused(lib, lib.fh_rmsnorm(*dict(NORM, **kw).values()), needle)


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
    _refused(lib, lib.fh_w8a8_create(*args, None, ctypes.byref(out)), needle)
    assert not out.value


def test_weight_from_codes_and_null_handles(lib):
    out = P()
    _refused(lib, lib.fh_w8a8_create_codes(None, A, 8, 64, None, ctypes.byref(out)), "must not be NULL")
    _refused(lib, lib.fh_w8a8_create_codes(A, None, 8, 64, None, ctypes.byref(out)), "must not be NULL")
    _refused(lib, lib.fh_w8a8_create_codes(A, P((1 << 20) + 2), 8, 64, None, ctypes.byref(out)), "aligned")
    _refused(lib, lib.fh_w8a8_create_codes(A, A, 8, 64, None, None), "out is NULL")
    _refused(lib, lib.fh_w8a8_matmul(None, A, 64, A, 1, A, 8, 0, None, 0, None), "w is NULL")
    _refused(lib, lib.fh_w8a8_forward(None, A, 64, A, 1, 0, 1.0, 0, A, None, None, None, 0, None, 0, None), "w is NULL")
    _refused(lib, lib.fh_w8a8_workspace(None, A, 64, 1, 0), "w is NULL")
    _refused(lib, lib.fh_w8a8_get(None, A, A, None), "w is NULL")
    lib.fh_w8a8_destroy(None)


def _rules(**kw):
    base = dict(history=A.value, ld_history=10, history_len=10, n_prompt=None, n_history=None, repetition=None,
                frequency=None, presence=None, bias_ids=None, bias=None, ld_bias=0, bias_len=0, n_bias=None, mask=None,
                ld_mask=0, mask_rows=0, mask_row=None)
    return _abi.FhLogitRules(**dict(base, **kw))


CALL = dict(z=A, ld=100, ids=None, ld_ids=0, B=3, n=100, v=100, rules=None, mode=0, T=1.0, seed=0, out=A, ld_out=100,
            token=A, logit=None, lse=None, ws=A, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,needle", [
    ({"z": None}, "logits is NULL"),
    ({"B": 0}, "B outside"),
    ({"B": 65536}, "B outside"),
    ({"n": 0, "v": 0}, "n and v"),
    ({"v": 101}, "n = v"),
    ({"out": None, "token": None}, "no output"),
    ({"ld_out": 104}, "differ on the same storage"),
    ({"mode": 1}, "mode"),
    ({"mode": 4}, "mode"),
    ({"mode": 2, "T": 0.0}, "temperature"),
    ({"mode": 2, "T": float("nan")}, "temperature"),
    ({"ld": 99}, "ld_logits"),
    ({"ids": A, "ld_ids": 99}, "ld_ids"),
    ({"ld_out": 99}, "ld_out"),
    ({"z": P((1 << 20) + 2)}, "aligned"),
    ({"ws": None, "n": 20000, "v": 20000, "ld": 20000, "ld_out": 20000}, "workspace"),
    ({"ws_bytes": 8, "n": 20000, "v": 20000, "ld": 20000, "ld_out": 20000}, "workspace"),
    ({"ws": P((1 << 20) + 4), "n": 20000, "v": 20000, "ld": 20000, "ld_out": 20000}, "16-byte aligned"),
    ({"rules": {"ld_history": 9}}, "ld_history"),
    ({"rules": {"history_len": -1}}, "history_len"),
    ({"rules": {"history_len": (1 << 30) + 1, "ld_history": 1 << 31}}, "history_len"),
    ({"rules": {"history": None, "n_history": A.value}}, "need a history"),
    ({"rules": {"bias": A.value}}, "go together"),
    ({"rules": {"bias": A.value, "bias_ids": A.value, "bias_len": 4, "ld_bias": 3}}, "ld_bias"),
    ({"rules": {"bias": A.value, "bias_ids": A.value, "bias_len": -4}}, "bias_len"),
    ({"rules": {"n_bias": A.value}}, "n_bias"),
    ({"rules": {"mask": A.value, "mask_rows": 0}}, "mask_rows"),
    ({"rules": {"mask": A.value, "mask_rows": 2, "ld_mask": 4}}, "fewer rows"),
    ({"rules": {"mask": A.value, "mask_rows": 3, "ld_mask": 3}}, "ld_mask"),
    ({"rules": {"mask_row": A.value}}, "mask_row needs"),
    ({"rules": {"repetition": (1 << 20) + 2}}, "aligned"),
])
def test_rules_refusals(lib, kw, needle):
    kw = dict(kw)
    if "rules" in kw:
        kw["rules"] = ctypes.byref(_rules(**kw["rules"]))
    _refused(lib, lib.fh_logits_apply(*dict(CALL, **kw).values()), needle)


def test_workspace_sizes(lib):
    assert lib.fh_logits_workspace(3, 20000) > 0
    assert lib.fh_logits_workspace(3, 100) == 0
    for B, n in [(0, 10), (65536, 10), (1, 0), (1, (1 << 30) + 1)]:
        _refused(lib, lib.fh_logits_workspace(B, n), "outside")


# ------------------------------------------------------------------ binding

def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("kw,needle", [
    ({"x": torch.zeros(2, 8, dtype=torch.float16)}, "x must be"),
    ({"x": bf(8)}, "x must be"),
    ({"residual": bf(2, 7)}, "residual: expected"),
    ({"residual": torch.zeros(2, 8)}, "residual: expected"),
    ({"weight": bf(7)}, "weight: expected"),
    ({"weight": bf(16)[::2]}, "weight: must be contiguous"),
    ({"out": bf(3, 8)}, "out: expected"),
    ({"out": bf(8, 2).t()}, "elements of a row"),
    ({"out": bf(1, 8).expand(2, 8)}, "rows must not overlap"),
    ({"out_q": torch.zeros(2, 8, dtype=torch.int8)}, "go together"),
    ({"out_q": torch.zeros(2, 8, dtype=torch.uint8), "out_scale": torch.zeros(2)}, "out_q: expected"),
    ({"out_q": torch.zeros(2, 8, dtype=torch.int8), "out_scale": torch.zeros(1)}, "out_scale: expected"),
    ({"out": bf(2, 8)}, "one GPU"),
])
def test_binding_norm_refusals(kw, needle):
    args = dict(dict(x=bf(2, 8), residual=None, weight=None, eps=1e-6, weight_offset=0.0), **kw)
    with pytest.raises(ValueError, match=needle):
        serve.fh_rmsnorm(**args)


@pytest.fixture
def weight():
    serve._WEIGHTS[0x5EED] = (12, 16, torch.device("cpu"))
    yield 0x5EED
    serve._WEIGHTS.pop(0x5EED, None)


def test_binding_product_refusals(weight):
    q, s = torch.zeros(2, 16, dtype=torch.int8), torch.zeros(2)
    tok = torch.zeros(2, dtype=torch.int32)
    for args, needle in [
        ((0xBAD, q, s, torch.zeros(2, 12)), "unknown int8 weight"),
        ((weight, q[:, :15], s, torch.zeros(2, 12)), "q: expected"),
        ((weight, q[0], s, torch.zeros(2, 12)), r"q must be \[B x k\]"),
        ((weight, q.float(), s, torch.zeros(2, 12)), "q: expected"),
        ((weight, q, s[:1], torch.zeros(2, 12)), "q_scale: expected"),
        ((weight, q, s, torch.zeros(2, 11)), "out: expected"),
        ((weight, q, s, torch.zeros(2, 12, dtype=torch.float16)), "float32 or bfloat16"),
        ((weight, q, s, torch.zeros(2, 12)), "one GPU"),
    ]:
        with pytest.raises(ValueError, match=needle):
            serve.fh_w8a8_matmul(*args)
    for kw, needle in [({"out_token": tok[:1]}, "out_token"), ({"out_lse": s.double()}, "out_lse"),
                       ({"out_logits": torch.zeros(2, 13)}, "out_logits"),
                       ({"workspace": torch.zeros(8)}, "workspace")]:
        with pytest.raises(ValueError, match=needle):
            serve.fh_w8a8_forward(weight, q, s, 0, 1.0, 0, **dict({"out_token": tok}, **kw))
    with pytest.raises(ValueError, match="either E"):
        serve.W8A8Head()
    with pytest.raises(ValueError, match="either E"):
        serve.W8A8Head(torch.zeros(2, 2), codes=q, scales=s)
    with pytest.raises(ValueError, match="codes must be"):
        serve.W8A8Head(codes=q.float(), scales=s)
    with pytest.raises(ValueError, match="scales: expected"):
        serve.W8A8Head(codes=q, scales=s[:1])
    with pytest.raises(ValueError, match="one GPU"):
        serve.W8A8Head(codes=q, scales=s)


def test_binding_destroys_a_weight_once(monkeypatch):
    """A handle is freed memory after its release: another one is refused
    before the library sees it, through the function or a head that holds it."""
    freed = []

    class Library:
        def fh_w8a8_destroy(self, w):
            freed.append(w)

    monkeypatch.setattr(_abi, "load", Library)
    serve._WEIGHTS[0x5EED] = (12, 16, torch.device("cpu"))
    head = object.__new__(serve.W8A8Head)
    head.w = 0x5EED
    serve.fh_w8a8_destroy(0x5EED)
    with pytest.raises(ValueError, match="unknown int8 weight"):
        serve.fh_w8a8_destroy(0x5EED)
    with pytest.raises(ValueError, match="unknown int8 weight"):
        head.close()
    head.close()  # holds nothing any more
    serve.fh_w8a8_destroy(None)
    serve.fh_w8a8_destroy(ctypes.c_void_p())
    assert freed == [0x5EED]


@pytest.mark.parametrize("kw,needle", [
    ({"history": torch.zeros(2, 5)}, "history: expected"),
    ({"history": torch.zeros(5, dtype=torch.int32)}, "history must be"),
    ({"n_history": torch.zeros(2, dtype=torch.int32)}, "need a history"),
    ({"history": torch.zeros(2, 5, dtype=torch.int32), "repetition": torch.zeros(3)}, "repetition: expected"),
    ({"history": torch.zeros(2, 5, dtype=torch.int32), "n_prompt": torch.zeros(2)}, "n_prompt: expected"),
    ({"bias": torch.zeros(2, 3)}, "go together"),
    ({"n_bias": torch.zeros(2, dtype=torch.int32)}, "bias_ids and bias go together"),
    ({"bias": torch.zeros(2, 3), "bias_ids": torch.zeros(2, 4, dtype=torch.int32)}, "bias_ids: expected"),
    ({"bias": torch.zeros(2, 3), "bias_ids": torch.zeros(2, 6, dtype=torch.int32)[:, :3]}, "same row stride"),
    ({"mask": torch.zeros(2, 3, dtype=torch.int32)}, "mask: expected"),
    ({"mask_row": torch.zeros(2, dtype=torch.int32)}, "mask_row needs"),
    ({"mask": torch.zeros(2, 4, dtype=torch.int32)}, "one GPU"),
    ({"mask": torch.zeros(1, 4, dtype=torch.int32), "history": torch.zeros(2, 5, dtype=torch.int32)}, "fewer rows"),
])
def test_binding_rules_refusals(kw, needle):
    with pytest.raises(ValueError, match=needle):
        serve.LogitRules(100, **kw)


def test_binding_lists_of_one_row_have_any_stride():
    """One row's stride says nothing (refused here for its place alone)."""
    ids = torch.zeros(1, 40, dtype=torch.int32)[:, 3:6]
    for bias in (torch.ones(1, 3), torch.ones(1, 60)[:, :3]):
        with pytest.raises(ValueError, match="one GPU"):
            serve.LogitRules(50, bias_ids=ids, bias=bias)


def test_binding_empty_lists_have_any_stride():
    ids = torch.zeros(3, 40, dtype=torch.int32)[:, :0]
    for bias in (torch.ones(3, 0), torch.ones(3, 60)[:, :0]):
        with pytest.raises(ValueError, match="one GPU"):
            serve.LogitRules(50, bias_ids=ids, bias=bias)


def test_binding_apply_refusals():
    z = torch.zeros(2, 100)
    none = serve.LogitRules(100)
    for kw, needle in [({"logits": z.double()}, "logits: expected"), ({"logits": z[0]}, "logits must be"),
                       ({"ids": torch.zeros(2, 99, dtype=torch.int32)}, "ids: expected"),
                       ({"out_logits": torch.zeros(2, 99)}, "out_logits: expected"),
                       ({"v": 101}, "rules are of"),
                       ({"out_token": torch.zeros(2)}, "out_token: expected"),
                       ({"out_token": torch.zeros(2, dtype=torch.int32)}, "one GPU")]:
        args = dict(dict(logits=z, ids=None, v=100, rules=none, mode=0, temperature=1.0, seed=0), **kw)
        with pytest.raises(ValueError, match=needle):
            serve.fh_logits_apply(**args)


def test_binding_ids_without_rules_need_the_number_of_tokens():
    """The candidates' number says nothing about the vocabulary: taken for it,
    every id at or above it would be no token."""
    z, ids = torch.zeros(2, 8), torch.full((2, 8), 5000, dtype=torch.int32)
    with pytest.raises(ValueError, match="ids without rules need v"):
        serve.logits_apply(z, ids=ids)
    for kw in ({"v": 10000}, {"rules": serve.LogitRules(10000)}):
        with pytest.raises(ValueError, match="one GPU"):
            serve.logits_apply(z, ids=ids, **kw)


# ------------------------------------------------------------ definitions' pins

def test_oracle_rules_by_hand():
    z = np.array([[2.0, -2.0, 1.0, 0.5, 3.0, np.nan]])
    hist = np.array([[0, 1, 1, 3, 3, 9, -1, 4]])  # prompt 0 1 1; output 3 3; 4 does not count
    mask = np.array([[0b011111]], np.int32)
    got, _ = serve_oracle.apply_rules(
        z, None, 6, history=hist, n_prompt=[3], n_history=[7], repetition=[2.0], frequency=[0.25], presence=[0.5],
        bias_ids=np.array([[2, 2, 4, 7]]), bias=np.array([[1.0, 2.0, -np.inf, 5.0]]), mask=mask)
    assert got.tolist() == [[1.0, -4.0, 4.0, 0.25 - 0.5 - 0.5, -np.inf, -np.inf]]
    assert serve_oracle.lse(np.full((1, 3), -np.inf), 1.0)[0] == -np.inf


def test_oracle_norm_and_product_by_hand():
    y, s = serve_oracle.rmsnorm([[3.0, 4.0]], [[1.0, -1.0]], [1.0, 2.0], 0.0, 1.0)
    assert s.tolist() == [[4.0, 3.0]] and np.allclose(y, np.array([[8.0, 9.0]]) / np.sqrt(12.5))
    assert serve_oracle.product([[1, -2]], [0.5], [[3, 4], [-128, 127]], [1.0, 2.0]).tolist() == [[-2.5, -382.0]]


def test_the_current_device_is_torchs(monkeypatch):
    """A call on the current GPU changes no device, one on another does: by
    torch.cuda.current_device and torch.cuda.device, as a program may replace them."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: ("device", dev))
    assert serve._on(torch.device("cuda", 3), None) is serve._SAME
    assert serve._on(torch.device("cuda", 1), None) == ("device", torch.device("cuda", 1))
