"""GPU parity of fh_rmsnorm against the float64 definition.

Tolerances, u = 2^-24 (float32's half step): s = x + r rounds once (u).  The sum
of squares is of positive terms: with at least 64 lanes a term goes through at
most d / 64 + 16 roundings, of which the root halves the effect.  The mean, eps,
the root, the reciprocal, its product with s, offset + w and its product round
at most once each, s itself once more: 10 u.  So y is within
(d / 128 + 20) u of itself; a bfloat16 output adds 2^-8.  Where offset + w
cancels, its rounding is relative to the result, so nothing is added.  The scale
is max |y| / 127 (u more); a code is off by half a step plus 127 times y's and
the scale's relative errors and the division's."""

import numpy as np
import pytest
import torch

from oracle import serve_oracle

from _gpu import need_gpu, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    from lm_output_head_amd import load_library
    load_library()


def f64(t):
    return t.double().cpu().numpy()


def check(x, r, w, eps, off, got):
    B, d = x.shape
    y, s = serve_oracle.rmsnorm(f64(x), None if r is None else f64(r), None if w is None else f64(w), eps, off)
    rel = (d / 128 + 20) * U
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 0.0
    if "out" in got:
        assert got["out"].dtype == x.dtype
        assert np.all(np.abs(f64(got["out"]) - y) <= (rel + half * (1 + rel)) * np.abs(y) + 1e-38)
    if r is not None and "residual" in got:
        assert np.all(np.abs(f64(got["residual"]) - s) <= (U + half * (1 + U)) * np.abs(s))
    if "q" in got:
        q, sc = f64(got["q"]), f64(got["q_scale"])
        want = np.abs(y).max(1) / 127
        assert np.all(np.abs(sc - want) <= (rel + U) * want + 1e-38)
        assert q.min() >= -127 and q.max() <= 127
        step = np.where(sc > 0, sc, 1.0)[:, None]
        assert np.all(np.abs(q - y / step) <= 0.5 + 128 * (2 * rel + 2 * U))
        assert np.all(q[sc == 0] == 0)


def make(B, d, dt, seed, res):
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(B, d, generator=g) * 3).to(dt).cuda()
    r = torch.randn(B, d, generator=g).to(dt).cuda() if res else None
    w = torch.randn(d, generator=g).to(dt).cuda()
    return x, r, w


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,d", [(1, 1), (1, 2048), (3, 7), (2, 64), (5, 1152), (17, 1000), (4, 2560), (2, 8192),
                                 (300, 96), (3, 4104), (2, 16385), (1, 70001),
                                 # lanes, waves and chunks of each kind
                                 (70, 16), (33, 61), (65, 127), (9, 130), (31, 256), (5, 513), (2050, 700), (2051, 1153),
                                 (1030, 2570), (600, 7001), (3, 24000), (2, 49153)])
def test_sizes(dt, B, d):
    from lm_output_head_amd import rmsnorm
    x, r, w = make(B, d, dt, B * d, True)
    say("norm", dt, B, d)
    check(x, r, w, 1e-6, 0.0, rmsnorm(x, w, residual=r, want_q=True))
    check(x, None, w, 1e-5, 1.0, rmsnorm(x, w, eps=1e-5, weight_offset=1.0))
    check(x, None, None, 1e-6, 0.0, rmsnorm(x, want_out=False, want_q=True))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("off", [0, 1])
def test_strides_alignment_and_what_lies_between(dt, off):
    """Rows inside wider ones at an odd offset: only the rows are written."""
    from lm_output_head_amd import fh_rmsnorm
    for B, d, ld in [(4, 256, 264), (5, 250, 333), (3, 2048, 2056)]:
        x, r, w = make(B, d, dt, ld + off, True)
        wide = [torch.full((B + 1, ld), 7, dtype=t, device="cuda") for t in (dt, dt, dt, dt, torch.int8)]
        at = slice(off, off + d)
        xs, rs, os_, ss, qs = [t[:B, at] for t in wide]
        xs.copy_(x)
        rs.copy_(r)
        ws = torch.zeros(d + 1, dtype=dt, device="cuda")[off:off + d]
        ws.copy_(w)
        scale = torch.full((B + 1,), 7.0, device="cuda")
        say("norm strides", dt, B, d, ld, off)
        fh_rmsnorm(xs, rs, ws, 1e-6, 0.0, os_, ss, qs, scale[:B])
        check(x, r, w, 1e-6, 0.0, {"out": os_, "residual": ss, "q": qs, "q_scale": scale[:B]})
        for t in wide[2:]:
            mark = t.clone()
            mark[:B, at] = 7
            assert torch.all(mark == 7)
        assert scale[B] == 7 and torch.equal(xs, x) and torch.equal(rs, r)


@pytest.mark.parametrize("dt,d", [(torch.bfloat16, 2048), (torch.float32, 1000), (torch.bfloat16, 40000)])
def test_in_place(dt, d):
    from lm_output_head_amd import fh_rmsnorm, rmsnorm
    x, r, w = make(6, d, dt, 5, True)
    ref = rmsnorm(x, w, residual=r, want_q=True)
    x2, r2 = x.clone(), r.clone()
    q, sc = torch.empty(6, d, dtype=torch.int8, device="cuda"), torch.empty(6, device="cuda")
    say("norm in place", dt, d)
    fh_rmsnorm(x2, r2, w, 1e-6, 0.0, x2, r2, q, sc)
    assert torch.equal(x2, ref["out"]) and torch.equal(r2, ref["residual"])
    assert torch.equal(q, ref["q"]) and torch.equal(sc, ref["q_scale"])


def test_zero_and_non_finite_rows():
    from lm_output_head_amd import rmsnorm
    x = torch.randn(5, 512, device="cuda").bfloat16()
    x[1] = 0
    x[2, 17] = float("inf")
    x[3, 500] = float("nan")
    say("norm zero and non-finite rows")
    got = rmsnorm(x, want_q=True)
    torch.cuda.synchronize()
    assert torch.all(got["out"][1] == 0) and got["q_scale"][1] == 0 and torch.all(got["q"][1] == 0)
    assert got["out"][2, 17].isnan() and got["out"][3].isnan().all()
    assert got["q_scale"][2].isnan() and got["q_scale"][3].isnan()
    keep = [0, 4]
    check(x[keep], None, None, 1e-6, 0.0, {k: v[keep] for k, v in got.items()})


@pytest.mark.parametrize("d", [96, 40000])
def test_smallest_rows_keep_their_codes(d):
    """Rows whose largest |y| is near the smallest normal: 127 / max |y| is past
    float32's range, the codes are not.  y's and the scale's last bits are of
    2^-149, so the tolerances are absolute here."""
    from lm_output_head_amd import rmsnorm
    g = torch.Generator().manual_seed(3)
    x = torch.randn(4, d, generator=g).cuda()
    w = torch.full((d,), 1e-37, device="cuda")
    got = rmsnorm(x, w, want_q=True)
    y, _ = serve_oracle.rmsnorm(f64(x), None, f64(w), 1e-6, 0.0)
    assert np.all(np.abs(f64(got["out"]) - y) <= 1e-4 * np.abs(y) + 2.0 ** -148)
    q, top = f64(got["q"]), np.abs(y).max(1, keepdims=True)
    assert np.all(np.abs(q - y * 127 / top) <= 0.5 + 0.02) and np.all(np.abs(q).max(1) == 127)


def test_last_positions_of_a_batch():
    """x = hidden[:, -1] of [B x T x d] is taken without a copy."""
    from lm_output_head_amd import rmsnorm
    hidden = torch.randn(3, 9, 640, device="cuda").bfloat16()
    w = torch.randn(640, device="cuda").bfloat16()
    say("norm of last positions")
    a, b = rmsnorm(hidden[:, -1], w, want_q=True), rmsnorm(hidden[:, -1].contiguous(), w, want_q=True)
    assert all(torch.equal(a[k], b[k]) for k in a)
    check(hidden[:, -1], None, w, 1e-6, 0.0, a)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [5, 600])
def test_millions_of_rows(dt, d):
    """More rows than a launch holds workgroups of 1024 threads: the first and
    the last are as a call of their own gives them."""
    from lm_output_head_amd import rmsnorm
    B = (1 << 22) + 3
    x = torch.randn(1 << 12, d, device="cuda").to(dt).repeat((1 << 10) + 1, 1)[:B]
    say("norm of millions of rows", dt, d)
    a = rmsnorm(x, want_q=True)
    for lo in (0, B - 700):
        b = rmsnorm(x[lo:lo + 700], want_q=True)
        for k in b:
            assert torch.all((a[k][lo:lo + 700].double() - b[k].double()).abs() <= (1 if k == "q" else 2.0 ** -7) * b[k].double().abs().clamp(min=1))


def quotients(y, scale):
    """rint(y / scale) within [-127, 127] in float32, 0 where the scale is 0:
    numpy's float32 division is correctly rounded, subnormal values included."""
    y, scale = y.cpu().numpy(), scale.cpu().numpy()[:, None]
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        return np.where(scale > 0, np.clip(np.rint(y / scale), -127, 127), 0).astype(np.int8)


@pytest.mark.parametrize("B,d", [(60000, 96), (4096, 1153), (3000, 2560), (900, 9000), (150, 40000)])
def test_codes_are_the_rounded_quotients(B, d):
    """out_q = rint(y / out_scale), one division in float32, for every code: a
    float32 `out` is y itself.  A product with 127 / max |y| differs from it next
    to halves, in about one of a million codes."""
    from lm_output_head_amd import rmsnorm
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(B, d, generator=g, device="cuda") * 3
    w = torch.randn(d, generator=g, device="cuda")
    say("norm codes", B, d)
    got = rmsnorm(x, w, want_q=True)
    assert np.array_equal(got["q"].cpu().numpy(), quotients(got["out"], got["q_scale"]))


@pytest.mark.parametrize("d", [96, 2560, 40000])
@pytest.mark.parametrize("m", [1, 9, 30, 64, 200, 5000, 3 << 20])
def test_codes_of_rows_near_zero(d, m):
    """max |y| down to the smallest subnormal: a scale of 0 has codes 0, a
    subnormal scale (one significant bit and up) those of its own quotients."""
    from lm_output_head_amd import rmsnorm
    g = torch.Generator().manual_seed(d + m)
    x = torch.randn(5, d, generator=g).cuda()
    w = torch.full((d,), m * 2.0 ** -149, dtype=torch.float64).float().cuda()
    say("norm codes near zero", d, m)
    got = rmsnorm(x, w, want_q=True)
    top = got["out"].abs().amax(1).cpu().numpy()
    assert np.array_equal(got["q_scale"].cpu().numpy(), top / np.float32(127))
    assert np.array_equal(got["q"].cpu().numpy(), quotients(got["out"], got["q_scale"]))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("d", [5, 600])
def test_each_of_millions_of_rows(dt, d):
    """Every row of a large call is what the same lanes give it in a call of
    4096 rows, bit for bit."""
    from lm_output_head_amd import rmsnorm
    B, part = (1 << 22) + 3, 4096
    g = torch.Generator(device="cuda").manual_seed(d)
    x = torch.randn(part, d, generator=g, device="cuda").to(dt)
    say("each of millions of rows", dt, d)
    a = rmsnorm(x.repeat(B // part + 1, 1)[:B], want_q=True)
    b = rmsnorm(x, want_q=True)
    check(x, None, None, 1e-6, 0.0, b)
    for k in b:
        whole = B // part * part
        assert torch.all(a[k][:whole].reshape(B // part, *b[k].shape) == b[k]), k
        assert torch.equal(a[k][whole:], b[k][:B - whole]), k


def test_rows_past_one_launch_of_the_long_kernel():
    """2^29 + 5 rows of 3: eight lanes a row would be 2^32 threads, so
    workgroups walk over rows, some 512 each.  A row this short is one lane's
    sum either way, so slices through the eight-lane kernel give the same bits."""
    from lm_output_head_amd import rmsnorm
    B, d, part = (1 << 29) + 5, 3, 1 << 26
    g = torch.Generator(device="cuda").manual_seed(29)
    x = torch.randn(B, d, generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.tensor([0.5, -1.25, 2.0], device="cuda").bfloat16()
    say("norm of 2^29 + 5 rows")
    a = rmsnorm(x, w, want_q=True)
    for lo in range(0, B, part):
        b = rmsnorm(x[lo:lo + part], w, want_q=True)
        for k in b:
            assert torch.equal(a[k][lo:lo + part], b[k]), (k, lo)
    check(x[-2000:], None, w, 1e-6, 0.0, {k: t[-2000:] for k, t in a.items()})
