"""How the fp8 product's bfloat16 results are summed.

By default they are the float32 results rounded once: the same sums, so the same
bits.  What `native` may lose is held to its bound: of eight neighbouring products
each of the seven others is off by less than 2^-13 of the largest one's power of two, a
subnormal code's counted as 2^-6's, so the eight by less than 2^-10 of their sum of
magnitudes (counted so), beside the float32 sums'
(256 + 2 + k / 128 + 8) 2^-24 (test_gpu_fp8 counts it) and half a step of bfloat16,
2^-8.  Of normally distributed codes it loses 1.5e-5 of the results (2-norm), 1.2e-5
s on average for results of deviation s.  A step of bfloat16 is at least 2^-8 |z|,
so a result with |z| >= s / 2 becomes another value with probability
1.2e-5 / (2^-8 / 2) = 0.62% at most; 0.7% leaves five deviations of a million draws.

Whole numbers up to 8 and scales of powers of two leave nothing to round or to lose
(products from 1 to 64, sums below 2^24)."""

import numpy as np
import pytest
import torch

from oracle import fp8_oracle

from _gpu import need_gpu, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
F8 = torch.float8_e4m3fn
BF = torch.bfloat16

# each shape of tile, of either form; k of whole blocks, of whole chunks, and neither
SHAPES = [(20, 3000, 640), (32, 12000, 592), (33, 46100, 592), (33, 46100, 640), (64, 46100, 1152), (333, 5003, 592),
          (333, 5003, 600), (1000, 4096, 592), (700, 10000, 592), (700, 10000, 1152), (500, 14260, 256), (128, 4096, 4096)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    from lm_output_head_amd import load_library
    load_library()


def operands(B, n, k, seed, outliers=0.0):
    """Normally distributed codes, a channel in 64 larger by `outliers`, and scales."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    G, N = (k + 127) // 128, (n + 127) // 128
    q, w = (torch.randn(r, k, generator=g, device="cuda") * (448 / 4) for r in (B, n))
    if outliers:
        q[:, ::64] *= outliers
        q /= outliers
    qs = torch.rand(B, G, generator=g, device="cuda") + 0.5
    ws = (torch.rand(N, G, generator=g, device="cuda") + 0.5) / 4000
    return q.clamp(-448, 448).to(F8), qs, w.clamp(-448, 448).to(F8), ws


@pytest.mark.parametrize("B,n,k", SHAPES)
def test_bfloat16_results_are_the_float32_ones_rounded(B, n, k):
    from lm_output_head_amd import FP8Head
    for outliers in (0.0, 12.0, 60.0):
        q, qs, w, ws = operands(B, n, k, n + k, outliers)
        head = FP8Head(codes=w, scales=ws)
        say("fp8 bf16 sums", B, n, k, outliers)
        assert torch.equal(head.matmul(q, qs, dtype=BF), head.matmul(q, qs).to(BF))
        head.close()


@pytest.mark.parametrize("B,n,k", SHAPES)
def test_products_that_cancel_leave_what_is_beside_them(B, n, k):
    """Of each eight of k two products of 448 x 448 cancel beside one of 1 x 2."""
    from lm_output_head_amd import FP8Head
    eights = k // 8
    g = torch.Generator().manual_seed(k)
    at = torch.rand(eights, 8, generator=g).argsort(1)[:, :3] + 8 * torch.arange(eights)[:, None]
    q, w = torch.zeros(B, k), torch.zeros(n, k)
    for i, (a, b) in enumerate([(448.0, 448.0), (448.0, -448.0), (1.0, 2.0)]):
        q[:, at[:, i]], w[:, at[:, i]] = a, b
    # tokens and channels differ by a power of two
    t, c = 2.0 ** (torch.arange(B) % 3 - 1), 2.0 ** (torch.arange((n + 127) // 128) % 3 - 1)
    G = (k + 127) // 128
    want = 2.0 * eights * t[:, None].double() * c.repeat_interleave(128)[None, :n].double()
    head = FP8Head(codes=w.to(F8).cuda(), scales=c[:, None].repeat(1, G).cuda())
    qc, qs = q.to(F8).cuda(), t[:, None].repeat(1, G).cuda()
    say("fp8 cancel", B, n, k)
    for dt in (torch.float32, BF):
        assert torch.equal(head.matmul(qc, qs, dtype=dt).cpu(), want.to(dt))
    head.close()


def whole(B, n, k, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    G, N = (k + 127) // 128, (n + 127) // 128
    q, w = (torch.randint(-8, 9, (r, k), generator=g, device="cuda").float() for r in (B, n))
    qs, ws = (2.0 ** torch.randint(-1, 2, (r, G), generator=g, device="cuda").float() for r in (B, N))
    a = q.double() * qs.double().repeat_interleave(128, 1)[:, :k]
    b = w.double() * ws.double().repeat_interleave(128, 1)[:, :k].repeat_interleave(128, 0)[:n]
    return q.to(F8), qs, w.to(F8), ws, a @ b.t().contiguous()


@pytest.mark.parametrize("native", [False, True])
@pytest.mark.parametrize("B,n,k", SHAPES)
def test_whole_numbers_are_exact(B, n, k, native):
    from lm_output_head_amd import FP8Head
    q, qs, w, ws, want = whole(B, n, k, n)
    head = FP8Head(codes=w, scales=ws)
    say("fp8 whole numbers", B, n, k, native)
    assert torch.equal(head.matmul(q, qs, dtype=BF, native=native), want.to(BF))
    head.close()


@pytest.mark.parametrize("native", [False, True])
@pytest.mark.parametrize("B,n,k", [s for s in SHAPES if s[0] >= 20])
def test_nan_and_infinity_stay_in_their_rows(B, n, k, native):
    """A NaN code of a token or of the weight, in a row's first chunk (which stands in
    for those past its end) and in its last, a NaN and an infinite scale."""
    from lm_output_head_amd import FP8Head
    q, qs, w, ws = operands(B, n, k, 3)
    say("fp8 NaN in bf16", B, n, k, native)
    ref = FP8Head(codes=w, scales=ws).matmul(q, qs, dtype=BF, native=native)
    qb, wb = q.view(torch.uint8).clone(), w.view(torch.uint8).clone()
    qs, ws = qs.clone(), ws.clone()
    qb[1, k - 1], qb[B - 1, 3], wb[17, 5], wb[n - 1, k - 1] = 0xFF, 0x7F, 0x7F, 0xFF
    qs[2, qs.shape[1] - 1], ws[2, 1] = float("nan"), float("inf")
    got = FP8Head(codes=wb.view(F8), scales=ws).matmul(qb.view(F8), qs, dtype=BF, native=native)
    bad = torch.zeros(B, n, dtype=torch.bool, device="cuda")
    bad[[1, 2, B - 1]], bad[:, [17, n - 1]], bad[:, 256:384] = True, True, True
    assert torch.equal(got[~bad], ref[~bad]) and torch.isnan(got[[1, 2, B - 1]]).all()
    assert torch.isnan(got[:, [17, n - 1]]).all() and not torch.isfinite(got[:, 256:384]).any()


@pytest.mark.parametrize("B,n,k", [(20, 3000, 640), (33, 46100, 592), (333, 5003, 600), (1000, 4096, 592), (700, 10000, 592)])
@pytest.mark.parametrize("outliers", [0.0, 60.0])
def test_native_is_within_its_bound(B, n, k, outliers):
    from lm_output_head_amd import FP8Head
    q, qs, w, ws = operands(B, n, k, n + 1, outliers)
    head = FP8Head(codes=w, scales=ws)
    say("fp8 native", B, n, k, outliers)
    got, exact = head.matmul(q, qs, dtype=BF, native=True), head.matmul(q, qs)
    head.close()
    rows = slice(0, n, max(1, n // 600))  # the definition of some 600 channels
    code = lambda t: t.view(torch.uint8).cpu().numpy()  # noqa: E731
    want, size = [], []
    for j in range(0, n, 128):
        cols = [c for c in range(*rows.indices(n)) if j <= c < j + 128]
        if cols:
            a, b = fp8_oracle.product(code(q), qs.cpu().numpy(), code(w)[cols], ws[j // 128:j // 128 + 1].cpu().numpy())
            want.append(a)
            size.append(b)
    want, size = np.concatenate(want, 1), np.concatenate(size, 1)
    tol = ((256 + 2 + k / 128 + 8) * U + 2.0 ** -10) * size
    mine = got[:, rows].double().cpu().numpy()
    assert np.all(np.abs(mine - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))
    if not outliers:
        large = exact.abs() >= exact.std() / 2
        other = (got != exact.to(BF))[large]
        assert float(other.float().mean()) <= 0.007, float(other.float().mean())


def test_native_bound_counts_subnormal_codes_as_the_smallest_normal():
    """Eights of one product that cancels with the next eight's and seven small ones, from 6
    binades below it to 17, the tokens' codes from 1 down to the smallest."""
    from lm_output_head_amd import FP8Head
    B, n, k = 700, 10000, 592
    ones = lambda r: torch.ones(r, (k + 127) // 128, device="cuda")  # noqa: E731
    d = torch.arange(12) + 6  # of channel j: j % 12
    w = (256 * 2.0 ** -d[torch.arange(n) % 12].float())[:, None].repeat(1, k)
    w[:, ::16], w[:, 8::16] = 448, -448
    tokens = torch.tensor([1.0, 2.0 ** -6, 7 * 2.0 ** -9, 2.0 ** -7, 2.0 ** -8, 2.0 ** -9])
    q = tokens[torch.arange(B) % 6][:, None].repeat(1, k)
    head = FP8Head(codes=w.to(F8).cuda(), scales=ones((n + 127) // 128))
    say("fp8 native, subnormal")
    got = head.matmul(q.to(F8).cuda(), ones(B), dtype=BF, native=True).double().cpu()
    want = q.double() @ w.double().t().contiguous()
    size = q.double().clamp_min(2.0 ** -6) @ w.double().abs().t().contiguous()
    tol = ((256 + 2 + k / 128 + 8) * U + 2.0 ** -10) * size
    assert torch.all((got - want).abs() <= tol + 2.0 ** -8 * (want.abs() + tol))
    assert torch.equal(head.matmul(q.to(F8).cuda(), ones(B), dtype=BF).double().cpu(), want.to(BF).double())


def test_native_of_a_small_call_is_the_default():
    from lm_output_head_amd import FP8Head
    for B, n, k in [(1, 3000, 640), (20, 3000, 640), (32, 46100, 592)]:
        q, qs, w, ws = operands(B, n, k, 1)
        head = FP8Head(codes=w, scales=ws)
        say("fp8 native, small", B, n, k)
        assert torch.equal(head.matmul(q, qs, dtype=BF, native=True), head.matmul(q, qs, dtype=BF))


def test_native_rows_strides_workspace_and_what_lies_between():
    from lm_output_head_amd import FlashHeadError, FP8Head, fh_fp8_matmul_native, fh_fp8_workspace
    B, n, k = 333, 5003, 600  # rows of no whole chunks: the workspace holds their copy
    q, qs, w, ws, want = whole(B, n, k, 2)
    head = FP8Head(codes=w, scales=ws)
    wide = torch.full((B, k + 9), 0x7F, dtype=torch.uint8, device="cuda")
    wide[:, 3:3 + k] = q.view(torch.uint8)
    qv = wide[:, 3:3 + k].view(F8)
    out = torch.full((B + 1, n + 5), 7, dtype=BF, device="cuda")
    need = fh_fp8_workspace(head.w, qv, False)
    assert need > 0
    say("fp8 native strides")
    with pytest.raises(FlashHeadError, match="workspace"):
        fh_fp8_matmul_native(head.w, qv, qs, out[:B, 3:3 + n], torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
    fh_fp8_matmul_native(head.w, qv, qs, out[:B, 3:3 + n], torch.empty(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(out[:B, 3:3 + n], want.to(BF))
    out[:B, 3:3 + n] = 7
    assert torch.all(out == 7)


@pytest.mark.parametrize("native", [False, True])
@pytest.mark.parametrize("k", [592, 600])
def test_captured_bfloat16_products_replay_as_eager_ones(k, native):
    """On a stream of its own, captured, replayed over new codes with eager work between;
    at k = 600 the call copies its rows into the workspace first."""
    from lm_output_head_amd import FP8Head
    B, n = 333, 5003
    q, qs, w, ws = operands(B, n, k, 5)
    head = FP8Head(codes=w, scales=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    say("fp8 bf16 captured", k, native)
    aside = head.matmul(q, qs, dtype=BF, native=native, stream=s)
    s.synchronize()
    assert torch.equal(aside, head.matmul(q, qs, dtype=BF, native=native))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = head.matmul(q, qs, dtype=BF, native=native)
    for rep in range(4):
        q2, qs2, _, _ = operands(B, n, k, 6 + rep)
        q.copy_(q2)
        qs.copy_(qs2)
        say("fp8 bf16 replay", rep)
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        want = head.matmul(q, qs, dtype=BF, native=native)
        torch.cuda.synchronize()
        assert torch.equal(got, want), rep
