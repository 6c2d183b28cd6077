"""GPU parity of the int8 product and the dense head on it.

Tolerances, u = 2^-24: the int32 sum is exact; its conversion, the scales'
product and the last product round once each: 3 u (1 + u)^2 of the value, under
4 u; a bfloat16 output adds 2^-8.  The head's choice: serve_oracle.check_choice
with these errors of the logits."""

import numpy as np
import pytest
import torch

from oracle import serve_oracle

from _gpu import host, need_gpu, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    from lm_output_head_amd import load_library
    load_library()


def make(B, n, k, seed):
    rng = np.random.default_rng(seed)
    w = rng.integers(-128, 128, (n, k)).astype(np.int8)
    q = rng.integers(-128, 128, (B, k)).astype(np.int8)
    ws = rng.uniform(0.5, 2, n).astype(np.float32) / 4000
    qs = rng.uniform(0.5, 2, B).astype(np.float32) / np.sqrt(k).astype(np.float32)
    return q, qs, w, ws


def dev(a):
    return torch.from_numpy(a).cuda()


SIZES = [(1, 1, 1), (1, 16, 64), (3, 17, 65), (5, 130, 16), (16, 128, 128), (17, 1000, 192), (33, 515, 2048),
         (64, 272, 1152), (70, 301, 100), (128, 96, 2560), (129, 640, 320), (300, 1030, 80), (257, 2000, 576),
         (1, 5003, 8192), (2, 40, 131071), (520, 513, 704),
         # each way of cutting a call up, and odd and even numbers of blocks of k
         (3, 9001, 70), (16, 8200, 448), (7, 32785, 48), (16, 33000, 320), (20, 25001, 320), (32, 24600, 448),
         (40, 32801, 320), (64, 33000, 448), (100, 65601, 320), (128, 65600, 192), (300, 32801, 320),
         (257, 33001, 448), (200, 4000, 320), (129, 70001, 130), (2, 33001, 320), (3, 33000, 1600),
         (1, 9001, 2900), (9, 32770, 130), (100, 6000, 1600), (128, 3200, 4200), (200, 7000, 3100), (30, 6001, 100)]


@pytest.mark.parametrize("B,n,k", SIZES)
def test_product(B, n, k):
    from lm_output_head_amd import W8A8Head
    q, qs, w, ws = make(B, n, k, n + k)
    want = serve_oracle.product(q, qs, w, ws)
    head = W8A8Head(codes=dev(w), scales=dev(ws))
    say("product", B, n, k)
    for dt, extra in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        got = head.matmul(dev(q), dev(qs), dtype=dt)
        torch.cuda.synchronize()
        assert got.dtype == dt
        assert np.all(np.abs(got.double().cpu().numpy() - want) <= (4 * U + extra * (1 + 4 * U)) * np.abs(want)), dt
    head.close()


def test_largest_sums_are_exact():
    """All codes -128 at the largest k: 128^2 131071 is just below 2^31."""
    from lm_output_head_amd import W8A8Head
    k = 131071
    q = torch.full((3, k), -128, dtype=torch.int8, device="cuda")
    q[1] = 127
    w = torch.full((18, k), -128, dtype=torch.int8, device="cuda")
    head = W8A8Head(codes=w, scales=torch.ones(18, device="cuda"))
    say("largest sums")
    got = head.matmul(q, torch.ones(3, device="cuda"))
    assert torch.all(got[0] == float(128 * 128 * k)) and torch.all(got[1] == float(-127 * 128 * k))


@pytest.mark.parametrize("B,n,k,off,ld", [(5, 100, 128, 0, 144), (5, 100, 128, 0, 136), (6, 77, 128, 3, 200),
                                          (40, 333, 100, 1, 111), (1, 64, 256, 5, 300), (130, 130, 96, 16, 112)])
def test_strides_alignment_and_what_lies_between(B, n, k, off, ld):
    from lm_output_head_amd import W8A8Head, fh_w8a8_matmul, fh_w8a8_workspace
    q, qs, w, ws = make(B, n, k, ld)
    want = serve_oracle.product(q, qs, w, ws)
    head = W8A8Head(codes=dev(w), scales=dev(ws))
    wide = torch.full((B + 1, ld + off), 99, dtype=torch.int8, device="cuda")
    qv = wide[:B, off:off + k] if off + k <= ld else wide[:B, off:off + k]
    qv.copy_(dev(q))
    size = fh_w8a8_workspace(head.w, qv, False)
    wsp = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    say("product strides", B, n, k, off, ld, "workspace", size)
    for dt, extra in ((torch.float32, 0.0), (torch.bfloat16, 2.0 ** -8)):
        out = torch.full((B + 1, n + 5), 7, dtype=dt, device="cuda")
        fh_w8a8_matmul(head.w, qv, dev(qs), out[:B, 3:3 + n], wsp)
        got = out[:B, 3:3 + n].double().cpu().numpy()
        assert np.all(np.abs(got - want) <= (4 * U + extra * (1 + 4 * U)) * np.abs(want))
        out[:B, 3:3 + n] = 7
        assert torch.all(out == 7)
    head.close()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_quantised_weight(dt):
    """Codes and scales of fh_w8a8_create: the scale max |W| / 127 to one
    rounding, codes within half a step of W / scale (the division's rounding
    more), the copy out equal to what a second handle takes in."""
    from lm_output_head_amd import W8A8Head
    W = torch.randn(131, 200, device="cuda").to(dt)
    W[7] = 0
    W[9] *= 1e30
    say("quantised weight", dt)
    head = W8A8Head(W)
    codes, scales = head.codes()
    w, c, s = W.double().cpu().numpy(), codes.cpu().numpy().astype(np.float64), scales.double().cpu().numpy()
    want = np.abs(w).max(1) / 127
    assert np.all(np.abs(s - want) <= U * want) and s[7] == 0 and not c[7].any()
    assert np.all(np.abs(c - w / np.where(s > 0, s, 1)[:, None]) <= 0.5 + 128 * U) and np.abs(c).max() == 127
    again = W8A8Head(codes=codes, scales=scales)
    c2, s2 = again.codes()
    assert torch.equal(c2, codes) and torch.equal(s2, scales)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("k", [1, 5, 77, 135, 600])
def test_quantised_weight_of_any_width(dt, k):
    """Rows that are no whole loads, a large element in the last place."""
    from lm_output_head_amd import W8A8Head
    W = torch.randn(37, k, device="cuda").to(dt)
    W[:, -1] = -5
    say("quantised weight", dt, k)
    codes, scales = W8A8Head(W).codes()
    w, c, s = W.double().cpu().numpy(), codes.cpu().numpy().astype(np.float64), scales.double().cpu().numpy()
    want = np.abs(w).max(1) / 127
    assert np.all(np.abs(s - want) <= U * want)
    assert np.all(c[np.abs(w).max(1) == 5, -1] == -127)  # a draw of more than 5 makes another element the largest
    assert np.all(np.abs(c - w / s[:, None]) <= 0.5 + 128 * U)
    W[36, -1] = float("nan")
    with pytest.raises(Exception, match="infinity or NaN"):
        W8A8Head(W)


def test_non_finite_weights_are_refused():
    from lm_output_head_amd import FlashHeadError, W8A8Head
    for bad in (float("inf"), float("nan")):
        W = torch.ones(20, 40, device="cuda")
        W[19, 39] = bad
        with pytest.raises(FlashHeadError, match="infinity or NaN"):
            W8A8Head(W)


@pytest.mark.parametrize("B,n,k", [(1, 1, 16), (1, 5000, 2048), (3, 1000, 100), (16, 4099, 128), (33, 700, 1152),
                                   (64, 3000, 256), (130, 1111, 192), (300, 640, 64),
                                   (3, 9001, 70), (7, 32785, 48), (20, 25001, 80), (40, 32801, 64), (100, 65601, 64),
                                   (300, 33001, 64), (200, 4000, 320), (9, 32770, 130), (100, 6000, 1600),
                                   (128, 3200, 4200), (200, 7000, 3100)])
@pytest.mark.parametrize("mode,T", [(0, 1.0), (2, 0.7)])
def test_head(B, n, k, mode, T):
    from lm_output_head_amd import W8A8Head
    q, qs, w, ws = make(B, n, k, n + B)
    want = serve_oracle.product(q, qs, w, ws)
    head = W8A8Head(codes=dev(w), scales=dev(ws))
    say("int8 head", B, n, k, mode)
    out = host(head.forward(dev(q), dev(qs), mode=mode, temperature=T, seed=12345678901, want_logits=True))
    tol = 4 * U * np.abs(want)
    assert np.all(np.abs(out["logits"] - want) <= tol)
    assert not serve_oracle.check_choice(want, tol, None, mode, T, 12345678901, out)
    again = host(head.forward(dev(q), dev(qs), mode=mode, temperature=T, seed=12345678901))
    assert all(np.array_equal(again[x], out[x]) for x in ("token", "token_logit", "lse"))
    head.close()


def test_ties_go_to_the_smaller_token():
    from lm_output_head_amd import W8A8Head
    w = torch.ones(700, 64, dtype=torch.int8, device="cuda")
    q = torch.ones(2, 64, dtype=torch.int8, device="cuda")
    head = W8A8Head(codes=w, scales=torch.ones(700, device="cuda"))
    out = host(head.forward(q, torch.tensor([1.0, -1.0], device="cuda")))
    assert out["token"].tolist() == [0, 0] and out["token_logit"].tolist() == [64.0, -64.0]


def test_non_finite_scales():
    """A NaN scale of a token leaves its row without a token; the others stand."""
    from lm_output_head_amd import W8A8Head
    q, qs, w, ws = make(3, 300, 64, 8)
    qs[1] = np.nan
    head = W8A8Head(codes=dev(w), scales=dev(ws))
    out = host(head.forward(dev(q), dev(qs)))
    assert out["token"][1] == -1 and np.isnan(out["lse"][1]) and out["token_logit"][1] == -np.inf
    want = serve_oracle.product(q, qs, w, ws)[[0, 2]]
    part = {k: v[[0, 2]] for k, v in out.items()}
    assert not serve_oracle.check_choice(want, 4 * U * np.abs(want), None, 0, 1.0, 0, part)


def test_workspace_of_the_call_is_checked():
    from lm_output_head_amd import FlashHeadError, W8A8Head, fh_w8a8_forward, fh_w8a8_workspace
    q, qs, w, ws = make(4, 100, 50, 1)
    head = W8A8Head(codes=dev(w), scales=dev(ws))
    size = fh_w8a8_workspace(head.w, dev(q), True)
    tok = torch.empty(4, dtype=torch.int32, device="cuda")
    with pytest.raises(FlashHeadError, match="workspace"):
        fh_w8a8_forward(head.w, dev(q), dev(qs), 0, 1.0, 0, tok,
                        workspace=torch.empty(size - 1, dtype=torch.uint8, device="cuda"))
    head.close()
    with pytest.raises(ValueError, match="unknown int8 weight|either"):
        head.matmul(dev(q), dev(qs))


def test_more_than_one_launch_holds_is_refused():
    from lm_output_head_amd import FlashHeadError, W8A8Head
    n = 256 * (1 << 14) + 1
    head = W8A8Head(codes=torch.ones(n, 1, dtype=torch.int8, device="cuda"), scales=torch.ones(n, device="cuda"))
    q, qs = torch.ones(65535, 1, dtype=torch.int8, device="cuda"), torch.ones(65535, device="cuda")
    say("too many tiles")
    with pytest.raises(FlashHeadError, match="too large for one call"):
        head.forward(q, qs)
    got = head.forward(q[:3], qs[:3])
    assert got["token"].tolist() == [0, 0, 0] and got["token_logit"].tolist() == [1.0] * 3


# weights that pass the caches by, of more than 64, 128 or 256 MB, each way of
# cutting them up
@pytest.mark.parametrize("n,k,Bs", [(70001, 1000, (1, 4)), (45001, 1600, (2,)), (24001, 2900, (3,)), (5001, 14000, (16,)),
                                    (20001, 3500, (5,)), (12001, 5700, (20, 30)), (19300, 7100, (32,)),
                                    (16001, 8500, (20,)), (25001, 10800, (50,)), (240001, 1152, (1, 16, 17, 40, 100, 130))])
def test_large_weights_are_as_their_slices(n, k, Bs):
    """Exact sums and one formula: rows 0 .. 999 and the last 1000 as a weight of
    their own, cut up another way, give the same bits."""
    from lm_output_head_amd import W8A8Head
    g = torch.Generator(device="cuda").manual_seed(n)
    w = torch.randint(-128, 128, (n, k), dtype=torch.int8, device="cuda", generator=g)
    ws = torch.rand(n, device="cuda", generator=g) / 4000
    head = W8A8Head(codes=w, scales=ws)
    cuts = [(lo, W8A8Head(codes=w[lo:lo + 1000].contiguous(), scales=ws[lo:lo + 1000])) for lo in (0, n // 2, n - 1000)]
    for B in Bs:
        say("large weight", B, n, k)
        q = torch.randint(-128, 128, (B, k), dtype=torch.int8, device="cuda", generator=g)
        qs = torch.rand(B, device="cuda", generator=g)
        for dt in (torch.float32, torch.bfloat16):
            z = head.matmul(q, qs, dtype=dt)
            for lo, part in cuts:
                assert torch.equal(z[:, lo:lo + 1000], part.matmul(q, qs, dtype=dt)), (B, dt, lo)
        out, z = head.forward(q, qs, want_logits=True), head.matmul(q, qs)
        assert torch.equal(out["logits"], z)
        top = z.amax(1)
        first = torch.where(z == top[:, None], torch.arange(n, device="cuda"), n).amin(1)  # ties: the smaller token
        assert torch.equal(out["token"].long(), first) and torch.equal(out["token_logit"], top)


def test_infinite_logits_are_drawn_before_large_ones():
    """A channel whose scale overflows the product: its +inf is drawn though
    every other z / T is past exp's range, the smallest token of several."""
    from lm_output_head_amd import W8A8Head
    n, k = 3000, 64
    w = torch.ones(n, k, dtype=torch.int8, device="cuda")
    for first, more in ((9, (11, 40, 2000)), (1502, ()), (2999, ()), (130, (131,))):
        scales = torch.ones(n, device="cuda")
        scales[[first, *more]] = 3e38
        head = W8A8Head(codes=w, scales=scales)
        for B in (1, 5, 40, 130):
            q, qs = torch.ones(B, k, dtype=torch.int8, device="cuda"), torch.full((B,), 2.0, device="cuda")
            say("int8 head, infinite logits", first, B)
            for mode, T in ((0, 1.0), (2, 0.5)):
                out = head.forward(q, qs, mode=mode, temperature=T, seed=6)
                assert out["token"].tolist() == [first] * B and torch.all(out["token_logit"] == float("inf"))
                assert torch.all(out["lse"] == float("inf"))
        head.close()


def test_a_refused_allocation_leaves_no_error_behind():
    """A weight larger than the card is refused before anything is read; the
    calls after it do not find its error."""
    import ctypes
    from lm_output_head_amd import FlashHeadError, W8A8Head, load_library, logits_apply, rmsnorm
    from lm_output_head_amd._abi import check
    lib = load_library()
    n, k = 1 << 27, 131071  # 1.8e13 bytes
    assert n * k > 16 * torch.cuda.get_device_properties(0).total_memory
    codes, scales = torch.ones(4, 64, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    x = torch.randn(3, 64, device="cuda")
    torch.cuda.synchronize()
    for create, args in ((lib.fh_w8a8_create_codes, (codes.data_ptr(), scales.data_ptr())),
                         (lib.fh_w8a8_create, (x.data_ptr(), 0))):
        w = ctypes.c_void_p()
        say("a weight larger than the card")
        with pytest.raises(FlashHeadError) as e:
            check(create(*args, n, k, None, ctypes.byref(w)))
        assert e.value.status == -2 and not w.value
        assert lib.hipPeekAtLastError() == 0
        rmsnorm(x)
        logits_apply(x)
        head = W8A8Head(codes=codes, scales=scales)
        assert head.matmul(codes, scales).shape == (4, 4)
        head.close()
