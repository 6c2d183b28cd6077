"""GPU parity of fh_logits_apply against the float64 definition.

Tolerances, u = 2^-24: the repetition rounds twice (its reciprocal and the
product), the penalty, the presence, each bias's addition and the bias's own
once each; the oracle returns the sum of magnitudes they are relative to (a bias
counted four times, for its running sum over the few entries of one token), so
8 u of it covers up to eight roundings.  The choice: serve_oracle.check_choice."""

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


def make_rules(rng, B, v, L, nb, density, R=3, shared=True):
    r = {}
    if L:
        r["history"] = rng.integers(-3, v + 3, (B, L)).astype(np.int32)
        r["history"][:, ::3] = rng.integers(0, min(v, 5), (B, (L + 2) // 3))  # some often
        r["n_history"] = rng.integers(-1, L + 5, B).astype(np.int32)
        r["n_prompt"] = rng.integers(-1, L + 1, B).astype(np.int32)
        r["repetition"] = rng.uniform(0.8, 1.5, B).astype(np.float32)
        r["frequency"] = rng.uniform(-0.2, 0.5, B).astype(np.float32)
        r["presence"] = rng.uniform(-0.2, 0.5, B).astype(np.float32)
    if nb:
        r["bias_ids"] = rng.integers(-1, v + 1, (B, nb)).astype(np.int32)
        r["bias_ids"][:, ::4] = r["bias_ids"][:, :1]  # the same token several times
        r["bias"] = rng.normal(0, 3, (B, nb)).astype(np.float32)
        r["n_bias"] = rng.integers(0, nb + 2, B).astype(np.int32)
    if density:
        R = R if shared else B
        bits = rng.random((R, (v + 31) // 32 * 32)) < density
        r["mask"] = np.packbits(bits.reshape(R, -1, 32), axis=2, bitorder="little").view(np.uint32)[:, :, 0].view(np.int32)
        if shared:
            r["mask_row"] = rng.integers(-1, R + 1, B).astype(np.int32)
    return r


def on_gpu(v, r):
    from lm_output_head_amd import LogitRules
    return LogitRules(v, **{k: torch.from_numpy(np.ascontiguousarray(a)).cuda() for k, a in r.items()})


def run_and_check(z, ids, v, r, mode, T, seed=9):
    from lm_output_head_amd import logits_apply
    zt = torch.from_numpy(z).cuda()
    it = None if ids is None else torch.from_numpy(ids).cuda()
    out = host(logits_apply(zt, on_gpu(v, r), ids=it, mode=mode, temperature=T, seed=seed))
    want, size = serve_oracle.apply_rules(z, ids, v, **r)
    tol = 8 * U * size
    assert np.array_equal(np.isneginf(out["logits"]), np.isneginf(want))
    fin = np.isfinite(want)
    assert np.all(np.abs(out["logits"][fin] - want[fin]) <= tol[fin])
    fails = serve_oracle.check_choice(want, tol, ids, mode, T, seed, out)
    assert not fails, fails
    return out


CASES = [(1, 1, 1, 1, 0.9), (1, 33, 0, 0, 0.5), (2, 1000, 50, 0, 0.0), (3, 4096, 300, 7, 0.25), (2, 4097, 0, 300, 0.25),
         (4, 5001, 1000, 20, 0.01), (2, 12293, 700, 600, 0.0), (5, 20000, 9000, 64, 0.3), (64, 300, 40, 3, 0.5), (64, 33000, 5000, 20, 0.5),
         (1, 128256, 1000, 16, 0.25), (3, 40057, 5000, 1, 0.9),
         # each way of cutting a call up
         (520, 3001, 200, 5, 0.5), (3, 1025, 100, 4, 0.5), (200, 8192, 3000, 20, 0.5)]


@pytest.mark.parametrize("B,v,L,nb,density", CASES)
@pytest.mark.parametrize("mode,T", [(0, 1.0), (2, 0.8)])
def test_dense(B, v, L, nb, density, mode, T):
    rng = np.random.default_rng(v + mode)
    say("rules dense", B, v, L, nb, density, mode)
    run_and_check(rng.normal(0, 3, (B, v)).astype(np.float32), None, v, make_rules(rng, B, v, L, nb, density), mode, T)


@pytest.mark.parametrize("B,v,n,L,nb,density", [(1, 10, 1, 3, 2, 0.5), (3, 1000, 64, 100, 10, 0.5), (2, 5000, 1024, 0, 30, 0.3),
                                                (2, 5000, 1025, 600, 0, 0.0), (4, 128256, 8192, 2000, 32, 0.25),
                                                (3, 3000, 3000, 500, 8, 0.9), (2, 2000, 5001, 500, 8, 0.9),
                                                (64, 20000, 8200, 5000, 20, 0.5), (5, 700, 2500, 400, 8, 0.9),
                                                (16, 20000, 12000, 3000, 20, 0.5), (64, 9000, 8000, 500, 30, 0.5),
                                                (130, 9000, 8192, 2000, 1100, 0.5), (130, 20000, 9000, 9000, 30, 0.5)])
@pytest.mark.parametrize("mode,T", [(0, 1.0), (2, 0.8)])
def test_candidates(B, v, n, L, nb, density, mode, T):
    """Listed tokens in any order, some twice, some no tokens (-1, v)."""
    rng = np.random.default_rng(n + mode)
    ids = np.stack([rng.permutation(v)[:n] if n <= v else rng.integers(0, v, n) for _ in range(B)]).astype(np.int32)
    if n > 8:
        ids[:, 5] = -1
        ids[:, 6] = v
        ids[:, 8] = ids[:, 7]
    z = rng.normal(0, 3, (B, n)).astype(np.float32)
    say("rules candidates", B, v, n, L, nb, density, mode)
    run_and_check(z, ids, v, make_rules(rng, B, v, L, nb, density), mode, T)


@pytest.mark.parametrize("name", ["history", "bias", "mask", "nothing", "own mask rows"])
def test_each_rule_alone(name):
    rng = np.random.default_rng(3)
    z = rng.normal(0, 3, (4, 3001)).astype(np.float32)
    r = {"history": lambda: make_rules(rng, 4, 3001, 99, 0, 0), "bias": lambda: make_rules(rng, 4, 3001, 0, 40, 0),
         "mask": lambda: make_rules(rng, 4, 3001, 0, 0, 0.2), "nothing": dict,
         "own mask rows": lambda: make_rules(rng, 4, 3001, 0, 0, 0.2, shared=False)}[name]()
    say("rule alone", name)
    run_and_check(z, None, 3001, r, 0, 1.0)


def test_rows_with_nothing_left_and_masked_non_finites():
    """Row 0: its mask allows nothing.  Row 1: infinities and NaN where the mask
    is shut.  Row 2: the only open token holds the type's lowest value.  Row 3:
    -inf everywhere.  Row 4: +inf is open.  Row 5: an open NaN."""
    from lm_output_head_amd import logits_apply
    v = 9000
    rng = np.random.default_rng(1)
    z = rng.normal(0, 3, (6, v)).astype(np.float32)
    bits = np.ones((6, (v + 31) // 32 * 32), bool)
    bits[0] = False
    for i, x in ((10, np.nan), (4500, np.inf), (8999, -np.inf), (4501, 3.0e38)):
        z[1, i] = x
        bits[1, i] = False
    bits[2] = False
    bits[2, 8000] = True
    z[2, 8000] = np.finfo(np.float32).min
    z[3] = -np.inf
    z[4, 77] = np.inf
    z[5, 4242] = np.nan
    words = np.packbits(bits.reshape(6, -1, 32), axis=2, bitorder="little").view(np.int32)[:, :, 0]
    say("rows with nothing left")
    for mode in (0, 2):
        out = host(logits_apply(torch.from_numpy(z).cuda(), on_gpu(v, {"mask": words}), mode=mode, temperature=0.5, seed=3))
        for b in (0, 3):
            assert out["token"][b] == -1 and out["lse"][b] == -np.inf and out["token_logit"][b] == -np.inf
            assert np.all(out["logits"][b] == -np.inf)
        want, size = serve_oracle.apply_rules(z[1:2], None, v, mask=words[1:2])
        part = {k: x[1:2] for k, x in out.items()}
        if mode == 0:
            assert not serve_oracle.check_choice(want, 8 * U * size, None, 0, 1.0, 3, part)
        assert np.isneginf(out["logits"][1]).sum() == 4 and not np.isnan(out["logits"][1]).any()
        assert out["token"][2] == 8000
        assert out["token"][4] == 77 and out["lse"][4] == np.inf and out["token_logit"][4] == np.inf
        assert np.isnan(out["lse"][5]) and out["token"][5] not in (-1, 4242)


def test_strides_in_place_and_what_lies_between():
    from lm_output_head_amd import fh_logits_apply, fh_logits_workspace
    rng = np.random.default_rng(5)
    B, v = 3, 5003
    z = rng.normal(0, 3, (B, v)).astype(np.float32)
    r = make_rules(rng, B, v, 200, 20, 0.3)
    wide = {k: np.full((B + 1, a.shape[1] + 5), 2 if a.dtype == np.int32 else 7, a.dtype) for k, a in r.items()
            if k in ("history", "bias_ids", "bias")}
    gpu = {k: torch.from_numpy(np.ascontiguousarray(a)).cuda() for k, a in r.items()}
    for k in wide:
        t = torch.from_numpy(wide[k]).cuda()
        t[:B, 2:-3] = gpu[k]
        gpu[k] = t[:B, 2:-3]
    from lm_output_head_amd import LogitRules
    rules = LogitRules(v, **gpu)
    want, size = serve_oracle.apply_rules(z, None, v, **r)
    buf = torch.full((B + 1, v + 6), 7.0, device="cuda")
    zt = buf[:B, 3:3 + v]
    zt.copy_(torch.from_numpy(z))
    tok = torch.full((B + 1,), -7, dtype=torch.int32, device="cuda")
    ws = torch.empty(fh_logits_workspace(B, v), dtype=torch.uint8, device="cuda")
    say("rules strides, in place")
    fh_logits_apply(zt, None, v, rules, 0, 1.0, 0, zt, tok[:B], workspace=ws)
    got = zt.double().cpu().numpy()
    fin = np.isfinite(want)
    assert np.array_equal(fin, np.isfinite(got)) and np.all(np.abs(got[fin] - want[fin]) <= (8 * U * size)[fin])
    zt.fill_(7.0)
    assert torch.all(buf == 7) and tok[B] == -7
    assert np.array_equal(tok[:B].cpu().numpy(), want.argmax(1))


def test_logits_alone_and_token_alone():
    from lm_output_head_amd import fh_logits_apply, fh_logits_workspace, logits_apply
    rng = np.random.default_rng(6)
    z = torch.from_numpy(rng.normal(0, 3, (2, 9999)).astype(np.float32)).cuda()
    r = on_gpu(9999, make_rules(rng, 2, 9999, 64, 8, 0.2))
    full = logits_apply(z, r, mode=2, temperature=0.6, seed=4)
    only = logits_apply(z, r, want_token=False)
    tok = torch.empty(2, dtype=torch.int32, device="cuda")
    fh_logits_apply(z, None, 9999, r, 2, 0.6, 4, out_token=tok,
                    workspace=torch.empty(fh_logits_workspace(2, 9999), dtype=torch.uint8, device="cuda"))
    assert torch.equal(only["logits"], full["logits"]) and torch.equal(tok, full["token"])


def test_penalties_without_a_history_do_nothing():
    from lm_output_head_amd import LogitRules, logits_apply
    z = torch.randn(3, 4000, device="cuda")
    two = torch.full((3,), 2.0, device="cuda")
    a = logits_apply(z, LogitRules(4000, repetition=two, frequency=two, presence=two))
    none = torch.zeros(3, 0, dtype=torch.int32, device="cuda")
    b = logits_apply(z, LogitRules(4000, history=none, repetition=two, frequency=two, presence=two))
    for o in (a, b):
        assert torch.equal(o["logits"], z) and torch.equal(o["token"].long(), z.argmax(1))


def test_empty_lists_with_their_lengths_do_nothing():
    from lm_output_head_amd import LogitRules, logits_apply
    z = torch.randn(3, 4000, device="cuda")
    n = torch.tensor([0, 5, -1], dtype=torch.int32, device="cuda")
    ids = torch.zeros(3, 6, dtype=torch.int32, device="cuda")
    r = LogitRules(4000, history=ids[:, :0], n_prompt=n, n_history=n, repetition=torch.full((3,), 2.0, device="cuda"),
                   bias_ids=ids[:, :0], bias=ids.float()[:, :0], n_bias=n)
    out = logits_apply(z, r)
    assert torch.equal(out["logits"], z) and torch.equal(out["token"].long(), z.argmax(1))


def test_same_choice_as_the_dense_head():
    """Without rules the choice over fh_dense_forward's logits is its own."""
    from lm_output_head_amd import FlashHead, logits_apply
    from synth import make_problem
    from _gpu import problem_tensors
    pb = make_problem("tiny")
    E, C, H = problem_tensors(pb)
    head = FlashHead(E, C, pb.C2T, max_batch=8)
    for mode in (0, 2):
        d = head.dense(H[:8], mode=mode, temperature=0.9, seed=21, want_logits=True)
        a = logits_apply(d["logits"], mode=mode, temperature=0.9, seed=21)
        assert torch.equal(a["token"], d["token"]) and torch.equal(a["token_logit"], d["token_logit"])
        assert torch.allclose(a["lse"], d["lse"], rtol=1e-5, atol=1e-6)
    head.close()


def smallest_infinite(z, ids):
    t = np.broadcast_to(np.arange(z.shape[1]), z.shape) if ids is None else ids
    return np.where(np.isposinf(z), t, np.iinfo(np.int32).max).min(1)


@pytest.mark.parametrize("B,n,listed", [(40, 300, False), (40, 3001, False), (40, 6000, False), (40, 20000, False),
                                        (520, 3001, False), (130, 33000, False), (40, 300, True), (40, 900, True),
                                        (40, 3000, True), (40, 9000, True), (130, 9000, True)])
def test_infinite_logits_are_drawn_before_large_ones(B, n, listed):
    """Every finite z / T is past exp's range (100 and more): +inf, one or
    several, is drawn all the same, the smallest token of them."""
    from lm_output_head_amd import logits_apply
    rng = np.random.default_rng(n + B)
    v = n + 1000 if listed else n
    ids = np.stack([rng.permutation(v)[:n] for _ in range(B)]).astype(np.int32) if listed else None
    z = rng.uniform(5, 30, (B, n)).astype(np.float32)
    for b in range(B):
        z[b, rng.integers(0, n, 1 + b % 3)] = np.inf
        if b % 4 == 1:  # neighbours of one thread's run
            i = int(rng.integers(0, n - 1))
            z[b, i:i + 2] = np.inf
    z[5, np.flatnonzero(np.isfinite(z[5]))[::7]] = np.nan
    z[6, np.flatnonzero(np.isfinite(z[6]))[::2]] = np.finfo(np.float32).max
    say("infinite logits", B, n, listed)
    gpu = None if ids is None else torch.from_numpy(ids).cuda()
    for mode, T in ((0, 1.0), (2, 0.05), (2, 0.001), (2, 1.0)):
        out = host(logits_apply(torch.from_numpy(z).cuda(), ids=gpu, v=v, mode=mode, temperature=T, seed=8))
        assert np.array_equal(out["token"], smallest_infinite(z, ids)), (mode, T)
        assert np.all(np.isposinf(out["token_logit"]))
        lse = np.full(B, np.inf)
        lse[5] = np.nan
        assert np.array_equal(out["lse"], lse, equal_nan=True)


@pytest.mark.parametrize("listed", [False, True])
def test_a_bias_of_infinity_forces_its_token(listed):
    from lm_output_head_amd import logits_apply
    rng = np.random.default_rng(4)
    B, n = 64, 5000
    z = rng.uniform(2, 30, (B, n)).astype(np.float32)
    ids = np.stack([rng.permutation(n) for _ in range(B)]).astype(np.int32) if listed else None
    r = {"bias_ids": rng.integers(0, n, (B, 9)).astype(np.int32), "bias": np.ones((B, 9), np.float32)}
    r["bias"][:, 4] = np.inf
    say("bias of infinity", listed)
    for T in (0.02, 0.25):
        out = host(logits_apply(torch.from_numpy(z).cuda(), on_gpu(n, r), v=n, mode=2, temperature=T, seed=1,
                                ids=None if ids is None else torch.from_numpy(ids).cuda()))
        assert np.array_equal(out["token"], r["bias_ids"][:, 4])


@pytest.mark.parametrize("B,n,listed", [(3, 900, False), (3, 3000, False), (3, 7000, False), (3, 12000, False),
                                        (300, 12000, False), (600, 2500, False), (3, 400, True), (3, 900, True),
                                        (3, 3000, True), (2, 9000, True), (130, 9000, True)])
def test_long_bias_lists_are_summed_in_order(B, n, listed):
    """The listed biases of a token are added up in float32 in the list's order
    and their sum to the logit, in one rounding, however long the list and
    whatever the size of the call."""
    from lm_output_head_amd import logits_apply
    rng = np.random.default_rng(n)
    v, nb = n, 2600
    z = rng.normal(0, 3, (1, n)).astype(np.float32)
    ids = rng.permutation(v)[None].astype(np.int32) if listed else None
    bias_ids = rng.integers(0, v, (1, nb)).astype(np.int32)
    bias = rng.normal(0, 3, (1, nb)).astype(np.float32)
    for t, places, adds in ((7, (0, 301, 2599), (1e8, -1e8, 0.5)),
                            (11, (255, 256, 511, 512, 1023, 1024, 2048), (1e8, 3, -1e8, 1e7, 5, -1e7, 0.25)),
                            (12, (1, 2, 3), (-3e7, 3e7, 1.5))):
        bias_ids[0, list(places)] = t
        bias[0, list(places)] = adds
    total = np.zeros(v, np.float32)
    for t, add in zip(bias_ids[0], bias[0]):
        total[t] = total[t] + add
    want = z + (total if ids is None else total[ids[0]])
    say("long bias lists", B, n, listed)
    r = {"bias_ids": np.repeat(bias_ids, B, 0), "bias": np.repeat(bias, B, 0)}
    gpu = None if ids is None else torch.from_numpy(np.repeat(ids, B, 0)).cuda()
    out = host(logits_apply(torch.from_numpy(np.repeat(z, B, 0)).cuda(), on_gpu(v, r), ids=gpu, v=v))
    assert np.array_equal(out["logits"], np.repeat(want, B, 0))


def test_lists_of_one_row_at_any_stride():
    """One row's stride says nothing: lists cut from wider ones of different widths."""
    from lm_output_head_amd import LogitRules, logits_apply
    z = torch.zeros(1, 50, device="cuda")
    ids = torch.arange(40, dtype=torch.int32, device="cuda").view(1, 40)
    r = LogitRules(50, bias_ids=ids[:, 3:6], bias=torch.ones(1, 3, device="cuda"))
    out = logits_apply(z, r)["logits"]
    want = torch.zeros(1, 50, device="cuda")
    want[0, 3:6] = 1
    assert torch.equal(out, want)


@pytest.mark.parametrize("cut", [False, True])
def test_a_mask_of_no_rows_allows_everything(cut):
    """No grammar at present: every mask_row is outside [0, 0)."""
    from lm_output_head_amd import LogitRules, logits_apply
    z = torch.randn(3, 4000, device="cuda")
    words = torch.zeros(2, 125, dtype=torch.int32, device="cuda")[:0] if cut else torch.zeros(
        0, 125, dtype=torch.int32, device="cuda")
    rows = torch.tensor([-1, 0, 5], dtype=torch.int32, device="cuda")
    out = logits_apply(z, LogitRules(4000, mask=words, mask_row=rows))
    assert torch.equal(out["logits"], z) and torch.equal(out["token"].long(), z.argmax(1))
