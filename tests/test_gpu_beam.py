"""GPU parity of decoding by beams: the choice of continuations (tolerances in
oracle/beam_oracle.py), the reordering of states (whole bytes, exactly), and both
after the heads and the rules, as a decode loop runs them."""

import numpy as np
import pytest
import torch

from oracle import beam_oracle, serve_oracle

from _gpu import host, need_gpu, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
NEG = -np.inf


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    from lm_output_head_amd import load_library
    load_library()


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def run(z, scores, keep, ids=None, v=None, lse=None, finished=None, eos=-1):
    from lm_output_head_amd import beam_select
    out = beam_select(dev(z), dev(scores), keep=keep, ids=dev(ids), v=v, lse=dev(lse), finished=dev(finished), eos=eos)
    return host(out)


def check(z, scores, keep, exact=False, **kw):
    out = run(z, scores, keep, **kw)
    for name in ("score", "token", "parent"):
        assert out[name].shape == (scores.shape[0], keep)
    assert not beam_oracle.check_select(z, scores, keep, out, exact, **kw)
    return out


def make(S, W, n, seed, mask=0.0):
    rng = np.random.default_rng(seed)
    z = (rng.normal(size=(S * W, n)) * 3).astype(np.float32)
    if mask:
        z[rng.random(z.shape) >= mask] = NEG
    scores = -np.sort(rng.uniform(5, 12, (S, W)), 1).astype(np.float32)
    return rng, z, scores


SIZES = [(1, 1, 1, 1), (1, 1, 1, 5), (1, 4, 1000, 8), (3, 5, 4097, 5), (2, 8, 151936, 16), (1, 64, 300, 64),
         (2, 32, 5000, 64), (7, 3, 255, 6), (1, 2, 1024, 64), (5, 1, 70001, 1), (1, 1, 16385, 64), (40, 2, 3, 7),
         (2, 16, 1025, 32), (1, 10, 262144, 20), (300, 4, 2000, 4), (1, 64, 20000, 64), (1, 16, 1024, 16)]


@pytest.mark.parametrize("S,W,n,keep", SIZES)
def test_sizes(S, W, n, keep):
    rng, z, scores = make(S, W, n, S + W + n)
    say("beams", S, W, n, keep)
    check(z, scores, keep)
    check(z, scores, keep, lse=rng.uniform(8, 12, S * W).astype(np.float32))


@pytest.mark.parametrize("S,W,n,keep", [(3, 4, 9000, 8), (2, 8, 300, 16), (1, 32, 40000, 64)])
@pytest.mark.parametrize("mask", [0.5, 0.01, 0.0005])
def test_masks(S, W, n, keep, mask):
    """Rows of few tokens and of none, their places far apart."""
    rng, z, scores = make(S, W, n, n, mask)
    z[0] = NEG
    say("beams under masks", S, W, n, keep, mask)
    check(z, scores, keep)


@pytest.mark.parametrize("low", [-3.4028234663852886e38, -1e4, -65504.0])
def test_masks_of_a_finite_value(low):
    """Rows masked with a type's lowest value: the masked tokens are equal, and come
    in order once the others are out."""
    rng, z, scores = make(2, 4, 5000, 9)
    z[rng.random(z.shape) < 0.9995] = low
    lse = np.full(8, 3.0, np.float32)
    say("beams, finite masks", low)
    check(z, scores, 32, lse=lse)
    check(np.full_like(z, low), scores, 32, exact=True, lse=lse)


@pytest.mark.parametrize("S,W,n,keep", [(2, 4, 50000, 8), (1, 64, 3000, 64), (2, 3, 700, 64), (1, 5, 200, 32)])
def test_equal_totals_come_in_order(S, W, n, keep):
    """Few different values, many ties within and between beams."""
    rng = np.random.default_rng(n)
    say("beams with ties", S, W, n, keep)
    lse = np.full(S * W, 2.0, np.float32)
    scores = np.full((S, W), -1.5, np.float32)
    check(np.zeros((S * W, n), np.float32), scores, keep, exact=True, lse=lse)
    z = rng.integers(0, 3, (S * W, n)).astype(np.float32)
    check(z, scores, keep, exact=True, lse=lse)
    check(np.where(z == 0, np.float32(-0.0), z - 1), scores, keep, exact=True, lse=lse)  # -0 is 0
    rare = (rng.random((S * W, n)) < 5.0 / n) * np.float32(4)
    check(rare, scores, keep, exact=True, lse=lse)
    check(np.sort(rng.normal(size=(S * W, n)).astype(np.float32), 1), scores, keep, lse=lse)
    # equal rows: the same log-sum-exp, whatever it rounds to
    check(np.repeat(z[:1], S * W, 0), scores, keep, exact=False)
    out = run(np.zeros((S * W, n), np.float32), scores, keep)
    assert out["parent"].tolist() == [[min(r // n, W - 1) if r < W * n else -1 for r in range(keep)]] * S


@pytest.mark.parametrize("S,W,n,keep", [(1, 8, 300000, 16), (1, 40, 9000, 64), (2, 3, 1100000, 64)])
def test_rows_that_do_not_stay_in_registers(S, W, n, keep):
    """More chunks than a lane holds, or more beams than waves hold: ordinary rows,
    ascending ones, equal ones, masked ones."""
    rng, z, scores = make(S, W, n, n)
    say("long beams", S, W, n, keep)
    check(z, scores, keep)
    lse = np.full(S * W, 4.0, np.float32)
    z[0].sort()
    check(z, scores, keep, lse=lse)
    z[1] = 0.5
    check(z, scores, keep, lse=lse)
    finished = (rng.random((S, W)) < 0.3).astype(np.int32)
    z[2, rng.random(n) < 0.9999] = NEG
    check(z, scores, keep, finished=finished, eos=7)


def test_first_step_and_dead_beams():
    rng, z, scores = make(3, 5, 3000, 4)
    scores[:, 1:] = NEG
    out = check(z, scores, 5)
    assert np.all(out["parent"] == 0)
    scores[1] = NEG
    scores[2, 0] = np.nan
    out = check(z, scores, 5)
    assert np.all(out["parent"][1:] == -1) and np.all(out["token"][1:] == -1) and np.all(np.isneginf(out["score"][1:]))


@pytest.mark.parametrize("n,ids", [(5000, False), (200, False), (2000, True)])
def test_finished_beams(n, ids):
    rng, z, scores = make(4, 6, n, 11)
    v = 9000 if ids else n
    tok = np.stack([rng.permutation(v)[:n] for _ in range(24)]).astype(np.int32) if ids else None
    finished = (rng.random((4, 6)) < 0.4).astype(np.int32) * 7
    finished[2] = 1
    finished[3, 0], scores[3, 0] = 1, NEG
    z[np.repeat(finished.ravel() != 0, n).reshape(24, n)] = np.nan
    scores[0] += 4 * finished[0]
    say("finished beams", n, ids)
    for keep in (3, 6, 40):
        check(z, scores, keep, ids=tok, v=v if ids else None, finished=finished, eos=42)
    z[1, 42] = 50.0  # a beam that finishes now
    out = check(z, scores, 6, finished=finished, eos=42, ids=tok, v=v if ids else None)
    assert out["finished"].sum() >= 6


@pytest.mark.parametrize("S,W,n,keep,live", [(3, 32, 1000, 64, 12), (2, 16, 700, 32, 3), (1, 64, 2000, 64, 30),
                                             (2, 4, 2000, 64, 1), (1, 10, 30000, 64, 1), (2, 32, 400, 64, 20)])
def test_few_beams_left(S, W, n, keep, live):
    """Not many more places of 256 than continuations: a border among the largest
    of each leaves thousands, and one among all of them is needed."""
    rng, z, scores = make(S, W, n, W + n)
    finished = np.ones((S, W), np.int32)
    for s in range(S):
        finished[s, rng.permutation(W)[:live]] = 0
    say("few beams left", S, W, n, keep, live)
    check(z, scores, keep, finished=finished, eos=7)
    check(z, scores, keep, finished=finished, eos=7, lse=rng.uniform(8, 12, S * W).astype(np.float32))


@pytest.mark.parametrize("S,W,n", [(3, 4, 8192), (2, 4, 8193), (3, 8, 4096), (2, 8, 4097), (3, 16, 2048), (2, 16, 2049),
                                   (3, 1, 8192), (2, 2, 1025), (1, 3, 6000), (1, 12, 1500), (1, 5, 3000)])
@pytest.mark.parametrize("listed", [False, True])
def test_rows_that_one_workgroup_scans(S, W, n, listed):
    """Up to two parts of 1024 a wave, and just beyond; with dead and finished beams."""
    rng, z, scores = make(S, W, n, W + n, 0.6)
    z[S * W // 2] = NEG
    finished = (rng.random((S, W)) < 0.3).astype(np.int32)
    scores[0, W // 3] = NEG
    kw = dict(finished=finished, eos=2)
    if listed:
        kw.update(ids=np.stack([rng.permutation(n + 50)[:n] for _ in range(S * W)]).astype(np.int32), v=n + 20)
    for keep in (1, W, 2 * W):
        say("short rows", S, W, n, listed, keep)
        check(z, scores, keep, **kw)


def test_candidates():
    """Listed tokens in no order, some of them no tokens, with the rows' sums over
    more than the list; a token listed twice is two continuations."""
    rng, z, scores = make(2, 4, 8192, 3)
    v = 128256
    ids = rng.integers(-3, v + 3, z.shape).astype(np.int32)
    ids[:, 77] = -1
    z[:, 77] = 60.0
    ids[:, 500] = ids[:, 900]
    z[:, 500], z[:, 900] = 20.0, 21.0
    z[3, ids[3] < 0] = np.nan  # no token: what its logit is does not matter
    lse = rng.uniform(20, 22, 8).astype(np.float32)
    say("beams over candidates")
    out = check(z, scores, 8, ids=ids, v=v, lse=lse)
    assert (out["token"] >= 0).all()
    check(z, scores, 8, ids=ids, v=v)


def test_non_finite_logits():
    rng, z, scores = make(1, 6, 4000, 8)
    z[0, 100], z[1, 200], z[2, 300], z[2, 301], z[3], z[4, ::2] = np.nan, np.inf, np.inf, -np.inf, np.nan, NEG
    out = check(z, scores, 16)
    assert set(out["parent"][0].tolist()) <= {4, 5}
    lse = np.full(6, 9.0, np.float32)
    lse[5] = np.nan
    out = check(z, scores, 16, lse=lse)
    assert out["parent"][0, :2].tolist() == [1, 2] and np.all(np.isposinf(out["score"][0, :2])) and 5 not in out["parent"]
    lse[:] = (-np.inf, 0, np.inf, 0, 0, 0)
    check(z, scores, 16, lse=lse)
    big = scores.copy()
    big[0, 5] = np.inf
    check(z, big, 16, lse=np.zeros(6, np.float32))
    check((z * np.float32(1e37)).astype(np.float32), scores, 16, lse=np.zeros(6, np.float32))


@pytest.mark.parametrize("off", [0, 1, 3])
def test_strides_and_what_lies_between(off):
    from lm_output_head_amd import fh_beam_select, fh_beam_workspace
    for S, W, n, keep, ld in [(2, 3, 5001, 7, 5003), (1, 4, 130, 4, 160)]:
        rng, z, scores = make(S, W, n, ld + off)
        ids = np.stack([rng.permutation(9000)[:n] for _ in range(S * W)]).astype(np.int32)
        wide = torch.full((S * W + 1, ld + 4), 1e30, device="cuda")
        wids = torch.full((S * W + 1, ld + 4), 5, dtype=torch.int32, device="cuda")
        wide[:-1, off:off + n], wids[:-1, off:off + n] = dev(z), dev(ids)
        outs = torch.full((4, S + 2, keep), 7.0, device="cuda")
        score, (tok, par, done) = outs[0, 1:-1], [t.view(torch.int32) for t in outs[1:, 1:-1]]
        size = fh_beam_workspace(S, W, n)
        ws = torch.full((size + 64,), 9, dtype=torch.uint8, device="cuda")
        say("beams strides", S, W, n, off)
        for use in (False, True):
            kw = {"ids": ids, "v": 9000} if use else {"ids": None, "v": n}
            fh_beam_select(wide[:-1, off:off + n], wids[:-1, off:off + n] if use else None, kw["v"], None, dev(scores),
                           torch.zeros(S, W, dtype=torch.int32, device="cuda"), 5, keep, score, tok, par, done, ws[:size])
            got = host({"score": score, "token": tok, "parent": par, "finished": done})
            assert not beam_oracle.check_select(z, scores, keep, got, eos=5, finished=np.zeros((S, W)), **kw)
            assert torch.all(outs[:, 0] == 7) and torch.all(outs[:, -1] == 7) and torch.all(ws[size:] == 9)


def test_outputs_on_their_inputs():
    from lm_output_head_amd import fh_beam_select, fh_beam_workspace
    rng, z, scores = make(3, 4, 3000, 2)
    finished = np.array([[0, 1, 0, 0]] * 3, np.int32)
    ref = run(z, scores, 4, finished=finished, eos=9)
    sc, fin, tok, par = dev(scores), dev(finished), dev(finished), dev(finished)
    ws = torch.empty(fh_beam_workspace(3, 4, 3000), dtype=torch.uint8, device="cuda")
    say("beams in place")
    fh_beam_select(dev(z), None, 3000, None, sc, fin, 9, 4, sc, tok, par, fin, ws)
    got = host({"score": sc, "finished": fin, "token": tok, "parent": par})
    assert all(np.array_equal(got[k], ref[k]) for k in ref)


# ---------------------------------------------------------------- reordering

def parents(S, W, seed, stay=0.3):
    rng = np.random.default_rng(seed)
    p = rng.integers(0, W, (S, W)).astype(np.int32)
    own = rng.random((S, W)) < stay
    p[own] = np.broadcast_to(np.arange(W, dtype=np.int32), (S, W))[own]
    p[rng.random((S, W)) < 0.05] = -1
    p[rng.random((S, W)) < 0.05] = W
    return p


def states_like(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if dtype.is_floating_point:
        return torch.randn(shape, generator=g, device="cuda").to(dtype)
    return torch.randint(-100, 100, shape, generator=g, device="cuda").to(dtype)


def raw(t):
    """The bytes of a tensor as an array with one more dimension."""
    return t.contiguous().view(torch.uint8).view(*t.shape, t.element_size()).cpu().numpy()


@pytest.mark.parametrize("S,W", [(1, 2), (3, 4), (2, 5), (1, 8), (2, 16), (1, 17), (2, 32), (1, 64), (5, 1)])
@pytest.mark.parametrize("shape,dtype,length_dim", [
    ((3, 50, 16), torch.bfloat16, 2), ((50, 3, 24), torch.bfloat16, 1), ((2, 33, 10), torch.float32, 2),
    ((1000,), torch.int32, 1), ((777,), torch.uint8, 1), ((), torch.int64, None), ((5,), torch.float16, None),
    ((3, 37, 5), torch.uint8, 2), ((129, 13), torch.int8, 1), ((2, 4100), torch.bfloat16, 2)])
def test_reorder(S, W, shape, dtype, length_dim):
    from lm_output_head_amd import beam_reorder
    x = states_like((S * W, *shape), dtype, S + W)
    p = parents(S, W, W)
    say("reorder", S, W, shape, dtype)
    old = raw(x)
    beam_reorder(x, dev(p))
    torch.cuda.synchronize()
    assert np.array_equal(raw(x), beam_oracle.reorder(old, p))
    if length_dim is not None:
        L = shape[length_dim - 1]
        lengths = np.random.default_rng(W).integers(-1, L + 3, S * W).astype(np.int32)
        old = raw(x)
        beam_reorder(x, dev(p), lengths=dev(lengths), length_dim=length_dim)
        torch.cuda.synchronize()
        assert np.array_equal(raw(x), beam_oracle.reorder(old, p, lengths, 0, length_dim))


def test_reorder_views_and_layers():
    """Views of wider states, layers before the rows, positions before and behind
    the heads, odd offsets: what is not part of the view stays."""
    from lm_output_head_amd import beam_reorder
    S, W = 2, 3
    p = parents(S, W, 5, 0.2)
    lengths = np.array([5, 9, 20, 0, 13, 40], np.int32)
    base = states_like((4, 2, 7, 3, 22, 18), torch.bfloat16, 1)  # layers, keys and values, rows, heads, positions, width
    for view, kw in [(base[:, :, :6], {"length_dim": 4}), (base[:, :, 1:7, :, 1:21, 1:18], {"length_dim": 4}),
                     (base[1:, 0, 1:, :, :, :17], {"dim": 1, "length_dim": 3}),
                     (base.transpose(3, 4)[:, :, :6], {"length_dim": 3}), (base[:, 1, :6, 2, 3:20], {"dim": 1}),
                     (base[2, 1, :6, :, :, 4], {"dim": 0, "length_dim": 2})]:
        if "dim" not in kw:
            kw["dim"] = 2
        use = dict(kw, lengths=dev(lengths)) if "length_dim" in kw else kw
        old, rest = raw(view), base.clone()
        say("reorder views", tuple(view.shape), kw)
        beam_reorder(view, dev(p), **use)
        torch.cuda.synchronize()
        want = beam_oracle.reorder(old, p, lengths if "length_dim" in kw else None, kw["dim"],
                                   kw.get("length_dim"))
        assert np.array_equal(raw(view), want)
        new = base.clone()
        view.copy_(torch.from_numpy(old).cuda().view(torch.bfloat16).view(view.shape))
        assert torch.equal(base.view(torch.int16), rest.view(torch.int16))  # nothing else had moved
        base.copy_(new)


def test_reorder_of_interleaved_states():
    """Keys and values as views of one cache, their bytes between each other's."""
    from lm_output_head_amd import beam_reorder
    S, W = 2, 4
    p = parents(S, W, 3)
    base = states_like((S * W, 30, 2, 3, 20), torch.bfloat16, 2)  # rows, positions, keys and values, heads, width
    k, v = base[:, :, 0], base[:, :, 1]
    old = raw(k), raw(v)
    lengths = np.arange(4, 28, 3).astype(np.int32)
    say("reorder interleaved")
    beam_reorder([k, v], dev(p), lengths=dev(lengths), length_dim=1)
    torch.cuda.synchronize()
    assert np.array_equal(raw(k), beam_oracle.reorder(old[0], p, lengths, 0, 1))
    assert np.array_equal(raw(v), beam_oracle.reorder(old[1], p, lengths, 0, 1))


def test_reorder_of_many_states():
    """More states than one launch takes, of two layouts, in one call."""
    from lm_output_head_amd import FlashHeadError, beam_reorder
    S, W = 3, 4
    p = parents(S, W, 1)
    xs = [states_like((S * W, 40, 6), torch.bfloat16, i) for i in range(130)] + [states_like((S * W, 40), torch.int32, 7)]
    old = [raw(x) for x in xs]
    lengths = np.full(S * W, 31, np.int32)
    say("reorder many")
    beam_reorder(xs, dev(p), lengths=dev(lengths), length_dim=1)
    torch.cuda.synchronize()
    assert all(np.array_equal(raw(x), beam_oracle.reorder(o, p, lengths, 0, 1)) for x, o in zip(xs, old))
    with pytest.raises(FlashHeadError, match="listed twice"):
        beam_reorder([xs[0], xs[0]], dev(p))
    beam_reorder([], dev(p))
    beam_reorder([torch.empty(S * W, 0, device="cuda")], dev(p))


def test_reorder_past_32_bits():
    """A cache whose rows lie more than 2^32 bytes apart from the first."""
    from lm_output_head_amd import beam_reorder
    W, L, D = 3, 1 << 20, 2048
    x = torch.zeros(2 * W, L, D, dtype=torch.int8, device="cuda")  # 12 GiB
    for r in range(2 * W):
        x[r, :, 0] = r + 1
        x[r, -1, -1] = 10 + r
    p = np.array([[2, 0, 1], [1, 1, 0]], np.int32)
    say("reorder past 32 bits")
    beam_reorder(x, dev(p), lengths=torch.full((2 * W,), L, dtype=torch.int32, device="cuda"), length_dim=1)
    src = [2, 0, 1, 4, 4, 3]
    for r in range(2 * W):
        assert torch.all(x[r, :, 0] == src[r] + 1) and x[r, -1, -1] == 10 + src[r] and not x[r, 5, 1:].any()


# ------------------------------------------------------------- a decode loop

class Loop:
    """Beams over an fp8 (or int8) head with rules, caches and histories in buffers
    that are updated in place, as a program keeps them."""

    V, K, L = 5003, 384, 60

    def __init__(self, kind, S, W, seed=0):
        from lm_output_head_amd import FP8Head, LogitRules, W8A8Head
        g = torch.Generator().manual_seed(seed)
        self.S, self.W, R = S, W, S * W
        E = (torch.randn(self.V, self.K, generator=g) / 20).bfloat16().cuda()
        self.head = FP8Head(E) if kind == "fp8" else W8A8Head(E)
        self.weight = torch.rand(self.K, generator=g).bfloat16().cuda()
        self.x = torch.zeros(R, self.K, dtype=torch.bfloat16, device="cuda")
        self.caches = [torch.zeros(R, 2, self.L, 16, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
        i32 = {"dtype": torch.int32, "device": "cuda"}
        self.history = torch.zeros(R, self.L, **i32)
        self.length = torch.zeros(R, **i32)
        self.scores = torch.zeros(S, W, device="cuda")
        self.finished = torch.zeros(S, W, **i32)
        self.old_length = torch.zeros(R, **i32)
        self.rules = LogitRules(self.V, history=self.history, n_history=self.length,
                                repetition=torch.full((R,), 1.3, device="cuda"),
                                presence=torch.full((R,), 0.2, device="cuda"))

    def start(self):
        self.length.fill_(3)
        self.history.zero_()
        self.scores.fill_(-float("inf"))
        self.scores[:, 0] = 0
        self.finished.zero_()
        for c in self.caches:
            c.zero_()

    def step(self, stream=None):
        from lm_output_head_amd import beam_reorder
        out = self.head.beam_step(self.x, self.scores, self.weight, rules=self.rules, finished=self.finished, eos=17,
                                  want_logits=True)
        self.scores.copy_(out["score"])
        self.finished.copy_(out["finished"])
        self.old_length.copy_(self.length)
        beam_reorder(self.caches, out["parent"], lengths=self.old_length, length_dim=2)
        beam_reorder([self.history], out["parent"], lengths=self.old_length, length_dim=1)
        beam_reorder(self.length, out["parent"])
        self.history.scatter_(1, self.length.long()[:, None], out["token"].view(-1, 1).clamp(min=0))
        self.length.add_(1)
        return out


def feed(loop, i):
    """New hidden states, and what a model would have written into its caches."""
    g = torch.Generator().manual_seed(i)
    loop.x.copy_(torch.randn(loop.x.shape, generator=g))
    for j, c in enumerate(loop.caches):
        c[:, :, 2 + i] = torch.randn(c.shape[0], 2, 16, generator=g).to(c.device) + j


@pytest.mark.parametrize("kind", ["fp8", "int8"])
def test_a_decode_loop(kind):
    """Every step against the float64 definitions on the GPU's own inputs to it."""
    loop = Loop(kind, 3, 4)
    loop.start()
    V = loop.V
    for i in range(8):
        feed(loop, i + 1)
        before = host({"scores": loop.scores, "finished": loop.finished, "history": loop.history, "length": loop.length})
        old = [raw(c) for c in loop.caches]
        say("beam loop", kind, i)
        out = host(loop.step())
        after = host({"history": loop.history, "length": loop.length, "scores": loop.scores})
        z = out["logits"].astype(np.float64)
        got = {k: out[k] for k in ("score", "token", "parent", "finished")}
        assert not beam_oracle.check_select(z, before["scores"], 4, got, finished=before["finished"], eos=17)
        p = out["parent"]
        assert np.all(p >= 0) and np.array_equal(after["scores"], out["score"])
        for c, o in zip(loop.caches, old):
            assert np.array_equal(raw(c), beam_oracle.reorder(o, p, before["length"], 0, 2))
        h = beam_oracle.reorder(before["history"], p, before["length"], 0, 1)
        h[np.arange(12), before["length"]] = out["token"].ravel()
        assert np.array_equal(after["history"], h) and np.all(after["length"] == 4 + i)
        # the logits: the head's product of the same step, under the rules' definition
        q, s = loop.head._states(loop.x, loop.weight, None, 1e-6, 0.0)
        plain = loop.head.matmul(q, s).cpu().numpy()
        want, size = serve_oracle.apply_rules(plain, None, V, history=before["history"], n_history=before["length"],
                                              repetition=np.full(12, np.float32(1.3)), presence=np.full(12, np.float32(0.2)))
        assert np.all(np.abs(z - want) <= 8 * U * size + 4 * U * 1.3 * np.abs(plain))
    if kind == "fp8":
        loop.head.close()


def test_captured_loops_replay_exactly():
    """Two graphs of whole steps over different buffers, replayed in turn and at once
    on two streams, with eager work between, equal eager loops."""
    loops = [Loop("fp8", 2, 3, 1), Loop("fp8", 1, 5, 2)]
    eager = [Loop("fp8", 2, 3, 1), Loop("fp8", 1, 5, 2)]
    graphs, outs = [], []
    for l in loops:
        l.start()
        l.step()  # every kernel is loaded before the capture
    torch.cuda.synchronize()
    say("beam loop capture")
    for l in loops:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(l.step())
        graphs.append(g)
    for l in loops + eager:
        l.start()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for i in range(6):
        for l in loops + eager:
            feed(l, i + 1)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            if i % 2:
                with torch.cuda.stream(st):
                    g.replay()
            else:
                g.replay()
        torch.cuda.synchronize()
        for l, e, o in zip(loops, eager, outs):
            ref = e.step()
            torch.cuda.synchronize()
            assert all(torch.equal(o[k], ref[k]) for k in ref), i
            assert torch.equal(l.history, e.history) and torch.equal(l.scores, e.scores)
            assert all(torch.equal(a, b) for a, b in zip(l.caches, e.caches))


def test_beams_after_the_retrieval_head():
    """The retrieved candidates of each beam, the log-sum-exp that the head gives."""
    from lm_output_head_amd import FlashHead, beam_select
    from synth import make_problem
    from _gpu import problem_tensors
    pb = make_problem("tiny")
    E, C, H = problem_tensors(pb)
    head = FlashHead(E, C, pb.C2T, max_batch=6)
    scores = np.array([[-1, -2.5, -3], [-4, -4.5, -np.inf]], np.float32)
    o = head.forward(H[:6].contiguous(), 16, want_retrieved=True)
    say("beams after retrieval")
    got = host(beam_select(o["logits"], dev(scores), keep=6, ids=o["ids"], v=pb.shape.v, lse=o["lse"]))
    o = host(o)
    assert not beam_oracle.check_select(o["logits"], scores, 6, got, ids=o["ids"], v=pb.shape.v, lse=o["lse"])
    head.close()


def test_select_on_another_stream():
    from lm_output_head_amd import beam_reorder, beam_select
    rng, z, scores = make(2, 4, 20000, 6)
    ref = run(z, scores, 8)
    zt, st = dev(z), dev(scores)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    x = states_like((8, 100), torch.int32, 1)
    old = raw(x)
    torch.cuda.synchronize()
    got = [beam_select(zt, st, keep=8, stream=s) for _ in range(5)]
    p = got[0]["parent"][:, :4]
    with torch.cuda.stream(s):
        p = p.contiguous()
    beam_reorder(x, p, stream=s)
    s.synchronize()
    for o in got:
        assert all(np.array_equal(host(o)[k], ref[k]) for k in ref)
    assert np.array_equal(raw(x), beam_oracle.reorder(old, ref["parent"][:, :4]))
