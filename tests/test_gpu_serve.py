"""The norm, the int8 head and the rules together, as a decode step runs them:
against the float64 definitions step by step, captured into graphs and replayed
with other inputs, on streams of their own, after the retrieval head."""

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


N, K = 10007, 640


class Step:
    """A head, a norm and rules in buffers that are updated in place."""

    def __init__(self, B, seed=0):
        from lm_output_head_amd import LogitRules, W8A8Head
        g = torch.Generator().manual_seed(seed)
        self.B = B
        self.E = (torch.randn(N, K, generator=g) / 25).bfloat16().cuda()
        self.weight = torch.randn(K, generator=g).bfloat16().cuda()
        self.head = W8A8Head(self.E)
        self.x = torch.zeros(B, K, dtype=torch.bfloat16, device="cuda")
        self.res = torch.zeros(B, K, dtype=torch.bfloat16, device="cuda")
        self.r = {"history": torch.zeros(B, 500, dtype=torch.int32, device="cuda"),
                  "n_history": torch.zeros(B, dtype=torch.int32, device="cuda"),
                  "n_prompt": torch.zeros(B, dtype=torch.int32, device="cuda"),
                  "repetition": torch.full((B,), 1.2, device="cuda"),
                  "frequency": torch.full((B,), 0.1, device="cuda"),
                  "presence": torch.full((B,), 0.2, device="cuda"),
                  "mask": torch.zeros(3, (N + 31) // 32, dtype=torch.int32, device="cuda"),
                  "mask_row": torch.zeros(B, dtype=torch.int32, device="cuda")}
        self.rules = LogitRules(N, **self.r)

    def fill(self, seed):
        g = torch.Generator().manual_seed(seed)
        B = self.B
        self.x.copy_(torch.randn(B, K, generator=g))
        self.res.copy_(torch.randn(B, K, generator=g) * 2)
        self.r["history"].copy_(torch.randint(0, N, (B, 500), generator=g))
        self.r["n_history"].copy_(torch.randint(0, 501, (B,), generator=g))
        self.r["n_prompt"].copy_(torch.randint(0, 501, (B,), generator=g))
        self.r["mask"].copy_(torch.randint(-2 ** 31, 2 ** 31, (3, (N + 31) // 32), generator=g))
        self.r["mask_row"].copy_(torch.randint(-1, 3, (B,), generator=g))

    def run(self, mode, seed=5):
        return self.head.step(self.x, self.weight, residual=self.res, rules=self.rules, mode=mode, temperature=0.75,
                              seed=seed, want_logits=True)


@pytest.mark.parametrize("B", [1, 5, 40])
@pytest.mark.parametrize("mode", [0, 2])
def test_step_against_the_definitions(B, mode):
    """Each operator against float64 on the GPU's own outputs of the one before."""
    from lm_output_head_amd import rmsnorm
    s = Step(B)
    s.fill(B)
    say("step", B, mode)
    out = host(s.run(mode))
    h = rmsnorm(s.x, s.weight, residual=s.res, want_out=False, want_q=True)
    h = host({k: h[k] for k in ("q", "q_scale")})
    codes, scales = (t.cpu().numpy() for t in s.head.codes())
    z = serve_oracle.product(h["q"], h["q_scale"], codes, scales)
    want, size = serve_oracle.apply_rules(z, None, N, **{k: t.cpu().numpy() for k, t in s.r.items()})
    tol = 8 * U * size + 4 * U * 1.25 * np.abs(z)
    fin = np.isfinite(want)
    assert np.array_equal(fin, np.isfinite(out["logits"]))
    assert np.all(np.abs(out["logits"][fin] - want[fin]) <= tol[fin])
    tol[~fin] = 0
    assert not serve_oracle.check_choice(want, tol, None, mode, 0.75, 5, out)
    # and against the head in float64 throughout: int8 on both sides of 640
    # products, each within half a step of its operand
    y, _ = serve_oracle.rmsnorm(s.x.double().cpu().numpy(), s.res.double().cpu().numpy(),
                                s.weight.double().cpu().numpy(), 1e-6, 0.0)
    E = s.E.double().cpu().numpy()
    bound = (0.51 * h["q_scale"][:, None] * np.abs(E).sum(1)[None, :]
             + 0.51 * scales[None, :] * (np.abs(y).sum(1)[:, None] + 0.51 * h["q_scale"][:, None] * K))
    assert np.all(np.abs(z - y @ E.T) <= bound)


@pytest.mark.parametrize("B,mode", [(1, 0), (8, 2), (40, 0)])
def test_captured_steps_replay_exactly(B, mode):
    """Two graphs of steps over different buffers, replayed in turn and at once
    on two streams, with eager work between, equal eager calls."""
    a, b = Step(B, 1), Step(B, 2)
    for s in (a, b):
        s.fill(0)
        s.run(mode)
    torch.cuda.synchronize()
    graphs, outs = [], []
    say("graph capture", B, mode)
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(s.run(mode))
        graphs.append(g)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for rep in range(4):
        for s in (a, b):
            s.fill(10 + rep)
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            if rep % 2:
                with torch.cuda.stream(st):
                    g.replay()
            else:
                g.replay()
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        got = [{k: v.clone() for k, v in o.items()} for o in outs]
        for s, o in zip((a, b), got):
            ref = s.run(mode)
            torch.cuda.synchronize()
            assert all(torch.equal(o[k], ref[k]) for k in ref), rep


def test_steps_on_two_streams_at_once():
    s = [Step(6, 3), Step(6, 4)]
    for x in s:
        x.fill(1)
    ref = [host(x.run(2)) for x in s]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i in (0, 1):
            got[i].append(s[i].head.step(s[i].x, s[i].weight, residual=s[i].res, rules=s[i].rules, mode=2,
                                         temperature=0.75, seed=5, want_logits=True, stream=streams[i]))
    torch.cuda.synchronize()
    for i in (0, 1):
        for o in got[i]:
            assert all(np.array_equal(host(o)[k], ref[i][k], equal_nan=True) for k in ref[i])


def test_step_without_rules_is_the_head():
    from lm_output_head_amd import rmsnorm
    s = Step(4)
    s.fill(3)
    h = rmsnorm(s.x, s.weight, residual=s.res, want_out=False, want_q=True)
    a = s.head.forward(h["q"], h["q_scale"], mode=2, temperature=0.75, seed=5)
    b = s.head.step(s.x, s.weight, residual=s.res, mode=2, temperature=0.75, seed=5)
    assert all(torch.equal(a[k], b[k]) for k in a)


@pytest.mark.parametrize("mode", [0, 2])
def test_rules_after_the_retrieval_head(mode):
    """The norm's h into fh_forward and fh_forward_adaptive, the rules on their
    candidates (an adaptive call's empty places are no tokens)."""
    from lm_output_head_amd import FlashHead, LogitRules, rmsnorm
    from synth import make_problem
    from _gpu import problem_tensors
    pb = make_problem("tiny")
    E, C, H = problem_tensors(pb)
    v, B = pb.shape.v, 6
    head = FlashHead(E, C, pb.C2T, max_batch=B)
    rng = np.random.default_rng(7)
    r = {"history": rng.integers(0, v, (B, 300)).astype(np.int32), "n_prompt": np.full(B, 100, np.int32),
         "repetition": np.full(B, 1.3, np.float32), "presence": np.full(B, 0.4, np.float32)}
    rules = LogitRules(v, **{k: torch.from_numpy(a).cuda() for k, a in r.items()})
    h = rmsnorm(H[:B].contiguous())["out"]
    say("rules after retrieval", mode)
    for o in (head.forward(h, 16, want_retrieved=True),
              head.forward_adaptive(h, 64, 0.7, temperature=0.3, want_retrieved=True),
              head.dense(h, want_logits=True)):
        a = host(head.logits_apply(o, rules, mode=mode, temperature=0.8, seed=2))
        o = host(o)
        want, size = serve_oracle.apply_rules(np.where(np.isneginf(o["logits"]), 0, o["logits"]), o.get("ids"), v, **r)
        tol = 8 * U * size
        assert not serve_oracle.check_choice(want, tol, o.get("ids"), mode, 0.8, 2, a)
    head.close()
