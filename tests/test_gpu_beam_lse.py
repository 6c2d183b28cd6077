"""How well the beams' choice knows a log-sum-exp that it computes itself.

u = 2^-24.  With x = z - m, m the largest of a part or a row, an exponential is within
(2 + |x|) 2 u of itself (its argument's two roundings, its own), counted once for the
part's and once for the parts'; their mean over the row's probabilities p is at most
4 u (2 + sum p |x|), and sum p |x| <= ln n (the entropy is ln n at most and the
largest's -ln p is not negative).  24 roundings of a part's sum, one of its product
with its exponential, one to spare: 2 4 u (2 + ln n) + 26 u = (42 + 8 ln n) u.  A total
is then rounded to float32."""

import math

import pytest
import torch

from _gpu import need_gpu, say

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    from lm_output_head_amd import load_library
    load_library()


@pytest.mark.parametrize("W", [1, 4, 8, 24, 40])
@pytest.mark.parametrize("n", [1, 2, 63, 1000, 1025, 4096, 20000, 128256, 300000])
def test_lse_is_within_its_bound(n, W):
    from lm_output_head_amd import beam_select
    S = 3
    g = torch.Generator(device="cuda").manual_seed(n + W)
    base = torch.randn(S * W, n, generator=g, device="cuda")
    bound = (42 + 8 * math.log(n)) * U
    for name, z in [("normal", base * 3), ("peaked", base * 30), ("flat", base * 0.01 + 20), ("equal", base * 0 - 7),
                    ("far up", base * 3 + 1000), ("masked", base.masked_fill(base < 0, -math.inf)),
                    ("lowest", base.masked_fill(base < 0, torch.finfo(torch.float32).min))]:
        say("beams' lse", n, W, name)
        # one beam of each sequence at a time, at 0: its best total is its largest logit less its lse
        for w in range(0, W, max(1, W // 3)):
            scores = torch.full((S, W), -math.inf, device="cuda")
            scores[:, w] = 0
            out = beam_select(z, scores, keep=1)
            rows = z.view(S, W, n)[:, w].double()
            want = rows.max(1).values - torch.logsumexp(rows, 1)
            none = rows.max(1).values == -math.inf
            assert torch.all(torch.isneginf(out["score"][none, 0])) and torch.all(out["token"][none, 0] == -1)
            err = (out["score"][:, 0].double() - want).abs()[~none]
            assert torch.all(err <= bound + U * (want.abs()[~none] + bound)), (name, w, float(err.max()), bound)


def test_neighbours_within_a_beam_are_in_order():
    """Logits one unit apart, in any order of places; with their lse as float32 knows it
    the totals are those of the definition, between beams too."""
    from lm_output_head_amd import beam_select
    n, W, keep = 3000, 4, 64
    z = torch.zeros(W, n, device="cuda")
    near = torch.full((keep,), 9.0, device="cuda")
    for i in range(1, keep):
        near[i] = torch.nextafter(near[i - 1], torch.tensor(-100.0, device="cuda"))
    at = torch.randperm(n, generator=torch.Generator().manual_seed(1))[:keep].cuda()
    z[2, at] = near
    scores = torch.full((1, W), -1e4, device="cuda")
    scores[0, 2] = 0
    say("beams' neighbours")
    out = beam_select(z, scores, keep=keep)
    assert torch.equal(out["token"][0].long(), at) and torch.all(out["parent"] == 2)
    # the same near logits in two beams, one a quarter of a unit lower by its score
    z[1, at] = near
    scores[0, 1] = -2.0 ** -22
    lse = torch.zeros(W, device="cuda")
    out = beam_select(z, scores, keep=keep, lse=lse)
    assert torch.equal(out["token"][0, ::2].long(), at[:keep // 2])
    assert torch.equal(out["token"][0, 1::2].long(), at[:keep // 2])
    assert out["parent"][0].tolist() == [2, 1] * (keep // 2)
