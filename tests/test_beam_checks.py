"""What decoding by beams refuses: through the C ABI (nothing is launched: argument
errors come first) and through the binding; the layouts that the binding makes of
states; and the float64 definitions' own pins.  CPU only."""

import ctypes

import numpy as np
import pytest
import torch

from lm_output_head_amd import _abi, beam
from oracle import beam_oracle

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


# ---------------------------------------------------------------- definitions

def test_select_by_hand():
    """Two beams over four tokens: totals 0 and -1 plus log 1/4 where the logits are
    equal, ties in order; a finished beam beside them; a dead one."""
    z = np.zeros((2, 4))
    score, token, parent = beam_oracle.select(z, [[0.0, -1.0]], 6)
    assert token.tolist() == [[0, 1, 2, 3, 0, 1]] and parent.tolist() == [[0, 0, 0, 0, 1, 1]]
    assert np.allclose(score, np.log(0.25) + np.array([[0, 0, 0, 0, -1, -1]]))
    score, token, parent = beam_oracle.select(z, [[0.0, -1.0]], 6, finished=np.array([[0, 1]]), eos=2)
    assert token.tolist() == [[2, 0, 1, 2, 3, -1]] and parent.tolist() == [[1, 0, 0, 0, 0, -1]]
    assert score[0, 0] == -1 and score[0, 5] == -np.inf
    score, token, parent = beam_oracle.select(z, [[-np.inf, -1.0]], 2)
    assert parent.tolist() == [[1, 1]]
    z[0, 1] = np.inf
    z[1, :] = -np.inf
    assert beam_oracle.select(z, [[0.0, -1.0]], 1)[1].tolist() == [[-1]]
    assert beam_oracle.select(z, [[0.0, -1.0]], 1, lse=np.zeros(2))[1].tolist() == [[1]]


def test_the_oracle_finds_mistakes():
    rng = np.random.default_rng(2)
    z, scores = rng.normal(size=(6, 50)), np.sort(rng.normal(size=(2, 3)))[:, ::-1]
    s, t, p = beam_oracle.select(z, scores, 4)
    out = {"score": s.astype(np.float32), "token": t, "parent": p}
    assert not beam_oracle.check_select(z, scores, 4, out)
    for name, at, value in (("score", (0, 1), s[0, 1] + 1e-3), ("token", (1, 0), (t[1, 0] + 1) % 50),
                            ("parent", (1, 3), (p[1, 3] + 1) % 3), ("token", (0, 2), -1)):
        bad = {k: v.copy() for k, v in out.items()}
        bad[name][at] = value
        assert beam_oracle.check_select(z, scores, 4, bad), (name, at)
    twice = {k: v.copy() for k, v in out.items()}
    for k in twice:
        twice[k][0, 1] = twice[k][0, 0]
    assert beam_oracle.check_select(z, scores, 4, twice)


def test_reorder_by_hand():
    x = np.arange(24).reshape(2, 4, 3)
    got = beam_oracle.reorder(x, [[1, 1], [-1, 0]], dim=1)
    assert np.array_equal(got[:, 0], x[:, 1]) and np.array_equal(got[:, 1], x[:, 1])
    assert np.array_equal(got[:, 2], x[:, 2]) and np.array_equal(got[:, 3], x[:, 2])
    got = beam_oracle.reorder(x, [[1, 0], [0, 0]], lengths=[2, 1, 9, -1], dim=1, length_dim=2)
    assert got[0].tolist() == [[3, 1, 2], [0, 1, 5], [6, 7, 8], [6, 7, 8]]


# ---------------------------------------------------------------------- C ABI

CALL = dict(z=A, ld=5000, ids=None, ld_ids=0, S=2, W=3, n=5000, v=5000, lse=None, scores=A, finished=None, eos=-1, keep=6,
            score=P(1 << 21), token=A, parent=A, done=None, ws=A, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,needle", [
    ({"z": None}, "logits and scores"),
    ({"scores": None}, "logits and scores"),
    ({"score": None}, "out_score"),
    ({"token": None}, "out_token"),
    ({"parent": None}, "out_parent"),
    ({"W": 0}, "beams outside"),
    ({"W": 65}, "beams outside"),
    ({"S": 0}, "sequences * beams"),
    ({"S": 21846}, "sequences * beams"),
    ({"S": 1 << 62}, "sequences * beams"),
    ({"n": 0, "v": 0}, "n and v"),
    ({"v": 5001}, "n = v"),
    ({"n": (1 << 30) + 1, "v": (1 << 30) + 1}, "n and v"),
    ({"keep": 0}, "keep outside"),
    ({"keep": 65}, "keep outside"),
    ({"eos": -2}, "eos outside"),
    ({"eos": 5000}, "eos outside"),
    ({"finished": A}, "need an eos"),
    ({"ld": 4999}, "ld_logits=4999"),
    ({"ids": A, "ld_ids": 4999}, "ld_ids"),
    ({"z": P((1 << 20) + 2)}, "aligned"),
    ({"score": A}, "need keep = beams"),
    ({"finished": A, "done": A, "eos": 2}, "need keep = beams"),
    ({"ws": None}, "workspace"),
    ({"ws_bytes": 6 * 25 * 4 - 1}, "workspace"),
    ({"ws": P((1 << 20) + 8)}, "16-byte aligned"),
])
def test_select_refusals(lib, kw, needle):
    _refused(lib, lib.fh_beam_select(*dict(CALL, **kw).values()), needle)


def test_workspace_sizes(lib):
    assert lib.fh_beam_workspace(2, 3, 5000) == 6 * 25 * 4  # five parts of 1024, four chunks and a sum each
    for args, needle in [((0, 1, 5), "sequences"), ((1, 0, 5), "beams"), ((1, 65, 5), "beams"), ((1, 1, 0), "n outside"),
                         ((1, 1, (1 << 30) + 1), "n outside"), ((65536, 1, 5), "sequences")]:
        _refused(lib, lib.fh_beam_workspace(*args), needle)


LAYOUT = dict(outer=2, mid=3, positions=10, run=8, ld_outer=6 * 240, ld_row=240, ld_mid=80, ld_position=8)


@pytest.mark.parametrize("kw,needle", [
    ({"run": -1}, "negative"),
    ({"mid": -1}, "negative"),
    ({"ld_position": 7}, "overlap"),
    ({"ld_mid": 79}, "overlap"),
    ({"ld_row": 239}, "overlap"),
    ({"ld_outer": 0}, "overlap"),
    ({"ld_row": 0}, "overlap"),
    ({"ld_row": -240}, "overlap"),
    ({"ld_outer": 1 << 60}, "too large"),
    ({"positions": 1 << 40, "run": 1 << 30}, "too large"),
])
def test_reorder_layout_refusals(lib, kw, needle):
    l = _abi.FhBeamLayout(**dict(LAYOUT, **kw))
    _refused(lib, lib.fh_beam_reorder((P * 1)(1 << 24), 1, ctypes.byref(l), 2, 3, A, None, None), needle)


@pytest.mark.parametrize("kw", [
    dict(run=1 << 32, positions=2, ld_position=1 << 33, mid=1, outer=1, ld_row=1 << 40),
    dict(run=1, positions=1 << 32, ld_position=2, mid=1, outer=1, ld_row=1 << 40),
    dict(run=1 << 50, positions=1, mid=1, outer=1, ld_row=1 << 51),
    dict(run=4096, positions=1, mid=1 << 24, outer=1 << 10, ld_mid=4096, ld_row=1 << 36, ld_outer=1 << 40)])
def test_states_too_large_for_one_call(lib, kw):
    l = _abi.FhBeamLayout(**dict(LAYOUT, **kw))
    _refused(lib, lib.fh_beam_reorder((P * 1)(1 << 24), 1, ctypes.byref(l), 2, 3, A, None, None), "too large for one call")


def test_reorder_refusals(lib):
    l, st = _abi.FhBeamLayout(**LAYOUT), (P * 2)(1 << 24, 1 << 25)
    by = ctypes.byref(l)
    for args, needle in [((st, 2, None, 2, 3, A, None), "must not be NULL"), ((st, 2, by, 2, 3, None, None), "must not be NULL"),
                         ((None, 2, by, 2, 3, A, None), "must not be NULL"), ((st, -1, by, 2, 3, A, None), "count"),
                         ((st, 2, by, 2, 65, A, None), "beams outside"), ((st, 2, by, 0, 3, A, None), "sequences"),
                         (((P * 2)(1 << 24, None), 2, by, 2, 3, A, None), "a state is NULL"),
                         ((st, 2, by, 2, 3, P((1 << 20) + 2), None), "aligned"),
                         ((st, 2, by, 2, 3, P((1 << 25) + 2876), None), "must not lie in a state"),
                         ((st, 2, by, 2, 3, A, P(1 << 24)), "must not lie in a state"),
                         (((P * 3)(1 << 24, 1 << 25, 1 << 24), 3, by, 2, 3, A, None), "listed twice")]:
        _refused(lib, lib.fh_beam_reorder(*args, None), needle)
    # nothing to do: nothing is launched
    assert lib.fh_beam_reorder(None, 0, by, 2, 3, A, None, None) == 0
    assert lib.fh_beam_reorder(st, 2, ctypes.byref(_abi.FhBeamLayout(**dict(LAYOUT, mid=0))), 2, 3, A, None, None) == 0


# -------------------------------------------------------------------- binding

def test_binding_select_refusals():
    z, sc = torch.zeros(6, 10), torch.zeros(2, 3)
    i = torch.zeros(2, 3, dtype=torch.int32)
    for kw, needle in [({"logits": z[0]}, "logits must be"), ({"scores": sc[0]}, "scores"),
                       ({"logits": z[:5]}, "logits: expected"), ({"logits": z.double()}, "logits: expected"),
                       ({"scores": sc.double()}, "scores: expected"), ({"scores": torch.zeros(3, 2).t()}, "contiguous"),
                       ({"lse": sc}, "lse: expected"), ({"finished": i.bool()}, "finished: expected"),
                       ({"ids": torch.zeros(6, 9, dtype=torch.int32), "v": 9}, "ids: expected"),
                       ({"ids": torch.zeros(6, 10, dtype=torch.int32)}, "ids need v"), ({}, "one GPU")]:
        with pytest.raises(ValueError, match=needle):
            beam.beam_select(**dict({"logits": z, "scores": sc}, **kw))
    out = dict(out_score=torch.zeros(2, 4), out_token=torch.zeros(2, 4, dtype=torch.int32),
               out_parent=torch.zeros(2, 4, dtype=torch.int32))
    for kw, needle in [({"out_score": torch.zeros(2, 3)}, "out_score"), ({"out_token": torch.zeros(2, 4)}, "out_token"),
                       ({"out_parent": i}, "out_parent"), ({"out_finished": i}, "out_finished"),
                       ({"workspace": torch.zeros(8)}, "workspace"), ({}, "one GPU")]:
        with pytest.raises(ValueError, match=needle):
            beam.fh_beam_select(z, None, 10, None, sc, None, -1, 4, **dict(out, **kw))


def test_layouts():
    def of(t, dim=0, length_dim=None):
        return beam._layout(t, t.shape[dim], dim, length_dim)
    b = torch.bfloat16
    x = torch.zeros(6, 4, 50, 16, dtype=b)  # rows, heads, positions, width
    assert of(x) == (1, 1, 1, 6400, 0, 6400, 0, 0)
    assert of(x, 0, 2) == (1, 4, 50, 32, 0, 6400, 1600, 32)
    assert of(x, 0, 3) == (1, 200, 16, 2, 0, 6400, 32, 2)
    assert of(x[:, :, :20], 0) == (1, 1, 4, 640, 0, 6400, 0, 1600)
    assert of(x[:, 1:3, :20, :8]) == (1, 2, 20, 16, 0, 6400, 1600, 32)
    assert of(x.transpose(1, 2), 0, 1) == of(x, 0, 2)
    y = torch.zeros(3, 2, 6, 50, 4, 16, dtype=b)  # layers, keys and values, rows, positions, heads, width
    assert of(y, 2, 3) == (6, 1, 50, 128, 38400, 6400, 0, 128)
    assert of(y, -4, -3) == of(y, 2, 3)
    assert of(torch.zeros(6, 100, dtype=torch.int32), 0, 1) == (1, 1, 100, 4, 0, 400, 0, 4)
    assert of(torch.zeros(6, dtype=torch.int64)) == (1, 1, 1, 8, 0, 8, 0, 0)
    assert of(torch.zeros(100, 6).t(), 0) == (1, 1, 100, 4, 0, 4, 0, 24)
    for t, dim, length_dim, needle in [(x, 0, 0, "length_dim"), (x, 2, 1, "length_dim"), (x, 0, 4, "length_dim"),
                                       (x[..., ::2], 0, 2, "levels"),
                                       (y.transpose(0, 1), 2, 3, "levels"), (x[:, ::2, ::2, ::2], 0, None, "levels")]:
        with pytest.raises(ValueError, match=needle):
            of(t, dim, length_dim)
    with pytest.raises(ValueError, match="no 5 rows"):
        beam._layout(x, 5, 0, None)
    with pytest.raises(ValueError, match="no 6 rows"):
        beam._layout(x, 6, 4, None)


def test_binding_reorder_refusals():
    x, p = torch.zeros(6, 10), torch.zeros(2, 3, dtype=torch.int32)
    n = torch.zeros(6, dtype=torch.int32)
    for kw, needle in [({"parent": p.view(6)}, "parent must be"), ({"lengths": n}, "go together"),
                       ({"length_dim": 1}, "go together"), ({"states": x[:5]}, "no 6 rows"),
                       ({"lengths": n.view(2, 3), "length_dim": 1}, "one GPU|lengths"), ({}, "one GPU"),
                       ({"parent": p.long()}, "one GPU|parent")]:
        with pytest.raises(ValueError, match=needle):
            beam.beam_reorder(**dict({"states": x, "parent": p}, **kw))


def test_reorder_check_refuses_as_the_call_and_launches_nothing(lib):
    by, st = ctypes.byref(_abi.FhBeamLayout(**LAYOUT)), (P * 2)(1 << 24, 1 << 25)
    for args, needle in [((st, 2, None, 2, 3, A, None), "must not be NULL"), ((st, 2, by, 2, 65, A, None), "beams outside"),
                         ((st, 2, by, 2, 3, P((1 << 25) + 2876), None), "must not lie in a state"),
                         ((st, 2, ctypes.byref(_abi.FhBeamLayout(**dict(LAYOUT, ld_row=239))), 2, 3, A, None), "overlap"),
                         ((st, 2, ctypes.byref(_abi.FhBeamLayout(**dict(LAYOUT, run=1 << 50, positions=1, mid=1, outer=1,
                                                                        ld_row=1 << 51))), 2, 3, A, None),
                          "too large for one call"),
                         (((P * 2)(1 << 24, 1 << 24), 2, by, 2, 3, A, None), "listed twice")]:
        _refused(lib, lib.fh_beam_reorder_check(*args), needle)
    assert lib.fh_beam_reorder_check(st, 2, by, 2, 3, A, None) == 0
    assert lib.fh_beam_reorder_check(None, 0, by, 2, 3, A, None) == 0


def test_one_storage_in_two_layouts_is_refused():
    x, p = torch.zeros(6, 10), torch.zeros(2, 3, dtype=torch.int32)
    for states, kw in [([x, x[:, :4]], {}), ([x, torch.zeros(6, 3), x.view(6, 5, 2).transpose(1, 2)], {}),
                       ([x, x[:, :4]], {"lengths": torch.zeros(6, dtype=torch.int32), "length_dim": 1})]:
        with pytest.raises(ValueError, match="listed twice"):
            beam.beam_reorder(states, p, **kw)
    # nothing lies in an empty one
    with pytest.raises(ValueError, match="one GPU"):
        beam.beam_reorder([x, torch.zeros(6, 3), x[:, :0]], p)


def test_lists_that_reach_into_a_state_are_refused(lib):
    """parent and lengths of 6 beams are 24 bytes: in a state that begins within them
    too, and not in one that begins right behind them or ends right before."""
    l = _abi.FhBeamLayout(**LAYOUT)
    by, first, behind = ctypes.byref(l), 1 << 24, (1 << 24) + 2 * 6 * 240
    for at in (first - 20, first - 4, first, behind - 4):
        _refused(lib, lib.fh_beam_reorder_check((P * 1)(first), 1, by, 2, 3, P(at), None), "must not lie in a state")
        _refused(lib, lib.fh_beam_reorder_check((P * 1)(first), 1, by, 2, 3, A, P(at)), "must not lie in a state")
        _refused(lib, lib.fh_beam_reorder((P * 1)(first), 1, by, 2, 3, A, P(at), None), "must not lie in a state")
    for at in (first - 24, behind):
        assert lib.fh_beam_reorder_check((P * 1)(first), 1, by, 2, 3, P(at), P(at)) == 0
