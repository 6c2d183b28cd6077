"""beam_reorder over states of several layouts: all of them or none."""

import pytest
import torch

from _gpu import need_gpu, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    need_gpu()
    from lm_output_head_amd import load_library
    load_library()


def state(*shape, dt=torch.int32):
    return torch.arange(torch.Size(shape).numel(), device="cuda").view(shape).to(dt)


def parents(S, W):
    """Every beam continues the one behind it."""
    return ((torch.arange(W, dtype=torch.int32, device="cuda") + 1) % W).repeat(S, 1)


def refused():
    """Calls whose second layout is refused, each by a check of its own."""
    from lm_output_head_amd import FlashHeadError
    first, parent = state(6, 10), parents(2, 3)
    yield "strides overlap", [first, state(1, 20).expand(6, 20)], dict(parent=parent), FlashHeadError
    held = state(40)
    held[14:20] = parent.reshape(-1)
    yield "parent in a state", [first, held[:36].view(6, 6)], dict(parent=held[14:20].view(2, 3)), FlashHeadError
    held = state(6, 9)
    held.view(-1)[12:18] = 4
    yield ("lengths in a state", [first, held],
           dict(parent=parent, lengths=held.view(-1)[12:18], length_dim=1), FlashHeadError)
    yield "another GPU", [first, torch.zeros(6, 4)], dict(parent=parent), ValueError
    yield "no rows", [first, state(5, 4)], dict(parent=parent), ValueError


@pytest.mark.parametrize("i", range(5))
def test_a_refused_call_moves_nothing(i):
    from lm_output_head_amd import beam_reorder
    name, states, kw, error = list(refused())[i]
    before = [t.clone() for t in states]
    say("reorder refused", name)
    with pytest.raises(error):
        beam_reorder(states, **kw)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(states, before)), name


def test_states_of_several_layouts():
    from lm_output_head_amd import beam_reorder
    states = [state(6, 10), state(6, 3, dt=torch.int64), state(6, 4, 50, 8, dt=torch.bfloat16), state(6, 10)]
    want = [t.view(2, 3, *t.shape[1:]).roll(-1, 1).reshape(t.shape) for t in states]
    say("reorder layouts")
    beam_reorder(states, parents(2, 3))
    assert all(torch.equal(a, b) for a, b in zip(states, want))


def test_one_storage_in_two_layouts_is_not_moved():
    from lm_output_head_amd import beam_reorder
    x = state(6, 10)
    before = x.clone()
    say("reorder of one storage twice")
    with pytest.raises(ValueError, match="listed twice"):
        beam_reorder([x, x[:, :4]], parents(2, 3))
    assert torch.equal(x, before)


def test_keys_and_values_that_interleave():
    """States of two layouts whose bytes lie between each other's."""
    from lm_output_head_amd import beam_reorder
    both = state(6, 4, 12)
    want = both.view(2, 3, 4, 12).roll(-1, 1).reshape(6, 4, 12)
    say("reorder interleaved")
    beam_reorder([both[:, :, :5], both[:, :, 5:9], both[:, :, 9:]], parents(2, 3))
    assert torch.equal(both, want)
