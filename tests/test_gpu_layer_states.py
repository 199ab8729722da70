"""States that decode steps update in place, next to autograd graphs that
saved them (needs an MI355X)."""
import pytest
import torch

import gated_delta_rule_66_amd as gdr

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rand(*shape, dtype=BF, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def conv():
    x, w, state = rand(2, 9, 16), rand(16, 4), rand(2, 3, 16)
    train = lambda s: gdr.causal_conv1d(x.requires_grad_(True), w, initial_state=s)[0]  # noqa: E731
    step = lambda s: gdr.causal_conv1d_update(x[:, 0].detach(), s, w)  # noqa: E731
    return train, step, state


def scan():
    x, dt, A, b, c = rand(2, 9, 2, 64), rand(2, 9, 2), rand(2), rand(2, 9, 1, 64), rand(2, 9, 1, 64)
    state = rand(2, 2, 64, 64, dtype=torch.float32)
    train = lambda s: gdr.chunk_selective_scan(x.requires_grad_(True), dt, A, b, c,  # noqa: E731
                                               initial_state=s)[0]
    one = lambda v: v[:, :1].detach()  # noqa: E731
    step = lambda s: gdr.fused_recurrent_selective_scan(  # noqa: E731
        one(x), one(dt), A, one(b), one(c), initial_state=s, inplace_final_state=True)
    return train, step, state


def delta_rule():
    q, k, v, g, beta = (rand(1, 70, 1, 128), rand(1, 70, 1, 128) / 12, rand(1, 70, 1, 128),
                        -rand(1, 70, 1).abs(), rand(1, 70, 1).sigmoid())
    state = rand(1, 1, 128, 128, dtype=torch.float32)
    train = lambda s: gdr.chunk_gated_delta_rule(q.requires_grad_(True), k, v, g, beta,  # noqa: E731
                                                 initial_state=s)[0]
    one = lambda t: t[:, :1].detach()  # noqa: E731
    step = lambda s: gdr.fused_recurrent_gated_delta_rule(  # noqa: E731
        one(q), one(k), one(v), one(g), one(beta), initial_state=s, inplace_final_state=True)
    return train, step, state


@pytest.mark.parametrize("make", [conv, scan, delta_rule])
def test_a_graph_that_saved_the_state_notices_the_step(make):
    train, step, state = make()
    train(state).sum().backward()                   # as long as it is untouched, it runs
    y = train(state)
    before = state._version
    step(state)
    assert state._version > before
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    y = train(state.clone())                        # a graph with a state of its own does not mind
    step(state)
    y.sum().backward()


@pytest.mark.parametrize("make", [conv, scan])
def test_states_that_require_grad(make):
    _, step, state = make()
    state.requires_grad_(True)
    before = state.detach().clone()
    with pytest.raises(gdr.GdrError) as e:
        step(state)
    assert e.value.name == "GDR_ERR_ARG" and torch.equal(state.detach(), before)
    with torch.no_grad():
        step(state)
    assert not torch.equal(state.detach(), before)


@pytest.mark.parametrize("make", [conv, scan])
def test_inference_mode(make):
    _, step, state = make()
    want = state.clone()
    step(want)
    with torch.inference_mode():
        s = state.clone()
        step(s)
    assert s.is_inference() and torch.equal(s, want)
