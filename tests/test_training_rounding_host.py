"""How 8-bit first moments are rounded, on the host: what a state says about it,
what the interface refuses, and, with a CPU model of the recurrence, that
rounding at random follows the gradient where rounding to nearest does not."""
import ctypes
import os
import warnings

import pytest

torch = pytest.importorskip("torch")

import adamw8_model as model  # noqa: E402


@pytest.fixture(scope="module")
def ga():
    import gradient_aggregation_amd as ga
    if not os.path.exists(ga.LIB_PATH):
        from gradient_aggregation_amd import build
        build.build()
    return ga


def test_states_say_how_they_are_rounded(ga):
    one = torch.zeros(1)
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        assert ga.AdamWState(one, one, one, one, m_rounding="random").m_rounding == "random"
        assert ga.AdamWState(one, one, one, one, m_rounding="nearest").m_rounding == "nearest"
        ga.AdamWState(one, one)                                    # 32 bits: nothing to choose
    with pytest.warns(UserWarning, match="nearest"):
        assert ga.AdamWState(one, one, one, one).m_rounding == "nearest"
    with pytest.raises(ValueError):
        ga.AdamWState(one, one, one, one, m_rounding="up")


def test_what_was_made_before_there_was_a_choice(ga):
    """Parameters in their earlier order, and states without the attribute (a
    pickled one, say)."""
    p = ga.AdamWParams(1e-3, 0.9, 0.999, 1e-8, 0.1, 5)
    assert (p.t, p.m_rounding) == (5, 0) and p.weight_decay == pytest.approx(0.1)
    assert ga.AdamWParams(lr=1.0, t=3).t == 3 and ga.AdamWParams(t=3, m_rounding=1).m_rounding == 1
    assert ga.AdamWState.__new__(ga.AdamWState).m_rounding == "nearest"


def test_step_refuses_an_unknown_rounding(ga):
    block = (ctypes.c_int32 * 256)()
    handle, step = ctypes.addressof(block), ga.lib().ga_adamw_step
    state = ga.AdamWStatePtrs(16, 16, 16, 16)
    p = lambda rounding: ga.AdamWParams(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, t=1, m_rounding=rounding)
    block[3] = 8                                                    # the handle's state_bits
    for bad in (-1, 2, 7):
        assert step(handle, 16, p(bad), 16, state, None, None, 0, None) == ga.GA_ERR_INVALID
        assert b"m_rounding" in ga.lib().ga_last_error()
    for good in (0, 1):                                             # goes on to the alignment of w
        assert step(handle, 16, p(good), 8, state, None, None, 0, None) == ga.GA_ERR_ALIGN
    block[3] = 32                                                   # not read with binary32 states
    assert step(handle, 16, p(7), 8, ga.AdamWStatePtrs(16, 16), None, None, 0, None) == ga.GA_ERR_ALIGN


@pytest.mark.parametrize("factor,noise,beta1,beta2", model.TURNS)
def test_model_of_turned_gradients(factor, noise, beta1, beta2):
    """Weights that share blocks with steady ones, and whose gradient turns,
    falls or goes: the bound holds rounding at random and not to nearest."""
    turn = model.Turn(2048, factor, noise)
    args = (turn, 2048, turn.steps, beta1, beta2)
    want = model.exact(*args, watch=(turn.BEFORE,))
    bound = turn.bound(beta1, want)
    assert abs(turn.moved(model.run(*args, watch=(turn.BEFORE,))) - turn.moved(want)) <= bound
    assert abs(turn.moved(model.run(*args, m_how="nearest", watch=(turn.BEFORE,))) - turn.moved(want)) > bound


@pytest.mark.parametrize("factor", [0.7, 0.5])
def test_model_of_second_moments(factor):
    """Second moments that move by far less than a code's step per step, while
    the largest of their block stays: rounded at random they follow, to nearest
    and down they do not."""
    turn = model.Turn(2048, factor)
    args = (turn, 2048, turn.steps, 0.9, 0.999)
    want = model.exact(*args)[-1]
    off = {how: abs(turn.second(model.run(*args, v_how=how)[-1], want) - 1) for how in ("random", "nearest", "down")}
    assert off["random"] <= turn.second_bound() < min(off["nearest"], off["down"]), off
