"""Pins of the gated block's activation: closed forms, and the slopes against differences."""
import math

import numpy as np
import pytest

import oracle

ACTS = ["silu", "gelu", "gelu_tanh"]


@pytest.mark.parametrize("act", ACTS)
def test_closed_forms(act):
    g = np.array([-30.0, -3.0, -0.5, 0.0, 0.25, 2.0, 30.0])
    want = {"silu": lambda v: v / (1 + math.exp(-v)), "gelu": lambda v: 0.5 * v * math.erfc(-v / math.sqrt(2)),
            "gelu_tanh": lambda v: 0.5 * v * (1 + math.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))}[act]
    got = oracle.gated_forward(g, np.full_like(g, 3.0), act)
    assert np.allclose(got, [3 * want(v) for v in g], rtol=1e-13, atol=1e-15)
    assert np.all(np.isfinite(oracle.gate(np.array([-800.0, 800.0]), act)[1]))


@pytest.mark.parametrize("act", ACTS)
def test_gradients_against_differences(act):
    rng = np.random.default_rng(1)
    g, v, dh = rng.normal(size=(3, 200)) * 2
    dg, dv = oracle.gated_backward(dh, g, v, act)
    e = 1e-5
    ng = dh * (oracle.gated_forward(g + e, v, act) - oracle.gated_forward(g - e, v, act)) / (2 * e)
    nv = dh * (oracle.gated_forward(g, v + e, act) - oracle.gated_forward(g, v - e, act)) / (2 * e)
    assert np.allclose(dg, ng, rtol=1e-7, atol=1e-8) and np.allclose(dv, nv, rtol=1e-7, atol=1e-8)


def test_slopes_stay_below_the_bound_of_the_gpu_tests():
    g = np.linspace(-12, 12, 200001)
    for act in ACTS:
        assert np.abs(oracle.gate(g, act)[1]).max() < 1.13
