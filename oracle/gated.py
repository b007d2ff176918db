"""The gated feed-forward block's first half in float64: h = act(g) v, and its gradients at g and v."""
import math

import numpy as np

_erfc = np.vectorize(math.erfc, otypes=[float])


def gate(g, act):
    """(q, act') with act(g) = g q."""
    g = np.asarray(g, dtype=np.float64)
    if act == "gelu":
        phi = 0.5 * _erfc(-g / math.sqrt(2.0)) if g.size else g
        return phi, phi + g * np.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    v, dv = (g, np.ones_like(g)) if act == "silu" else (c * (g + 0.044715 * g ** 3), c * (1 + 3 * 0.044715 * g * g))
    e = np.exp(-np.abs(v))
    q, p = np.where(v >= 0, 1, e) / (1 + e), np.where(v >= 0, e, 1) / (1 + e)  # sigmoid(v), sigmoid(-v)
    return q, q + g * dv * q * p


def gated_forward(g, v, act):
    return g * gate(g, act)[0] * v


def gated_backward(dh, g, v, act):
    """(dg, dv)."""
    q, slope = gate(g, act)
    return dh * v * slope, dh * g * q
