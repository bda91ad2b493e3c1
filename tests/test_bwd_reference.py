"""The backward pass's double-precision reference against central differences of the forward
oracle (CPU). The loss is sum(out * dout) + sum(final_state * dfinal). For a smooth loss the
difference quotient with step e is off by e^2 / 6 times a third derivative, plus about
2^-52 |loss| / e of rounding: with e = 1e-4 and values of order one both are below 1e-6 of the
gradients' scale (third derivatives of these losses stay within 30 times it)."""
import numpy as np
import pytest

import oracle
from tests import bwd_reference as ref

EPS, TOL = 1e-4, 2e-6


def _case(seed, B, D, L, N, heads=0, conv=0, z=True, hist=False, h0=False, bias=True, skip=True):
    r = np.random.default_rng(seed)
    n = lambda *s: r.standard_normal(s)  # noqa: E731
    c = {"u": n(B, D, L), "delta": 0.5 * n(B, D, L), "B": n(B, N, L), "C": n(B, N, L),
         "A": -r.uniform(0.5, 2.0, heads) if heads else -r.uniform(0.5, 2.0, (D, N))}
    c["D"] = n(D) if skip else None
    c["z"] = n(B, D, L) if z else None
    c["delta_bias"] = n(D) if bias else None
    c["conv_w"] = 0.5 * n(D, conv) if conv else None
    c["conv_b"] = n(D) if conv else None
    c["hist"] = n(B, D, conv - 1) if hist else None
    c["h0"] = n(B, D, N) if h0 else None
    return c, n(B, D, L), n(B, D, N)


def _loss(c, dout, dfinal, softplus, reverse, starts=None, size=None):
    """The forward oracle's loss; packed sequences one by one. size[0] gets sum|terms|."""
    size = [0.0] if size is None else size
    def one(c, dout):
        y, h = oracle.selective_scan(c["u"], c["delta"], c["A"], c["B"], c["C"], c["D"], c["z"],
                                     c["delta_bias"], softplus, reverse, c["conv_w"], c["conv_b"],
                                     return_final_state=True, h0=c["h0"],
                                     conv_hist=c["hist"])
        hd = 0.0 * h if dfinal is None else h * dfinal
        size[0] += float(np.sum(np.abs(y * dout)) + np.sum(np.abs(hd)))
        return float(np.sum(y * dout)) + float(np.sum(hd))
    if starts is None:
        return one(c, dout)
    total = 0.0
    for i, j in zip(starts[:-1], starts[1:]):
        if j > i:
            part = {k: v[:, :, i:j] if k in ("u", "delta", "B", "C", "z") and v is not None else v
                    for k, v in c.items()}
            total += one(part, dout[:, :, i:j])
    return total


NAMES = {"u": "du", "delta": "ddelta", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "z": "dz",
         "delta_bias": "ddelta_bias", "conv_w": "dconv_weight", "conv_b": "dconv_bias",
         "h0": "dinitial_state", "hist": "dconv_history"}


@pytest.mark.parametrize("kw,softplus,reverse,starts", [
    (dict(B=2, D=3, L=5, N=2), True, False, None),
    (dict(B=1, D=2, L=6, N=3, conv=4), True, False, None),
    (dict(B=1, D=2, L=6, N=3, conv=3, z=False), False, True, None),
    (dict(B=2, D=4, L=4, N=2, heads=2, conv=2, skip=False), True, False, None),
    (dict(B=1, D=2, L=3, N=2, conv=4, hist=True, h0=True), True, False, None),
    (dict(B=1, D=2, L=1, N=1, bias=False), True, False, None),
    (dict(B=1, D=2, L=7, N=2, conv=4), True, False, [0, 1, 1, 4, 7]),
])
def test_against_differences(kw, softplus, reverse, starts):
    c, dout, dfinal = _case(3, **kw)
    dfinal = None if starts is not None else dfinal
    g = ref.scan_grads(dout, c["u"], c["delta"], c["A"], c["B"], c["C"], c["D"], c["z"],
                       c["delta_bias"], softplus, reverse, c["conv_w"], c["conv_b"], dfinal,
                       c["h0"], c["hist"], starts)
    size = [0.0]
    _loss(c, dout, dfinal, softplus, reverse, starts, size)
    rounding = 2 * (2 * kw["L"] + 8) * 2.0 ** -53 * size[0] / (2 * EPS)
    assert set(g) == {NAMES[k] for k, v in c.items() if v is not None}
    for k, v in c.items():
        if v is None:
            continue
        num = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            keep = v[i]
            v[i] = keep + EPS
            up = _loss(c, dout, dfinal, softplus, reverse, starts)
            v[i] = keep - EPS
            num[i] = (up - _loss(c, dout, dfinal, softplus, reverse, starts)) / (2 * EPS)
            v[i] = keep
        scale = max(1.0, float(np.max(np.abs(num))))
        assert np.max(np.abs(g[NAMES[k]] - num)) <= TOL * scale + rounding, NAMES[k]


@pytest.mark.parametrize("width,silu", [(1, True), (3, False), (4, True)])
def test_conv_against_differences(width, silu):
    r = np.random.default_rng(5)
    x, w, b, dout = (r.standard_normal(s) for s in ((2, 3, 6), (3, width), (3,), (2, 3, 6)))
    dx, dw, db, _ = ref.conv_grads(dout, x, w, b, silu)
    for v, g in ((x, dx), (w, dw), (b, db)):
        for i in np.ndindex(v.shape):
            keep, vals = v[i], []
            for e in (EPS, -EPS):
                v[i] = keep + e
                vals.append(float(np.sum(oracle.causal_conv1d(x, w, b, silu) * dout)))
            v[i] = keep
            num = (vals[0] - vals[1]) / (2 * EPS)
            assert abs(num - g[i]) <= TOL * max(1.0, abs(num))


def test_a_planted_mistake_is_caught():
    """A reference that forgets the decay in the adjoint differs from the oracle's gradient."""
    c, dout, dfinal = _case(7, B=1, D=2, L=4, N=2)
    g = ref.scan_grads(dout, c["u"], c["delta"], c["A"], c["B"], c["C"], c["D"], c["z"], c["delta_bias"])
    wrong = ref.scan_grads(dout, c["u"], c["delta"], np.zeros_like(c["A"]), c["B"], c["C"], c["D"],
                           c["z"], c["delta_bias"])
    assert np.max(np.abs(g["du"] - wrong["du"])) > 1e-3
