"""What is not finite in a conv's input reaches as far as the conv does, no further: gradients
beyond its taps keep the bits that they have without it."""
import numpy as np
import pytest
import torch

from tests.bwd_helpers import case, gpu, host

pytestmark = pytest.mark.gpu


def ssm():
    import mamba_selective_scan_sm_b200 as m
    return m


def far(L, at, reach):
    t = np.arange(L)
    return np.abs(t - at) > reach


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("L,at", [(64, 30), (64, 0), (61, 45), (2200, 2050)])
@pytest.mark.parametrize("width", [1, 2, 3, 4])
@pytest.mark.parametrize("bad", [np.nan, np.inf])
def test_conv_gradient(dtype, L, at, width, bad):
    m = ssm()
    c = case(1, dtype, 2, 3, L, 1, conv=width)
    f = lambda k: gpu(c[k], "f32")  # noqa: E731
    args = lambda x, dy: (gpu(dy, dtype), gpu(x, dtype), f("conv_w"), f("conv_b"))  # noqa: E731
    for silu in (True, False):
        want = host(m.ssm_causal_conv1d_bwd(*args(c["u"], c["dout"]), silu).dx)
        x = c["u"].copy()
        x[:, :, at] = bad
        got = host(m.ssm_causal_conv1d_bwd(*args(x, c["dout"]), silu).dx)
        keep = far(L, at, width - 1 if silu else -1)
        assert np.array_equal(got[..., keep], want[..., keep])
        if silu:
            assert not np.isfinite(got[..., at]).any()
        dy = c["dout"].copy()
        dy[:, :, at] = bad
        got = host(m.ssm_causal_conv1d_bwd(*args(c["u"], dy), silu).dx)
        reach = (np.arange(L) > at) | (np.arange(L) <= at - width)
        assert np.array_equal(got[..., reach], want[..., reach]) and not np.isfinite(got[..., at]).any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("L,at", [(64, 30), (45, 15), (200, 130)])
@pytest.mark.parametrize("width", [1, 2, 3, 4])
def test_scan_gradient(dtype, cl, reverse, L, at, width):
    """NaN at one position of x (in scan order `at`): the conv's output is NaN from there to
    width - 1 steps on. dB holds it there and nowhere else, du width - 1 steps before too."""
    m = ssm()
    c = case(2, dtype, 1, 32, L, 16, conv=width)

    def call(u):
        t = lambda v: gpu(v, dtype, cl)  # noqa: E731
        f = lambda k: gpu(c[k], "f32")  # noqa: E731
        return m.ssm_selective_scan_bwd(t(c["dout"]), t(u), t(c["delta"]), f("A"), t(c["B"]), t(c["C"]), f("D"),
                                        t(c["z"]), f("delta_bias"), True, reverse, f("conv_w"), f("conv_b"),
                                        channel_last=cl)
    scan = lambda a: a[..., ::-1] if reverse else a  # noqa: E731
    want = call(c["u"])
    u = c["u"].copy()
    scan(u)[:, :, at] = np.nan
    got = call(u)
    t = np.arange(L)
    for k, hit in (("dB", (t >= at) & (t < at + width)), ("du", np.abs(t - at) < width)):
        a, o = scan(host(getattr(got, k), cl)), scan(host(getattr(want, k), cl))
        assert np.isnan(a[..., hit]).all(), k
        assert np.array_equal(a[..., ~hit], o[..., ~hit]), k


@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("width", [2, 3])
def test_packed_sequences(cl, width):
    """The same within packed sequences: not past a sequence's end either."""
    m = ssm()
    L, starts, at = 120, [0, 30, 33, 80, 120], 40
    c = case(3, "f32", 1, 32, L, 16, conv=width)
    st = torch.tensor(starts, dtype=torch.int32, device="cuda")

    def call(u):
        t = lambda v: gpu(v, "f32", cl)  # noqa: E731
        f = lambda k: gpu(c[k], "f32")  # noqa: E731
        return m.ssm_selective_scan_bwd(t(c["dout"]), t(u), t(c["delta"]), f("A"), t(c["B"]), t(c["C"]), f("D"),
                                        t(c["z"]), f("delta_bias"), conv_weight=f("conv_w"), conv_bias=f("conv_b"),
                                        channel_last=cl, seq_starts=st)
    want = call(c["u"])
    for at in (40, 79, 31):
        u = c["u"].copy()
        u[:, :, at] = np.nan
        got = call(u)
        end = min(s for s in starts if s > at)
        t = np.arange(L)
        hit = (t >= at) & (t < min(at + width, end))
        a, o = host(got.dB, cl), host(want.dB, cl)
        assert np.isnan(a[..., hit]).all() and np.array_equal(a[..., ~hit], o[..., ~hit])
