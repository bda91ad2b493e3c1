"""Without the softplus delta may be negative: states then grow, and the slots that fill a lane up
behind the last state must not."""
import numpy as np
import pytest

from tests.bwd_helpers import case
from tests.test_gpu_scan_bwd import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("segments", [1, 2])
@pytest.mark.parametrize("N", [1, 3, 5, 7, 13, 20, 50, 100, 16])
def test_negative_delta(N, segments, cl):
    """delta within -0.05 and 0.1 on 33 channels (a CTA's last ones stand empty), A from -0.5 to -8: over 40
    steps a state grows to e^16 at most, and the tolerances are relative to what it makes of the sums."""
    c = case(70, "f32", 1, 33, 40, N, conv=4, bias=False, h0=True, dfinal=True)
    r = np.random.default_rng(71)
    c["delta"] = r.uniform(-0.05, 0.1, c["delta"].shape).astype(np.float32)
    c["A"] = -r.uniform(0.5, 8.0, c["A"].shape).astype(np.float32)
    run(c, "f32", cl, softplus=False, num_segments=segments)


@pytest.mark.parametrize("N", [3, 13, 100])
def test_a_large_negative_delta_at_one_step(N):
    """One step of delta = -1: the states grow e^8 times at most, once."""
    c = case(72, "f32", 1, 33, 24, N, bias=False)
    c["delta"] = np.abs(c["delta"]) * np.float32(0.1)
    c["delta"][:, :, 10] = -1.0
    c["A"] = -np.random.default_rng(73).uniform(0.5, 8.0, c["A"].shape).astype(np.float32)
    run(c, "f32", softplus=False)
