"""The gradient of the standalone causal conv on the GPU against the reference."""
import numpy as np
import pytest
import torch

from tests import bwd_reference as ref
from tests.bwd_helpers import case, check, gpu, host

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,L", [(1, 1, 1), (2, 3, 2), (1, 5, 3), (2, 7, 9), (1, 4, 1023), (1, 3, 1024),
                                   (2, 2, 1030), (1, 2, 2500), (3, 33, 64)])
@pytest.mark.parametrize("width,silu,bias", [(4, True, True), (3, False, True), (2, True, False), (1, True, True)])
def test_conv_grads(dtype, B, D, L, width, silu, bias):
    import mamba_selective_scan_sm_b200 as m
    c = case(1, dtype, B, D, L, 1, conv=width)
    b = c["conv_b"] if bias else None
    g = m.ssm_causal_conv1d_bwd(gpu(c["dout"], dtype), gpu(c["u"], dtype), gpu(c["conv_w"], "f32"),
                                gpu(b, "f32"), silu)
    dx, dw, db, _ = ref.conv_grads(c["dout"], c["u"], c["conv_w"], b, silu)
    check("dx", host(g.dx), dx, dtype)
    check("dw", host(g.dw), dw, dtype)
    if bias:
        check("db", host(g.dbias), db, dtype)
    else:
        assert g.dbias is None


def test_conv_grads_misaligned_and_repeated():
    import mamba_selective_scan_sm_b200 as m
    c = case(2, "bf16", 2, 3, 200, 1, conv=4)
    buf = torch.zeros(2 * 3 * 200 + 3, dtype=torch.bfloat16, device="cuda")
    x = buf[3:].view(2, 3, 200)
    x.copy_(gpu(c["u"], "bf16"))
    args = (gpu(c["dout"], "bf16"), x, gpu(c["conv_w"], "f32"), gpu(c["conv_b"], "f32"))
    g, again = m.ssm_causal_conv1d_bwd(*args), m.ssm_causal_conv1d_bwd(*args)
    assert all(torch.equal(a, b) for a, b in zip(g, again))
    dx, dw, db, _ = ref.conv_grads(c["dout"], c["u"], c["conv_w"], c["conv_b"])
    for k, a, o in (("dx", g.dx, dx), ("dw", g.dw, dw), ("db", g.dbias, db)):
        check(k, host(a), o, "bf16")


@pytest.mark.parametrize("shape", [(0, 3, 4), (2, 0, 4), (2, 3, 0)])
def test_conv_grads_empty(shape):
    import mamba_selective_scan_sm_b200 as m
    x = torch.zeros(shape, device="cuda")
    g = m.ssm_causal_conv1d_bwd(x, x.clone(), torch.ones(shape[1], 4, device="cuda"),
                                torch.ones(shape[1], device="cuda"))
    assert g.dx.shape == x.shape and torch.all(g.dw == 0) and torch.all(g.dbias == 0)


def test_conv_grads_extremes():
    import mamba_selective_scan_sm_b200 as m
    c = case(3, "f32", 1, 4, 50, 1, conv=4)
    c["u"][0, 0] *= 100.0
    c["u"][0, 1] *= -100.0
    g = m.ssm_causal_conv1d_bwd(gpu(c["dout"], "f32"), gpu(c["u"], "f32"), gpu(c["conv_w"], "f32"))
    dx, dw, _, _ = ref.conv_grads(c["dout"], c["u"], c["conv_w"])
    check("dx", host(g.dx), dx, "f32")
    check("dw", host(g.dw), dw, "f32")
    assert np.all(np.isfinite(host(g.dx)))
