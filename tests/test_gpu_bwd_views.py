"""The scan's gradient into free columns of the tensors that hold its inputs."""
import pytest
import torch

from tests.bwd_helpers import case, gpu
from tests.test_gpu_scan_bwd import call, compare, reference, ssm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,L,N,pad", [(48, 37, 16, 0), (32, 64, 8, 0), (35, 20, 13, 3), (128, 33, 64, 0)])
def test_gradients_beside_their_inputs(dtype, D, L, N, pad):
    """u, z, du and dz as columns of one tensor (and some that belong to none), B, C, dB and dC as
    columns of another: the inputs and the columns of none keep their bits."""
    m, B = ssm(), 2
    c = case(40, dtype, B, D, L, N, conv=4)
    t = lambda k: gpu(c[k], dtype, True)  # noqa: E731
    f = lambda k: gpu(c[k], "f32")  # noqa: E731
    el = torch.float32 if dtype == "f32" else torch.bfloat16
    wide = torch.full((B, L, 4 * D + pad), 7.0, dtype=el, device="cuda")
    bc = torch.full((B, L, 4 * N + pad), 7.0, dtype=el, device="cuda")
    u, du, z, dz = (wide[..., i * D:(i + 1) * D] for i in range(4))
    Bm, dB, Cm, dC = (bc[..., i * N:(i + 1) * N] for i in range(4))
    for v, k in ((u, "u"), (z, "z"), (Bm, "B"), (Cm, "C")):
        v.copy_(t(k))
    g = m.ssm_selective_scan_bwd(t("dout"), u, t("delta"), f("A"), Bm, Cm, f("D"), z, f("delta_bias"), True, False,
                                 f("conv_w"), f("conv_b"), channel_last=True, du=du, dz=dz, dB=dB, dC=dC)
    compare(g, reference(c), dtype, True)
    plain = call(c, dtype, True)
    assert torch.equal(du, plain.du) and torch.equal(dB, plain.dB)
    for v, k in ((u, "u"), (z, "z"), (Bm, "B"), (Cm, "C")):
        assert torch.equal(v, t(k)), k
    assert torch.all(wide[..., 4 * D:] == 7.0) and torch.all(bc[..., 4 * N:] == 7.0)
