"""The scan's gradient on rows that its asynchronous copies take, against the double-precision
reference: lengths of a multiple of 16 elements, channel-last 48 channels. (The sizes of
``test_gpu_scan_bwd.py`` are mostly odd ones, which plain loads fetch.)"""
import numpy as np
import pytest
import torch

from tests.bwd_helpers import case, gpu, host
from tests.test_gpu_scan_bwd import compare, reference, run, ssm

pytestmark = pytest.mark.gpu

both = pytest.mark.parametrize("dtype", ["f32", "bf16"])
layouts = pytest.mark.parametrize("cl", [False, True])


@both
@layouts
@pytest.mark.parametrize("L", [16, 80, 160])
@pytest.mark.parametrize("kw,opt", [
    (dict(conv=4), {}),
    (dict(conv=3, z=False), dict(reverse=True)),
    (dict(conv=2, skip=False, bias=False), {}),
    (dict(conv=1), {}),
    (dict(conv=4), dict(reverse=True)),
    (dict(conv=4, h0=True, hist=True, dfinal=True), {}),
    (dict(h0=True, dfinal=True), {}),
    (dict(dfinal=True), dict(reverse=True)),
    (dict(heads=4, conv=4), {}),
    (dict(heads=3, h0=True, dfinal=True), {}),
    (dict(heads=1), dict(reverse=True)),
])
def test_options(dtype, cl, L, kw, opt):
    run(case(31, dtype, 2, 48, L, 16, **kw), dtype, cl, **opt)


@both
@layouts
@pytest.mark.parametrize("B,D,N", [(1, 64, 1), (2, 48, 4), (1, 160, 8), (1, 80, 24), (2, 48, 32), (1, 64, 64), (1, 48, 128)])
def test_states(dtype, cl, B, D, N):
    run(case(32, dtype, B, D, 80, N, conv=4), dtype, cl)


@both
@layouts
@pytest.mark.parametrize("N,heads", [(4, 2), (8, 3), (16, 6), (32, 2), (64, 8), (128, 4)])
@pytest.mark.parametrize("segments", [1, 3])
def test_heads_states(dtype, cl, N, heads, segments):
    run(case(33, dtype, 2, 48, 80, N, heads=heads, conv=4), dtype, cl, num_segments=segments)


@both
@layouts
@pytest.mark.parametrize("segments", [0, 1, 3])
@pytest.mark.parametrize("L,starts", [(80, [0, 80]), (160, [0, 1, 17, 64, 64, 130, 160]), (160, [0, 16, 32, 33, 35, 36, 160])])
def test_packed(dtype, cl, segments, L, starts):
    run(case(34, dtype, 1, 48, L, 16, conv=4), dtype, cl, starts=starts, num_segments=segments)


@layouts
@pytest.mark.parametrize("N", [3, 8, 64, 128])
def test_packed_states(cl, N):
    run(case(35, "bf16", 1, 48, 96, N, conv=3), "bf16", cl, starts=[0, 5, 6, 24, 45, 96], num_segments=2)


@both
@layouts
@pytest.mark.parametrize("segments", [2, 5, 100])
@pytest.mark.parametrize("kw,opt", [
    (dict(conv=4, h0=True, hist=True, dfinal=True), {}), (dict(conv=4), dict(reverse=True)), (dict(heads=4), {})])
def test_segments(dtype, cl, segments, kw, opt):
    run(case(36, dtype, 2, 48, 160, 16, **kw), dtype, cl, num_segments=segments, **opt)


@layouts
@pytest.mark.parametrize("width", [2, 3, 4])
def test_history(cl, width):
    run(case(37, "bf16", 2, 48, 80, 16, conv=width, h0=True, hist=True, dfinal=True), "bf16", cl)


@both
@layouts
@pytest.mark.parametrize("reverse", [False, True])
def test_a_row_of_several_chunks(dtype, cl, reverse):
    """2080 steps: past a chunk of the conv's gradient along rows (2048), and past the steps after
    which the sweep's sums join the long ones."""
    run(case(38, dtype, 1, 48, 2080, 16, conv=4), dtype, cl, reverse=reverse, num_segments=1)


@both
@layouts
@pytest.mark.parametrize("B,D,L,N", [(1, 640, 96, 16), (2, 1040, 32, 8), (1, 416, 64, 64)])
def test_many_channels(dtype, cl, B, D, L, N):
    """More channels than a CTA holds many times over: their sums meet outside it."""
    run(case(39, dtype, B, D, L, N, conv=4), dtype, cl)


# ------------------------------------------------------------- 8-bit activations --

def from_8_bits(c, dtype, cl, reverse=False, starts=None, **kw):
    """The gradients from 8-bit u, delta and z are those of the values read back."""
    m = ssm()
    t = lambda k: gpu(c[k], dtype, cl)  # noqa: E731
    f = lambda k: gpu(c[k], "f32")  # noqa: E731
    kept = {k: m.ssm_checkpoint_pack(t(k), channel_last=cl) for k in ("u", "delta", "z") if c[k] is not None}
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    g = m.ssm_selective_scan_bwd(
        t("dout"), kept["u"], kept["delta"], f("A"), t("B"), t("C"), f("D"), kept.get("z"), f("delta_bias"), True,
        reverse, f("conv_w"), f("conv_b"), dfinal_state=f("dfinal"), initial_state=f("h0"),
        conv_history=gpu(c["hist"], dtype), seq_starts=st, channel_last=cl, **kw)
    back = dict(c, **{k: host(m.ssm_checkpoint_unpack(v, torch.float32, channel_last=cl), cl) for k, v in kept.items()})
    compare(g, reference(back, reverse=reverse, starts=starts), dtype, cl)


@both
@layouts
@pytest.mark.parametrize("N", [1, 4, 16, 32, 128])
@pytest.mark.parametrize("L,D,reverse", [(64, 48, False), (192, 48, False), (128, 32, True), (75, 40, False), (61, 33, True)])
def test_from_8_bits(dtype, cl, N, L, D, reverse):
    from_8_bits(case(41, dtype, 1, D, L, N, conv=4), dtype, cl, reverse)


@both
@layouts
@pytest.mark.parametrize("N", [4, 16, 64])
@pytest.mark.parametrize("kw,opt", [
    (dict(conv=4, h0=True, hist=True, dfinal=True), dict(num_segments=3)),
    (dict(conv=2), dict(num_segments=4, reverse=True)),
    (dict(conv=4), dict(num_segments=2, starts=[0, 1, 40, 64, 64, 100, 144])),
    (dict(conv=4, z=False), dict(starts=[0, 33, 144])),
    (dict(heads=4, conv=4), dict(num_segments=1)),
    (dict(heads=2, z=False), dict(num_segments=3)),
])
def test_from_8_bits_options(dtype, cl, N, kw, opt):
    from_8_bits(case(42, dtype, 1, 48, 144, N, **kw), dtype, cl, **opt)


def test_from_8_bits_strided():
    """Channel-last codes as columns of a wider tensor, at bases that no 16-byte copy takes and at others."""
    m = ssm()
    c = case(43, "bf16", 1, 48, 80, 16, conv=4)
    t = lambda k: gpu(c[k], "bf16", True)  # noqa: E731
    f = lambda k: gpu(c[k], "f32")  # noqa: E731
    kept = {k: m.ssm_checkpoint_pack(t(k), channel_last=True) for k in ("u", "delta", "z")}
    want = m.ssm_selective_scan_bwd(t("dout"), kept["u"], kept["delta"], f("A"), t("B"), t("C"), f("D"), kept["z"],
                                    f("delta_bias"), True, False, f("conv_w"), f("conv_b"), channel_last=True)
    for lead, width in ((0, 160), (5, 151)):
        views = {}
        for k, p in kept.items():
            wide = torch.full((1, 80, width), 99, dtype=torch.int8, device="cuda")
            wide[..., lead:lead + 48] = p.codes
            views[k] = m.Packed8(wide[..., lead:lead + 48], p.scales)
        g = m.ssm_selective_scan_bwd(t("dout"), views["u"], views["delta"], f("A"), t("B"), t("C"), f("D"), views["z"],
                                     f("delta_bias"), True, False, f("conv_w"), f("conv_b"), channel_last=True)
        assert all(torch.equal(a, b) for a, b in zip(g, want) if a is not None)
        assert np.isfinite(host(g.du)).all()
