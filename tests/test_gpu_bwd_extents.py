"""The gradients at the ends of their sizes: very many channels, the most batch rows, and calls of
every operator captured into a graph and replayed on new inputs."""
import numpy as np
import pytest
import torch

from tests.bwd_helpers import case, gpu
from tests.test_gpu_scan_bwd import ssm

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("N", [3, 16])
def test_very_many_channels(N, cl):
    """dB and dC as sums over 2^20 channels of terms of one sign. Every addition is off by 2^-25 at
    most on average: 32 to 128 channels of a CTA, 64 CTAs, then 512 such sums: 704 * 2^-25 = 2.1e-5."""
    D, L, d = (1 << 20) + 5, 2, 0.1
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    act, bc = ((1, L, D), (1, L, N)) if cl else ((1, D, L), (1, N, L))
    A = torch.full((D, N), -1.5, device="cuda")
    g = ssm().ssm_selective_scan_bwd(one(*act), one(*act), d * one(*act), A, one(*bc), one(*bc), delta_softplus=False,
                                     channel_last=cl)
    d = float(np.float32(d))
    a = np.exp(d * -1.5)
    h, lam = np.array([d, d * (1 + a)]), np.array([1 + a, 1.0])
    for v, want in ((g.dC, D * h), (g.dB, D * d * lam)):
        v = (v if cl else v.transpose(1, 2))[0].double().cpu().numpy()
        assert np.all(np.abs(v / want[:, None] - 1) <= 2.1e-5), v / want[:, None] - 1
    assert torch.all(g.dA == g.dA[0]) and torch.all(g.du == (g.du[:, :, :1] if cl else g.du[:, :1]))


@pytest.mark.parametrize("cl", [False, True])
def test_the_most_batch_rows(cl):
    """65535 rows alike: each row's gradients are those of one row, dA and dD 65535 times them (to
    the rounding of their sum)."""
    m, B, D, L, N = ssm(), 65535, 3, 5, 2
    c = case(60, "f32", 1, D, L, N, conv=3)
    t = lambda k, n: gpu(c[k], "f32", cl).expand(n, -1, -1).contiguous()  # noqa: E731
    f = lambda k: gpu(c[k], "f32")  # noqa: E731

    def call(n):
        return m.ssm_selective_scan_bwd(t("dout", n), t("u", n), t("delta", n), f("A"), t("B", n), t("C", n), f("D"),
                                        t("z", n), f("delta_bias"), True, False, f("conv_w"), f("conv_b"), channel_last=cl)
    one, all_ = call(1), call(B)
    for k in ("du", "ddelta", "dz", "dB", "dC"):
        v = getattr(all_, k)
        assert torch.equal(v, getattr(one, k).expand_as(v)), k
    for k in ("dA", "dD", "ddelta_bias", "dconv_weight", "dconv_bias"):
        v, o = getattr(all_, k).double(), getattr(one, k).double() * B
        assert torch.all((v - o).abs() <= 1e-6 * o.abs() + 1e-30), k
    with pytest.raises(m.SSMError) as e:
        call(B + 1)
    assert e.value.name == "SSM_ERR_UNSUPPORTED"


def test_more_decode_rows_than_a_grid_axis_holds():
    """A batch whose CTAs pass 65535 along an axis: the rows at both ends and at the seam are those
    of calls on them alone."""
    m, B, n = ssm(), 65535 * 32 + 70, 4
    g = torch.Generator(device="cuda").manual_seed(2)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    state, x, dt, Bt, Ct, z = r(B, 1, n), r(B, 1), r(B, 1), r(B, n), r(B, n), r(B, 1)
    A, D, w = -r(1, n).abs(), r(1), r(1, 4)
    conv = r(B, 1, 4)

    def step(lo, hi):
        codes, scales = torch.zeros(hi - lo, 1, n, dtype=torch.int8, device="cuda"), torch.zeros(hi - lo, 1, device="cuda")
        cs = conv[lo:hi].clone()
        cut = lambda v: v[lo:hi].contiguous()  # noqa: E731
        m.ssm_state_cache_write(cut(state), codes, scales)
        y = m.ssm_selective_state_update_cached(codes, scales, cs, cut(x), cut(dt), A, cut(Bt), cut(Ct), D, cut(z), None,
                                                True, w, None)
        return codes, scales, cs, y, m.ssm_state_cache_read(codes, scales)
    whole, seam = step(0, B), 65535 * 32
    for lo, hi in ((0, 100), (seam - 50, seam + 50), (B - 60, B)):
        assert all(torch.equal(a[lo:hi], b) for a, b in zip(whole, step(lo, hi)))


def test_captured_calls():
    """Pack, unpack, the conv's gradient, cache write, step and read in one graph, replayed on new
    inputs: what plain calls give."""
    m, (B, D, L, N) = ssm(), (2, 40, 100, 16)
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    bits = lambda: torch.randint(-2 ** 31, 2 ** 31, (B, D), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)  # noqa: E731
    new = lambda: [r(B, D, L), r(B, D, L), r(B, D, N), r(B, D), r(B, D), r(B, N), r(B, N), r(B, D, 4), bits()]  # noqa: E731
    A, Dv, w, wb = -r(D, N).abs(), r(D), r(D, 4), r(D)

    def run(x, dy, state, xt, dt, Bt, Ct, conv, rand, codes, scales):
        kept = m.ssm_checkpoint_pack(x)
        back = m.ssm_checkpoint_unpack(kept, torch.float32)
        grads = m.ssm_causal_conv1d_bwd(dy, back, w, wb)
        m.ssm_state_cache_write(state, codes, scales, rand=rand)
        cs = conv.clone()
        y = m.ssm_selective_state_update_cached(codes, scales, cs, xt, dt, A, Bt, Ct, Dv, None, None, True, w, wb, rand=rand)
        return [*kept, back, *grads, cs, y, m.ssm_state_cache_read(codes, scales)]
    cache = lambda: (torch.zeros(B, D, N, dtype=torch.int8, device="cuda"), torch.zeros(B, D, device="cuda"))  # noqa: E731
    ins, held = new(), cache()
    run(*ins, *held)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(*ins, *held)
    for _ in range(3):
        for v, o in zip(ins, new()):
            v.copy_(o)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, run(*ins, *cache())))
