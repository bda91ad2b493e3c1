"""The gradient of the selective scan on the GPU against the double-precision reference."""
import numpy as np
import pytest
import torch

from tests import bwd_reference as ref
from tests.bwd_helpers import case, check, gpu, host

pytestmark = pytest.mark.gpu

LAST = ("du", "ddelta", "dz", "dB", "dC")


def ssm():
    import mamba_selective_scan_sm_b200 as m
    return m


def call(c, dtype, cl=False, softplus=True, reverse=False, starts=None, **kw):
    t = lambda k, sw=True: gpu(c[k], dtype, swap=cl and sw)  # noqa: E731
    f = lambda k: gpu(c[k], "f32")  # noqa: E731
    st = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    return ssm().ssm_selective_scan_bwd(
        t("dout"), t("u"), t("delta"), f("A"), t("B"), t("C"), f("D"), t("z"), f("delta_bias"),
        softplus, reverse, f("conv_w"), f("conv_b"), dfinal_state=f("dfinal"), initial_state=f("h0"),
        conv_history=t("hist", False), seq_starts=st, channel_last=cl, **kw)


def reference(c, softplus=True, reverse=False, starts=None):
    return ref.scan_grads(c["dout"], c["u"], c["delta"], c["A"], c["B"], c["C"], c["D"], c["z"],
                          c["delta_bias"], softplus, reverse, c["conv_w"], c["conv_b"], c["dfinal"],
                          c["h0"], c["hist"], starts)


def compare(g, want, dtype, cl=False):
    got = {k: v for k, v in g._asdict().items() if v is not None}
    assert set(got) == set(want)
    for k, o in want.items():
        check(k, host(got[k], swap=cl and k in LAST), o, dtype)


def run(c, dtype, cl=False, softplus=True, reverse=False, starts=None, **kw):
    compare(call(c, dtype, cl, softplus, reverse, starts, **kw),
            reference(c, softplus, reverse, starts), dtype, cl)


# every number of lanes per channel, odd sizes on each axis, one step to several tiles
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("B,D,L,N", [
    (1, 1, 1, 1), (2, 3, 2, 4), (1, 33, 31, 5), (2, 40, 64, 8), (1, 129, 17, 3), (2, 65, 33, 7),
    (2, 32, 64, 16), (1, 37, 100, 16), (1, 8, 257, 13), (1, 33, 40, 32), (1, 35, 33, 64),
    (2, 34, 19, 100), (1, 64, 24, 128),
])
def test_sizes(dtype, cl, B, D, L, N):
    run(case(1, dtype, B, D, L, N), dtype, cl)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("kw,opt", [
    (dict(conv=4), {}),
    (dict(conv=3, z=False), dict(reverse=True)),
    (dict(conv=2, skip=False, bias=False), {}),
    (dict(conv=1, hist=False), dict(softplus=True)),
    (dict(conv=4, h0=True, hist=True, dfinal=True), {}),
    (dict(h0=True, dfinal=True), {}),
    (dict(dfinal=True), dict(reverse=True)),
    (dict(z=False, skip=False, bias=False), {}),
    (dict(heads=4, conv=4), {}),
    (dict(heads=4, h0=True, dfinal=True), {}),
    (dict(heads=1), dict(reverse=True)),
])
def test_options(dtype, cl, kw, opt):
    run(case(2, dtype, 2, 40, 75, 16, **kw), dtype, cl, **opt)


@pytest.mark.parametrize("N,heads", [(4, 2), (8, 5), (32, 2), (64, 8), (128, 4)])
def test_heads_states(N, heads):
    run(case(3, "bf16", 2, 40, 50, N, heads=heads, conv=4), "bf16")


@pytest.mark.parametrize("cl", [False, True])
def test_delta_without_softplus(cl):
    c = case(4, "f32", 1, 20, 60, 16, bias=False)
    c["delta"] = np.abs(c["delta"]) * np.float32(0.1)
    run(c, "f32", cl, softplus=False)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("starts", [
    [0, 70], [0, 1, 2, 3, 70], [0, 0, 31, 32, 33, 64, 64, 70, 70], [0, 8, 16, 24, 40, 70],
])
@pytest.mark.parametrize("segments", [0, 1, 3])
def test_packed(dtype, cl, starts, segments):
    run(case(5, dtype, 1, 35, 70, 16, conv=4), dtype, cl, starts=starts, num_segments=segments)


@pytest.mark.parametrize("N", [3, 8, 64, 128])
def test_packed_states(N):
    run(case(6, "bf16", 1, 40, 45, N, conv=3), "bf16", starts=[0, 5, 6, 24, 45], num_segments=2)


@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("segments", [1, 2, 3, 5, 100])
@pytest.mark.parametrize("kw,opt", [
    (dict(conv=4, h0=True, hist=True, dfinal=True), {}),
    (dict(conv=2), dict(reverse=True)),
    (dict(heads=4), {}),
])
def test_segments(cl, segments, kw, opt):
    run(case(7, "f32", 2, 36, 161, 16, **kw), "f32", cl, num_segments=segments, **opt)


@pytest.mark.parametrize("N", [2, 6, 24, 50, 128])
def test_segments_states(N):
    run(case(8, "f32", 1, 33, 90, N, h0=True, dfinal=True), "f32", num_segments=3)


@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("L", [1, 2, 3, 5])
@pytest.mark.parametrize("width", [2, 3, 4])
def test_short_continued(cl, L, width):
    """Continued pieces shorter than the conv's window: the history's gradient reaches past them."""
    run(case(24, "f32", 2, 35, L, 16, conv=width, h0=True, hist=True, dfinal=True), "f32", cl)


@pytest.mark.parametrize("N", [16, 128])
def test_two_pieces_are_one_sequence(N):
    """The gradients of a sequence taken in two pieces: the second piece's dinitial_state and
    dconv_history go into the first one's dfinal_state and its last inputs."""
    L, cut, W = 60, 23, 4
    c = case(25, "f32", 1, 36, L, N, conv=W, h0=True, hist=True, dfinal=True)
    whole = reference(c)
    cuts = {k: (v[:, :, :cut], v[:, :, cut:]) for k, v in c.items() if k in ("u", "delta", "B", "C", "z", "dout")}
    first = dict(c, **{k: v[0] for k, v in cuts.items()}, dfinal=None)
    m, f = ssm(), (lambda v: gpu(v, "f32"))
    _, h = m.ssm_selective_scan_fwd(f(first["u"]), f(first["delta"]), f(c["A"]), f(first["B"]), f(first["C"]),
                                    f(c["D"]), f(first["z"]), f(c["delta_bias"]), True, False, f(c["conv_w"]),
                                    f(c["conv_b"]), return_final_state=True, initial_state=f(c["h0"]),
                                    conv_history=f(c["hist"]))
    second = dict(c, **{k: v[1] for k, v in cuts.items()}, h0=host(h), hist=c["u"][:, :, cut - W + 1:cut])
    second["h0"] = second["h0"].astype(np.float32)
    b = call(second, "f32")
    a = call(dict(first, dfinal=host(b.dinitial_state).astype(np.float32)), "f32")
    du = np.concatenate([host(a.du), host(b.du)], 2)
    du[:, :, cut - W + 1:cut] += host(b.dconv_history)
    check("du", du, whole["du"], "f32")
    for k in ("dA", "dD", "ddelta_bias", "dconv_weight", "dconv_bias"):
        check(k, host(getattr(a, k)) + host(getattr(b, k)), whole[k], "f32")
    check("dinitial_state", host(a.dinitial_state), whole["dinitial_state"], "f32")


def test_guards_around_the_outputs():
    """Nothing is written beside the outputs and the workspace."""
    m = ssm()
    c = case(26, "bf16", 1, 37, 45, 16, conv=4)
    B, D, L, N = 1, 37, 45, 16

    def guarded(n, dtype):
        buf = torch.full((n + 256,), 7, dtype=dtype, device="cuda")
        return buf, buf[128:128 + n]
    outs = {k: guarded(n, torch.bfloat16) for k, n in (("du", D * L), ("ddelta", D * L), ("dz", D * L),
                                                       ("dB", N * L), ("dC", N * L))}
    need = m.ssm_selective_scan_bwd_workspace_size(B, D, L, N, conv_width=4)
    ws, inner = guarded(need, torch.uint8)
    view = {k: v[1].view(1, -1, L) for k, v in outs.items()}
    g = call(c, "bf16", workspace=inner, **view)
    compare(g, reference(c), "bf16")
    for buf in [v[0] for v in outs.values()] + [ws]:
        assert torch.all(buf[:128] == 7) and torch.all(buf[-128:] == 7)


def test_extreme_values():
    """Large and very negative pre-softplus deltas, gates and conv outputs: decays that
    underflow to 0 and deltas near 0 leave finite gradients."""
    c = case(9, "f32", 1, 16, 40, 16, conv=4)
    c["delta"][:, 0], c["delta"][:, 1], c["delta"][:, 2] = 30.0, -60.0, 80.0
    c["z"][:, 3], c["z"][:, 4] = -80.0, 80.0
    c["u"][:, 5] *= 40.0
    run(c, "f32")


def test_strided_views():
    """x, z and their gradients as halves of one in_proj tensor, B, C as columns of x_proj."""
    B, D, L, N = 2, 48, 37, 16
    c = case(10, "bf16", B, D, L, N, conv=4)
    xz = torch.cat([gpu(c["u"], "bf16", True), gpu(c["z"], "bf16", True)], 2)
    bc = torch.cat([torch.zeros(B, L, 3, dtype=torch.bfloat16, device="cuda"),
                    gpu(c["B"], "bf16", True), gpu(c["C"], "bf16", True)], 2)
    dxz = torch.full((B, L, 2 * D + 5), 7.0, dtype=torch.bfloat16, device="cuda")
    dbc = torch.full((B, L, 3 + 2 * N), 7.0, dtype=torch.bfloat16, device="cuda")
    f = lambda k: gpu(c[k], "f32")  # noqa: E731
    g = ssm().ssm_selective_scan_bwd(
        gpu(c["dout"], "bf16", True), xz[..., :D], gpu(c["delta"], "bf16", True), f("A"),
        bc[..., 3:3 + N], bc[..., 3 + N:], f("D"), xz[..., D:], f("delta_bias"), True, False,
        f("conv_w"), f("conv_b"), channel_last=True, du=dxz[..., :D], dz=dxz[..., D:2 * D],
        dB=dbc[..., 3:3 + N], dC=dbc[..., 3 + N:])
    compare(g, reference(c), "bf16", True)
    assert torch.all(dxz[..., 2 * D:] == 7.0) and torch.all(dbc[..., :3] == 7.0)


def test_rows_of_more_steps_than_a_grid_axis_holds_chunks():
    """Either layout of one row of 2^22 + 100 steps, whose conv's gradient takes more than
    65535 chunks channel-last. Inputs within 1 and decays below 0.86 (7 steps of memory): a
    value collects 7 * 2^-22 of terms at most some ten times the rms, in both calls: 4e-5. The
    sums over all steps: 2^22 terms below 10, whose partial sums stay near 10 sqrt(L), rounded
    at random: 2^-24 * 10 L, 2.5; their own 2e-6 each the same way, less. 1e-2 sqrt(L) is 20."""
    B, D, L, N = 1, 3, (1 << 22) + 100, 1
    r = torch.Generator(device="cuda").manual_seed(5)
    f = lambda *s: 2 * torch.rand(*s, device="cuda", generator=r) - 1  # noqa: E731
    u, delta, dout, b, c, w = f(B, D, L), f(B, D, L), f(B, D, L), f(B, N, L), f(B, N, L), f(D, 4) / 2
    A = -torch.rand(D, N, device="cuda", generator=r) - 0.5
    t = lambda x: x.transpose(1, 2).contiguous()  # noqa: E731
    a = ssm().ssm_selective_scan_bwd(dout, u, delta, A, b, c, conv_weight=w)
    g = ssm().ssm_selective_scan_bwd(t(dout), t(u), t(delta), A, t(b), t(c), conv_weight=w, channel_last=True)
    for k in ("du", "ddelta", "dB", "dC"):
        check(k, host(getattr(g, k), True), host(getattr(a, k)), "f32")
    for k in ("dA", "dconv_weight"):
        want = host(getattr(a, k))
        assert np.all(np.abs(host(getattr(g, k)) - want) <= 1e-2 * np.sqrt(L)), k


@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("segments", [1, 3, 7])
@pytest.mark.parametrize("N,conv", [(1, 0), (5, 4), (16, 4), (32, 0), (64, 4), (128, 0)])
def test_a_packed_sequence_that_is_not_finite_leaves_the_others(N, conv, segments, cl):
    """NaN in one sequence's inputs, an infinity in another's incoming gradient: the other
    sequences' gradients keep their bits."""
    D, L, starts = 20, 203, [0, 37, 40, 88, 89, 150, 203]
    c = case(25, "f32", 1, D, L, N, conv=conv)
    want = call(c, "f32", cl, starts=starts, num_segments=segments)
    c["u"][0, :, 60], c["delta"][0, ::3, 41], c["dout"][0, :, 140] = np.nan, np.nan, np.inf
    got = call(c, "f32", cl, starts=starts, num_segments=segments)
    keep = np.r_[0:40, 88:89, 150:203]
    for k in LAST:
        a, o = host(getattr(got, k), cl), host(getattr(want, k), cl)
        assert np.all(np.isfinite(o)) and np.array_equal(a[..., keep], o[..., keep]), k
    assert np.isnan(host(got.dC, cl)[..., 60:88]).all()     # the bad one shows it


@pytest.mark.parametrize("cl", [False, True])
def test_activations_past_32_bit_offsets(cl):
    """2080 channels of 2^20 steps: the last 32 channels' gradients are those of a call on
    these alone."""
    m = ssm()
    D, L, N, last = 2080, 1 << 20, 1, 32
    r = torch.Generator(device="cuda").manual_seed(9)
    act = lambda *s: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(generator=r)  # noqa: E731
    shape, bc = ((1, L, D), (1, L, N)) if cl else ((1, D, L), (1, N, L))
    u, delta, dout, B, C = act(*shape), act(*shape), act(*shape), act(*bc), act(*bc)
    A, w = -torch.rand(D, N, device="cuda", generator=r) - 0.5, torch.randn(D, 4, device="cuda", generator=r) / 2
    kw = dict(channel_last=cl, num_segments=16)
    g = m.ssm_selective_scan_bwd(dout, u, delta, A, B, C, conv_weight=w, **kw)
    end = lambda t: t[..., D - last:] if cl else t[:, D - last:]  # noqa: E731
    o = m.ssm_selective_scan_bwd(end(dout), end(u), end(delta), A[D - last:], B, C, conv_weight=w[D - last:], **kw)
    assert torch.equal(end(g.du), o.du) and torch.equal(end(g.ddelta), o.ddelta)
    assert torch.equal(g.dA[D - last:], o.dA) and torch.equal(g.dconv_weight[D - last:], o.dconv_weight)
    del g, o
    packed = m.ssm_checkpoint_pack(u, channel_last=cl)
    back = end(m.ssm_checkpoint_unpack(packed, channel_last=cl))
    small = m.ssm_checkpoint_pack(end(u), channel_last=cl)
    assert torch.equal(back, m.ssm_checkpoint_unpack(small, channel_last=cl))


def test_misaligned_rows():
    """Rows whose length and base are not multiples of 16 bytes take the scalar loads."""
    c = case(11, "bf16", 2, 33, 61, 16, conv=4)
    want = reference(c)
    off = {}
    for k in ("u", "delta", "z", "dout", "B", "C"):
        flat = gpu(c[k], "bf16")
        buf = torch.zeros(flat.numel() + 1, dtype=torch.bfloat16, device="cuda")
        off[k] = buf[1:].view(flat.shape)
        off[k].copy_(flat)
    f = lambda k: gpu(c[k], "f32")  # noqa: E731
    g = ssm().ssm_selective_scan_bwd(off["dout"], off["u"], off["delta"], f("A"), off["B"], off["C"],
                                     f("D"), off["z"], f("delta_bias"), True, False, f("conv_w"),
                                     f("conv_b"))
    compare(g, want, "bf16")


def test_same_bits_every_time_and_on_another_stream():
    c = case(12, "bf16", 2, 70, 130, 16, conv=4)
    a = call(c, "bf16", num_segments=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = call(c, "bf16", num_segments=2)
    torch.cuda.current_stream().wait_stream(s)
    for k, v in a._asdict().items():
        if v is not None:
            assert torch.equal(v, getattr(b, k)), k


def test_a_given_stream_owns_what_the_call_allocates():
    """stream=: workspaces and outputs come from that stream's memory, so that work queued on the
    current stream right after the call cannot take them over."""
    m = ssm()
    c = case(27, "f32", 2, 64, 200, 16, conv=4)
    f = lambda k: gpu(c[k], "f32")  # noqa: E731
    args = (f("dout"), f("u"), f("delta"), f("A"), f("B"), f("C"), f("D"), f("z"), f("delta_bias"), True, False,
            f("conv_w"), f("conv_b"))
    want = m.ssm_selective_scan_bwd(*args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        got = m.ssm_selective_scan_bwd(*args, stream=side)
        junk = [torch.full((1 << 18,), float("nan"), device="cuda") for _ in range(40)]
        del junk
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(want, got) if x is not None)
    kept = m.ssm_checkpoint_pack(f("u"), stream=side)
    torch.cuda.synchronize()
    assert torch.equal(kept.codes, m.ssm_checkpoint_pack(f("u")).codes)


def test_two_calls_at_once_and_a_graph():
    """Calls on two streams with workspaces of their own, and a captured call replayed on new
    inputs, give what plain calls give."""
    m = ssm()
    cs = [case(s, "f32", 1, 40, 90, 16, conv=4) for s in (13, 14)]
    want = [call(c, "f32") for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = []
    for c, s in zip(cs, streams):
        with torch.cuda.stream(s):
            got.append(call(c, "f32"))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        assert all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)

    ins = {k: gpu(cs[0][k], "f32") for k in cs[0] if cs[0][k] is not None}
    args = lambda: (ins["dout"], ins["u"], ins["delta"], ins["A"], ins["B"], ins["C"], ins["D"],  # noqa: E731
                    ins["z"], ins["delta_bias"], True, False, ins["conv_w"], ins["conv_b"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        g = m.ssm_selective_scan_bwd(*args())
    for c, w in zip(cs, want):
        for k, v in ins.items():
            v.copy_(gpu(c[k], "f32"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(w, g) if x is not None)


@pytest.mark.parametrize("shape", [(0, 8, 5), (2, 0, 5), (2, 8, 0)])
@pytest.mark.parametrize("cl", [False, True])
def test_empty(shape, cl):
    c = case(15, "f32", *shape, 16, conv=4, h0=True, hist=True, dfinal=True)
    g = call(c, "f32", cl)
    for k in ("dA", "dD", "ddelta_bias", "dconv_weight", "dconv_bias", "dB", "dC"):
        assert torch.all(getattr(g, k) == 0), k
    if shape[2] == 0:
        assert torch.equal(g.dinitial_state, gpu(c["dfinal"], "f32"))
        assert torch.all(g.dconv_history == 0)


@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("B,D,L,opt", [(2, 40, 100, {}), (1, 33, 64, dict(reverse=True)), (1, 35, 200, {})])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_from_8_bits(dtype, cl, B, D, L, opt):
    """The gradients from 8-bit activations are those of the values read back."""
    m = ssm()
    c = case(16, dtype, B, D, L, 16, conv=4)
    kept = {k: m.ssm_checkpoint_pack(gpu(c[k], dtype, cl), channel_last=cl) for k in ("u", "delta", "z")}
    t = lambda k: gpu(c[k], dtype, cl)  # noqa: E731
    f = lambda k: gpu(c[k], "f32")  # noqa: E731
    g = m.ssm_selective_scan_bwd(t("dout"), kept["u"], kept["delta"], f("A"), t("B"), t("C"), f("D"),
                                 kept["z"], f("delta_bias"), True, opt.get("reverse", False),
                                 f("conv_w"), f("conv_b"), channel_last=cl)
    back = dict(c)
    for k, v in kept.items():
        back[k] = host(m.ssm_checkpoint_unpack(v, torch.float32, channel_last=cl), cl)
        assert np.max(np.abs(back[k] - c[k])) <= np.max(np.abs(c[k])) / 254 * (1 + 1e-6)
    compare(g, reference(back, **opt), dtype, cl)


def test_training_step_of_a_block():
    """Forward, activations kept in 8 bits, backward of scan and of a conv in front, together:
    the gradients of conv -> scan against the reference's chain."""
    m = ssm()
    B, D, L, N = 2, 40, 96, 16
    c = case(17, "f32", B, D, L, N, dfinal=True)
    w, wb = case(18, "f32", B, D, L, N, conv=4)["conv_w"], case(19, "f32", B, D, L, N, conv=4)["conv_b"]
    f = lambda v: gpu(v, "f32")  # noqa: E731
    x = f(c["u"])
    u = m.ssm_causal_conv1d_fwd(x, f(w), f(wb))
    m.ssm_selective_scan_fwd(u, f(c["delta"]), f(c["A"]), f(c["B"]), f(c["C"]), f(c["D"]), f(c["z"]),
                             f(c["delta_bias"]))
    kept = [m.ssm_checkpoint_pack(v) for v in (u, f(c["delta"]), f(c["z"]))]
    g = m.ssm_selective_scan_bwd(f(c["dout"]), kept[0], kept[1], f(c["A"]), f(c["B"]), f(c["C"]),
                                 f(c["D"]), kept[2], f(c["delta_bias"]), dfinal_state=f(c["dfinal"]))
    gc = m.ssm_causal_conv1d_bwd(g.du, x, f(w), f(wb))
    back = dict(c, **{k: host(m.ssm_checkpoint_unpack(v, torch.float32))
                      for k, v in zip(("u", "delta", "z"), kept)})
    want = reference(back)
    compare(g, want, "f32")
    dx, dw, db, _ = ref.conv_grads(want["du"], c["u"], w, wb)
    for k, a, o in (("dx", gc.dx, dx), ("dw", gc.dw, dw), ("db", gc.dbias, db)):
        check(k, host(a), o, "f32")


def test_bidirectional_is_the_sum_of_two_calls():
    m = ssm()
    c = case(20, "f32", 2, 24, 50, 16)
    r = case(21, "f32", 2, 24, 50, 16)
    a, b = call(c, "f32"), call(dict(c, A=r["A"], D=r["D"]), "f32", reverse=True)
    wa, wb = reference(c), reference(dict(c, A=r["A"], D=r["D"]), reverse=True)
    for k in ("du", "ddelta", "dz", "dB", "dC"):
        check(k, host(getattr(a, k) + getattr(b, k)), wa[k] + wb[k], "f32")


def test_bad_offsets_stay_inside():
    """Offsets out of order or range change results, not what is read or written."""
    c = case(22, "f32", 1, 33, 40, 16, conv=4)
    guard = torch.full((1 << 16,), 3.0, device="cuda")
    for starts in ([5, 9, 40], [0, 30, 10, 40], [0, 1000000, -7, 40], [-5, 2000000000, 3]):
        g = call(c, "f32", starts=starts)
        torch.cuda.synchronize()
        assert all(v.isfinite().all() for v in g if v is not None)
    assert torch.all(guard == 3.0)


def test_refusals():
    m = ssm()
    c = case(23, "f32", 1, 8, 10, 16)
    t = {k: gpu(v, "f32") for k, v in c.items() if v is not None}
    ok = (t["dout"], t["u"], t["delta"], t["A"], t["B"], t["C"])
    with pytest.raises(ValueError):
        m.ssm_selective_scan_bwd(t["dout"], t["u"][:, :, :9].contiguous(), *ok[2:])
    with pytest.raises(TypeError):
        m.ssm_selective_scan_bwd(t["dout"], t["u"].bfloat16(), *ok[2:])
    with pytest.raises(ValueError):
        m.ssm_selective_scan_bwd(t["dout"].cpu(), *ok[1:])
    with pytest.raises(ValueError):                       # time-invariant B, C
        m.ssm_selective_scan_bwd(*ok[:4], t["A"], t["A"])
    with pytest.raises(TypeError):
        m.ssm_selective_scan_bwd(t["dout"], m.ssm_checkpoint_pack(t["u"]), *ok[2:])
    with pytest.raises(m.SSMError) as e:
        m.ssm_selective_scan_bwd(*ok, initial_state=torch.zeros(1, 8, 16, device="cuda"), reverse=True)
    assert e.value.name == "SSM_ERR_UNSUPPORTED"
    with pytest.raises(m.SSMError) as e:
        m.ssm_selective_scan_bwd(*ok, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.name == "SSM_ERR_WORKSPACE"
    with pytest.raises(m.SSMError) as e:
        m.ssm_selective_scan_bwd(*ok, du=t["u"])
    assert e.value.name == "SSM_ERR_ALIAS"


def test_a_conv_of_no_taps_is_refused():
    """An empty weight has no address: it must not read as a call without a conv."""
    m = ssm()
    c = case(24, "f32", 1, 8, 10, 16)
    t = {k: gpu(v, "f32") for k, v in c.items() if v is not None}
    none = torch.zeros(8, 0, device="cuda")
    with pytest.raises(ValueError):
        m.ssm_selective_scan_bwd(t["dout"], t["u"], t["delta"], t["A"], t["B"], t["C"], conv_weight=none)
    with pytest.raises(ValueError):
        m.ssm_selective_state_update_cached(
            torch.zeros(1, 8, 16, dtype=torch.int8, device="cuda"), torch.zeros(1, 8, device="cuda"),
            torch.zeros(1, 8, 0, device="cuda"), t["u"][:, :, 0].contiguous(), t["u"][:, :, 0].contiguous(),
            t["A"], t["B"][:, :, 0].contiguous(), t["C"][:, :, 0].contiguous(), conv_weight=none)
