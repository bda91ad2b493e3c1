"""Sums over very long rows in the scan's gradient, where the terms have one sign and a plain
fp32 sum would lose them; and steps that leave the states as they are."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def ssm():
    import mamba_selective_scan_sm_b200 as m
    return m


def closed_form(L, A, d):
    """The gradients' sums for u = B = dout = 1, C = 1 / N, delta = d at every step, in double
    precision: h and lambda are geometric sums."""
    a = np.exp(d * A)                                        # lambda_t = (1 - a^(L-t)) / (1 - a) / N
    aL, n = a ** L, A.shape[1]                               # h_(t-1) = d (1 - a^t) / (1 - a)
    up, down = (1 - aL) / (1 - a), a * (1 - aL) / (1 - a)    # sums of a^t and of a^(L-t)
    lam = (L - down) / (1 - a) / n
    q = a * d * (L - down - up + L * aL) / (1 - a) ** 2 / n
    return d * q, (lam + q * A).sum(1)


@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("N", [1, 5, 16, 32, 128])
def test_terms_of_one_sign(N, cl):
    """2^19 and more steps in one segment. A decay of at most e^-0.25 = 0.78 is off by 2^-22
    relative, h and lambda by 4.5 times that, their product by 2.2e-6; 512 additions of one sign
    add at most 2^-25 each on average (1.5e-5) before a sum joins the others: 2e-5."""
    m = ssm()
    L, D, d = (1 << 19) + 40, 3, 0.5
    A = -np.linspace(0.5, 4.0, D * N).reshape(D, N).astype(np.float32)
    want_A, want_bias = closed_form(L, A.astype(np.float64), d)
    one = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    act, bc = ((1, L, D), (1, L, N)) if cl else ((1, D, L), (1, N, L))
    g = m.ssm_selective_scan_bwd(one(*act), one(*act), d * one(*act), torch.from_numpy(A).cuda(), one(*bc),
                                 one(*bc) / N, one(D), None, torch.zeros(D, device="cuda"), False,
                                 channel_last=cl, num_segments=1)
    for k, o in (("dA", want_A), ("ddelta_bias", want_bias), ("dD", np.full(D, float(L)))):
        got = getattr(g, k).cpu().numpy().astype(np.float64)
        assert np.all(np.abs(got - o) <= 2e-5 * np.abs(o)), (k, got / o - 1)


@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("segments", [1, 3])
@pytest.mark.parametrize("N,heads", [(1, 0), (5, 0), (16, 0), (24, 0), (128, 0), (16, 2), (128, 4)])
def test_steps_without_time_change_no_bit(N, heads, segments, cl):
    """delta = 0 at every step (and the steps that fill the last tile): the decay is 1 exactly,
    so the gradient of the last state is that of the first, and dC is g times that state."""
    m = ssm()
    B, D, L = 2, 36, 5003
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    A = -torch.rand(heads, generator=g, device="cuda") - 1 if heads else -r(D, N).abs() - 0.5
    h0, dhl = r(B, D, N), r(B, D, N)
    t = lambda v: v.transpose(1, 2).contiguous() if cl else v  # noqa: E731
    zero = torch.zeros(B, D, L, device="cuda")
    dout = zero.clone()
    dout[:, 7, 4000] = 1.0
    out = m.ssm_selective_scan_bwd(t(dout), t(r(B, D, L)), t(zero), A, t(r(B, N, L)), t(torch.zeros(B, N, L, device="cuda")),
                                   delta_softplus=False, initial_state=h0, dfinal_state=dhl, channel_last=cl,
                                   num_segments=segments)
    assert torch.equal(out.dinitial_state, dhl)
    dC = t(out.dC)
    assert torch.equal(dC[:, :, 4000], h0[:, 7])


@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("segments", [1, 4])
@pytest.mark.parametrize("lo,hi,e", [(1e-4, 1e-3, 2e-9), (0.01, 0.02, 1.4e-8), (0.05, 0.1, 1.4e-8)])
def test_states_keep_their_memory(lo, hi, e, segments, cl):
    """All terms of one sign. A state remembers 1 / (1 - a) steps and takes up the decay's mean error e
    once for each: dA, a product of two such states, is off by at most 2 e / (1 - a). The SFU's exp is
    low by 4.6e-9 to 8e-9 for exponents above -0.003 and the kernel raises its exponents by 0.9e-8,
    its values by 6.2e-9: e is at most 2e-9. Below -0.0055 it is low by 0.8e-8 to 3.1e-8, raised by
    2.15e-8: at most 1.4e-8. The decays' own roundings are of either sign, 2^-25 each at most: over
    8192 steps 90 of them add up, 2.7e-6 (and lambda's as much)."""
    from tests import bwd_reference as ref
    m, (D, L, N) = ssm(), (6, 8192, 4)
    r = np.random.default_rng(5)
    delta = r.uniform(lo, hi, (1, D, L)).astype(np.float32)
    A = -np.linspace(0.5, 2.0, D * N).reshape(D, N).astype(np.float32)
    u, dout = (r.uniform(0.5, 1.5, (1, D, L)).astype(np.float32) for _ in range(2))
    B, C = (r.uniform(0.5, 1.5, (1, N, L)).astype(np.float32) for _ in range(2))
    want = ref.scan_grads(dout, u, delta, A, B, C, softplus=False)["dA"]
    t = lambda v: torch.from_numpy(v.transpose(0, 2, 1).copy() if cl else v).cuda()  # noqa: E731
    g = m.ssm_selective_scan_bwd(t(dout), t(u), t(delta), torch.from_numpy(A).cuda(), t(B), t(C), delta_softplus=False,
                                 channel_last=cl, num_segments=segments)
    memory = 1.0 / (delta.mean() * -A.astype(np.float64))
    off = np.abs(g.dA.cpu().numpy() / want - 1)
    assert np.all(off <= 2 * e * memory + 2 * 2.7e-6), off / memory
