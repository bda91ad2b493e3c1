"""The rounding of the 8-bit state cache's decode step, decided on states that a step leaves as
they are: A = 0 and delta = 0, so that the new state is code * scale in fp32."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

ROWS = 1 << 21


def ssm():
    import mamba_selective_scan_sm_b200 as m
    return m


def held(values, n, seed):
    """A cache of one slot whose rows all hold the codes ``values`` (zeros behind them), at
    scales of many magnitudes and all mantissas; and the fp32 states it stands for."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    codes = torch.zeros(1, ROWS, n, dtype=torch.int8, device="cuda")
    codes[..., :len(values)] = torch.tensor(values, dtype=torch.int8, device="cuda")
    scales = torch.exp(torch.rand(1, ROWS, generator=g, device="cuda") * 40 - 20)
    return codes, scales, codes.float() * scales[..., None], g


def step(codes, scales, rand):
    n = codes.shape[2]
    zero, bc = torch.zeros(1, ROWS, device="cuda"), torch.zeros(1, n, device="cuda")
    ssm().ssm_selective_state_update_cached(codes, scales, None, zero, zero, torch.zeros(ROWS, n, device="cuda"),
                                            bc, bc, dt_softplus=False, rand=rand)


def quotients(h):
    h = h.double()
    return 127.0 * h / h.abs().amax(-1, keepdim=True)


@pytest.mark.parametrize("n", [4, 16, 48])
@pytest.mark.parametrize("values", [(127, 100, 1, -77), (-127, 3, -100, 50), (64, -64, 63, 1)])
def test_the_step_is_right_on_average(values, n):
    """Over random bits the mean code is the quotient. A quotient 127 h / max|h| of these states
    lies within 2e-5 of a whole number (a few roundings of 2^-24), or for the rows of 64 anywhere:
    its codes k and k + 1 have a variance of f (1 - f), f its fraction, and the mean over the rows
    a standard error from that. The step may be off by 4e-7 of a code by itself (its offset's
    24th bit 6e-8, a rounding at 2 1.2e-7, the row's largest state held below 128 by 1.2e-7): a
    probability p <= 4e-7 of the code beside, which is counted in 2^23 draws with a standard error
    of its own, sqrt(4e-7 / 2^23) = 2.2e-7 (one draw more or less moves the mean by 1.2e-7, so the
    count is a Poisson one). So the variance is f (1 - f) + p."""
    codes, scales, h, g = held(values, n, 1)
    want = quotients(h)
    total, times = torch.zeros(n, dtype=torch.float64, device="cuda"), 4
    for _ in range(times):
        c, s = codes.clone(), scales.clone()
        rand = torch.randint(-2 ** 31, 2 ** 31, (1, ROWS), generator=g, device="cuda", dtype=torch.int64)
        step(c, s, rand.to(torch.int32))
        off = c.double() - want
        assert float(off.abs().max()) < 1 + 1e-6 and int(c.abs().max()) <= 127
        total += off.mean((0, 1))
    f = want - want.floor()
    error = (((f * (1 - f)).mean((0, 1)) + 4e-7) / (ROWS * times)).sqrt()
    off = (total / times).abs()
    assert bool((off <= 6 * error + 4e-7).all()), (off, error)


@pytest.mark.parametrize("n", [4, 16, 48])
def test_the_step_takes_the_offsets_it_is_given(n):
    """floor(127 h / max|h| + offset), but for sums within 1e-6 of a whole number."""
    codes, scales, h, g = held((127, 99, -50, 7), n, 2)
    noise = torch.randn(h.shape, generator=g, device="cuda")
    zero = torch.zeros(1, ROWS, device="cuda")
    rand = torch.randint(-2 ** 31, 2 ** 31, (1, ROWS), generator=g, device="cuda", dtype=torch.int64)
    codes = torch.where(codes == 0, (noise * 30).clamp(-126, 126).to(torch.int8), codes)
    h = codes.float() * scales[..., None]
    c, s = codes.clone(), scales.clone()
    step(c, s, rand.to(torch.int32))
    k = torch.arange(n, device="cuda")
    bits = (rand[..., None] + k * 0x9E3779B9) & 0xFFFFFFFF
    v = quotients(h) + (bits >> 8).double() * 2.0 ** -24
    sure = (v - v.round()).abs() > 1e-6
    assert torch.equal(c[sure].double(), v[sure].floor()) and float(sure.double().mean()) > 0.5
    assert bool(((c.double() - v.floor()).abs() <= 1).all()) and not zero.any()
    assert torch.equal(s, h.abs().amax(-1) / torch.full_like(s, 127.0))   # (a division: by a number torch multiplies)


@pytest.mark.parametrize("n", [4, 16, 48])
def test_the_step_to_the_nearest(n):
    """Without random bits: round(127 h / max|h|), but for quotients within 1e-5 of a border
    (127 times a rounding of 2^-24, and of the reciprocal)."""
    codes, scales, h, g = held((127, 99, -50, 7), n, 3)
    B = torch.randn(1, n, generator=g, device="cuda")
    du = torch.rand(1, ROWS, generator=g, device="cuda") + 0.5
    c, s = torch.zeros_like(codes), torch.zeros_like(scales)
    one = torch.ones(1, ROWS, device="cuda")
    ssm().ssm_selective_state_update_cached(c, s, None, du, one, torch.zeros(ROWS, n, device="cuda"), B,
                                            torch.zeros_like(B), dt_softplus=False)
    new = du[..., None] * B                                 # 0 + (1 x) B, one rounding
    v = quotients(new)
    sure = ((v - v.floor()) - 0.5).abs() > 1e-5
    assert torch.equal(c[sure].double(), v[sure].round()) and float(sure.double().mean()) > 0.99
    assert torch.equal(s, new.abs().amax(-1) / torch.full_like(s, 127.0))


def test_steps_repeat_their_bits():
    """The same tokens on the same cache give the same codes, outputs and conv states again,
    also with a call on another cache between."""
    m, (b, d, n) = ssm(), (64, 1536, 16)
    g = torch.Generator(device="cuda").manual_seed(4)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    state, A, D, w, wb = r(b, d, n), -r(d, n).abs() - 0.5, r(d), r(d, 4) / 2, r(d)
    x, dt, z, B, C = (r(3, b, k).bfloat16() for k in (d, d, d, n, n))
    rand = torch.randint(-2 ** 31, 2 ** 31, (3, b, d), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    slots = torch.randperm(b, generator=g, device="cuda").to(torch.int32)
    conv0 = r(b, d, 4).bfloat16()

    def tokens():
        codes, scales = torch.zeros(b, d, n, dtype=torch.int8, device="cuda"), torch.zeros(b, d, device="cuda")
        conv = conv0.clone()
        m.ssm_state_cache_write(state, codes, scales, slots=slots, rand=rand[0])
        y = [m.ssm_selective_state_update_cached(codes, scales, conv, x[t], dt[t], A, B[t], C[t], D, z[t], D, True,
                                                 w, wb, slots=slots, rand=rand[t]) for t in range(3)]
        return [codes, scales, conv, *y]
    first = tokens()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, tokens()))


@pytest.mark.parametrize("random", [False, True])
def test_the_step_over_all_magnitudes(random):
    """Rows of every code at scales 2^k, the largest state from 2^-99 to 2^127: quotients are whole
    numbers, so every code stays (at random but for 3e-7 of them: none of 29,000 to expect). Below
    2^-100 a row becomes zeros."""
    m, n = ssm(), 128
    k = torch.arange(-112, 121, device="cuda")
    dim = len(k)
    row = torch.cat([torch.arange(0, 128, 2), -torch.arange(1, 129, 2)]).to(torch.int8)
    codes = row.cuda().repeat(1, dim, 1)
    scales = torch.exp2(k.double()).float()[None].contiguous()
    g = torch.Generator(device="cuda").manual_seed(6)
    zero, bc = torch.zeros(1, dim, device="cuda"), torch.zeros(1, n, device="cuda")
    want, ws = codes.clone(), scales.clone()
    top = codes.abs().amax(-1).float() * scales
    want[top < 2.0 ** -100], ws[top < 2.0 ** -100] = 0, 0
    for _ in range(2):
        rand = torch.randint(-2 ** 31, 2 ** 31, (1, dim), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
        m.ssm_selective_state_update_cached(codes, scales, None, zero, zero, torch.zeros(dim, n, device="cuda"), bc, bc,
                                            dt_softplus=False, rand=rand if random else None)
        assert torch.equal(codes, want) and torch.equal(scales, ws)


@pytest.mark.parametrize("random", [False, True])
@pytest.mark.parametrize("n", [3, 16, 64, 100])
def test_a_step_that_is_not_finite(n, random):
    """An infinity or a NaN in a channel's input makes that row of the slot read back as NaN, now and
    after the next token; every other row keeps its bits."""
    m, B, D = ssm(), 3, 40
    g = torch.Generator(device="cuda").manual_seed(7)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    state, A, x, dt, Bt, Ct = r(B, D, n), -r(D, n).abs() - 0.1, r(B, D), r(B, D), r(B, n), r(B, n)
    rand = torch.randint(-2 ** 31, 2 ** 31, (B, D), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    bad = [(0, 3, float("inf")), (1, 0, float("nan")), (2, 39, float("-inf"))]

    def tokens(spoil):
        codes, scales = torch.zeros(B, D, n, dtype=torch.int8, device="cuda"), torch.zeros(B, D, device="cuda")
        m.ssm_state_cache_write(state, codes, scales)
        first = x.clone()
        for b, d, v in bad if spoil else []:
            first[b, d] = v
        y = [m.ssm_selective_state_update_cached(codes, scales, None, u, dt, A, Bt, Ct, rand=rand if random else None)
             for u in (first, x)]
        return [*y, m.ssm_state_cache_read(codes, scales)]
    want, got = tokens(False), tokens(True)
    keep = torch.ones(B, D, dtype=torch.bool, device="cuda")
    for b, d, _ in bad:
        keep[b, d] = False
    for a, o in zip(got, want):
        assert torch.equal(a[keep], o[keep])
    assert torch.isnan(got[2][~keep]).all() and torch.isnan(got[1][~keep]).all()
    assert not torch.isfinite(got[0][~keep]).any()
