"""Activations and decode states in 8 bits on the GPU: codes decided exactly, values read back,
decode steps on a cache against the double-precision oracle."""
import numpy as np
import pytest
import torch

import oracle
from tests import bwd_reference as ref
from tests.bwd_helpers import check, gpu, host
from mamba_selective_scan_sm_b200.synth import round_bf16

pytestmark = pytest.mark.gpu


def ssm():
    import mamba_selective_scan_sm_b200 as m
    return m


def blocks(x):
    pad = -x.shape[2] % 64
    return np.pad(x, ((0, 0), (0, 0), (0, pad))).reshape(x.shape[0], x.shape[1], -1, 64)


# ------------------------------------------------------------------ activations --

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("B,D,L", [(1, 1, 1), (2, 3, 64), (1, 5, 65), (2, 9, 130), (1, 260, 7), (1, 33, 200)])
def test_pack_exact(dtype, cl, B, D, L):
    m = ssm()
    r = np.random.default_rng(1)
    x = r.standard_normal((B, D, L)).astype(np.float32)
    x[:, 0, ::3] = np.round(x[:, 0, ::3] * 254) / 254      # values near the borders
    x = round_bf16(x) if dtype == "bf16" else x
    kept = m.ssm_checkpoint_pack(gpu(x, dtype, cl), channel_last=cl)
    codes, scales = ref.pack_reference(blocks(x))
    codes = codes.reshape(B, D, -1)[:, :, :L]
    got = kept.codes.transpose(1, 2) if cl else kept.codes
    assert np.array_equal(got.cpu().numpy(), codes)
    gs = kept.scales.transpose(1, 2) if cl else kept.scales
    assert np.array_equal(gs.cpu().numpy(), scales)
    back = m.ssm_checkpoint_unpack(kept, torch.float32, channel_last=cl)
    want = codes * np.repeat(scales, 64, 2)[:, :, :L]
    assert np.array_equal(host(back, cl).astype(np.float32), want.astype(np.float32))
    low = m.ssm_checkpoint_unpack(kept, channel_last=cl)
    assert torch.equal(low, back.bfloat16())


@pytest.mark.parametrize("cl", [False, True])
def test_pack_ties(cl):
    """127 x / max on a half exactly: to even, as in rational arithmetic."""
    x = np.zeros((1, 1, 64), dtype=np.float32)
    x[0, 0, 0] = 127.0
    x[0, 0, 1:64] = np.arange(1, 64) - 31.5
    kept = ssm().ssm_checkpoint_pack(gpu(x, "f32", cl), channel_last=cl)
    assert np.array_equal(kept.codes.cpu().numpy().ravel(), np.rint(x.ravel()).astype(np.int8))


@pytest.mark.parametrize("cl", [False, True])
def test_pack_special_values(cl):
    m = ssm()
    x = np.random.default_rng(2).standard_normal((1, 6, 128)).astype(np.float32)
    x[0, 0, 3], x[0, 1, 70], x[0, 2, 0] = np.inf, np.nan, -np.inf
    x[0, 3, :64] = 0.0
    x[0, 4, :64] *= np.float32(1e-33)
    x[0, 5] *= np.float32(1e30)
    back = host(m.ssm_checkpoint_unpack(m.ssm_checkpoint_pack(gpu(x, "f32", cl), channel_last=cl),
                                        torch.float32, channel_last=cl), cl)
    bad = np.zeros((6, 2), dtype=bool)
    bad[0, 0] = bad[1, 1] = bad[2, 0] = True
    nan = np.isnan(back).reshape(6, 2, 64)
    assert np.array_equal(nan.all(2), bad) and np.array_equal(nan.any(2), bad)
    assert np.all(back[0, 3, :64] == 0) and np.all(back[0, 4, :64] == 0)
    assert np.max(np.abs(back[0, 5] - x[0, 5])) <= np.max(np.abs(x[0, 5])) / 254 * (1 + 1e-6)


def test_pack_strided_and_misaligned():
    m = ssm()
    r = np.random.default_rng(3)
    xz = torch.from_numpy(r.standard_normal((2, 70, 50)).astype(np.float32)).cuda().bfloat16()
    for lo, hi in ((0, 24), (1, 26), (24, 50)):
        v = xz[..., lo:hi]
        a = m.ssm_checkpoint_pack(v, channel_last=True)
        b = m.ssm_checkpoint_pack(v.contiguous(), channel_last=True)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)
    buf = torch.zeros(2 * 3 * 100 + 1, dtype=torch.bfloat16, device="cuda")
    x = buf[1:].view(2, 3, 100)
    x.copy_(xz.reshape(-1)[:600].view(2, 3, 100))
    a, b = m.ssm_checkpoint_pack(x), m.ssm_checkpoint_pack(x.clone())
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@pytest.mark.parametrize("shape", [(0, 3, 4), (2, 0, 4), (2, 3, 0)])
@pytest.mark.parametrize("cl", [False, True])
def test_pack_empty(shape, cl):
    m = ssm()
    kept = m.ssm_checkpoint_pack(torch.zeros(shape, device="cuda"), channel_last=cl)
    assert m.ssm_checkpoint_unpack(kept, channel_last=cl).shape == shape


# ----------------------------------------------------------------- decode states --

def dither(x, rand):
    """floor(127 x / max + offset) in double precision, and whether that is far from a border."""
    n = x.shape[-1]
    bits = (rand.astype(np.int64)[..., None] + np.arange(n) * 0x9E3779B9) & 0xFFFFFFFF
    v = 127.0 * x.astype(np.float64) / np.max(np.abs(x), -1, keepdims=True) + (bits >> 8) / 2.0 ** 24
    return np.clip(np.floor(v), -127, 127), np.abs(v - np.rint(v)) > 1e-9


@pytest.mark.parametrize("dim,n", [(1, 1), (5, 3), (7, 16), (33, 16), (4, 20), (9, 48), (3, 64), (5, 100), (4, 128)])
@pytest.mark.parametrize("random", [False, True])
def test_cache_write_and_read(dim, n, random):
    m = ssm()
    r = np.random.default_rng(4)
    state = r.standard_normal((4, dim, n)).astype(np.float32)
    slots = torch.tensor([5, -1, 0, 7], dtype=torch.int32, device="cuda")
    codes = torch.full((7, dim, n), 9, dtype=torch.int8, device="cuda")
    scales = torch.full((7, dim), 4.0, device="cuda")
    rand = r.integers(-2 ** 31, 2 ** 31, (4, dim)).astype(np.int32)
    m.ssm_state_cache_write(gpu(state, "f32"), codes, scales, slots=slots,
                            rand=torch.from_numpy(rand).cuda() if random else None)
    got, gs = codes.cpu().numpy(), scales.cpu().numpy()
    for row, slot in ((0, 5), (2, 0)):                     # 7 is past the end: padding too
        want, ws = ref.pack_reference(state[row])
        if random:
            want, sure = dither(state[row], rand[row])
            assert np.array_equal(got[slot][sure], want[sure])
        else:
            assert np.array_equal(got[slot], want)
        assert np.array_equal(gs[slot], ws)
    for slot in (1, 2, 3, 4, 6):
        assert np.all(got[slot] == 9) and np.all(gs[slot] == 4.0)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.full((4, dim, n), 2.0, dtype=dt, device="cuda")
        m.ssm_state_cache_read(codes, scales, slots=slots, out=out)
        assert torch.all(out[1] == 2.0) and torch.all(out[3] == 2.0)
        for row, slot in ((0, 5), (2, 0)):
            assert torch.equal(out[row], (codes[slot].float() * scales[slot][:, None]).to(dt))
    assert torch.all(m.ssm_state_cache_read(codes, scales, slots=slots)[1] == 0)
    assert torch.equal(m.ssm_state_cache_read(codes, scales), codes.float() * scales[:, :, None])


def test_cache_special_rows():
    m = ssm()
    state = np.random.default_rng(5).standard_normal((1, 5, 16)).astype(np.float32)
    state[0, 0, 3], state[0, 1, 2], state[0, 2], state[0, 3] = np.inf, np.nan, 0.0, 1e-35
    codes = torch.zeros(1, 5, 16, dtype=torch.int8, device="cuda")
    scales = torch.zeros(1, 5, device="cuda")
    m.ssm_state_cache_write(gpu(state, "f32"), codes, scales)
    back = m.ssm_state_cache_read(codes, scales)[0].cpu().numpy()
    assert np.all(np.isnan(back[:2])) and np.all(back[2:4] == 0) and np.all(np.isfinite(back[4]))


def test_a_cache_past_32_bit_offsets():
    """Slots whose codes lie past 2^31 bytes, at both ends of the cache."""
    m = ssm()
    num, dim, n = 70000, 2048, 16
    codes = torch.zeros(num, dim, n, dtype=torch.int8, device="cuda")
    scales = torch.zeros(num, dim, device="cuda")
    state = torch.randn(3, dim, n, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    slots = torch.tensor([num - 1, 0, 67000], dtype=torch.int32, device="cuda")
    m.ssm_state_cache_write(state, codes, scales, slots=slots)
    back = m.ssm_state_cache_read(codes, scales, slots=slots)
    top = state.abs().amax(-1, keepdim=True)
    assert torch.all((back - state).abs() <= top / 254 * (1 + 1e-5))
    one = torch.zeros(3, dim, device="cuda")
    bc = torch.ones(3, n, device="cuda")
    y = m.ssm_selective_state_update_cached(codes, scales, None, one, one, torch.zeros(dim, n, device="cuda"), bc, bc,
                                            dt_softplus=False, slots=slots)
    assert torch.allclose(y, back.sum(-1), rtol=1e-5, atol=1e-5)
    assert torch.equal(m.ssm_state_cache_read(codes, scales, slots=slots), back)
    assert not codes[1:67000].any() and not codes[67001:num - 1].any()


def test_dither_is_right_on_average():
    """A value a fifth of a step above a code: over random bits the stored mean is the value.
    4096 draws of a step's fraction have a standard error of 0.4 / 64 = 0.00625 steps; the
    test allows six."""
    m = ssm()
    rows = 4096
    state = np.zeros((rows, 1, 2), dtype=np.float32)
    state[:, 0, 0], state[:, 0, 1] = 127.0, 40.2
    rand = np.random.default_rng(6).integers(-2 ** 31, 2 ** 31, (rows, 1)).astype(np.int32)
    codes = torch.zeros(rows, 1, 2, dtype=torch.int8, device="cuda")
    scales = torch.zeros(rows, 1, device="cuda")
    m.ssm_state_cache_write(gpu(state, "f32"), codes, scales, rand=torch.from_numpy(rand).cuda())
    v = codes.cpu().numpy()[:, 0]
    assert np.all(v[:, 0] == 127) and set(np.unique(v[:, 1])) == {40, 41}
    assert abs(v[:, 1].mean() - 40.2) <= 6 * 0.00625


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("dim,n,heads,conv,z", [
    (7, 16, 0, 4, True), (64, 16, 0, 4, True), (33, 16, 3, 2, True), (5, 3, 0, 0, False), (6, 20, 2, 3, True),
    (8, 64, 0, 4, True), (8, 128, 4, 4, True), (4, 100, 0, 1, False), (130, 1, 0, 4, True)])
def test_decode_on_the_cache(dtype, dim, n, heads, conv, z):
    """One token at a time: out against the oracle's step from the values the cache held
    before, and each stored value within half a step of the oracle's new state."""
    m = ssm()
    r = np.random.default_rng(7)
    rnd = round_bf16 if dtype == "bf16" else (lambda v: v)
    act = lambda *s: rnd(r.standard_normal(s).astype(np.float32))  # noqa: E731
    f32 = lambda *s: r.standard_normal(s).astype(np.float32)  # noqa: E731
    A = (-r.uniform(1, 8, heads) if heads else -r.uniform(1, 8, (dim, n))).astype(np.float32)
    D, bias = f32(dim), f32(dim)
    w, wb = (0.5 * f32(dim, conv), f32(dim)) if conv else (None, None)
    rows = [3, 0, 4]                                       # slots of batch rows 0, 2, 3; row 1 padded
    slots = torch.tensor([3, -1, 0, 4], dtype=torch.int32, device="cuda")
    live = [0, 2, 3]
    codes = torch.zeros(5, dim, n, dtype=torch.int8, device="cuda")
    scales = torch.zeros(5, dim, device="cuda")
    m.ssm_state_cache_write(gpu(f32(4, dim, n), "f32"), codes, scales, slots=slots)
    conv_state = gpu(act(5, dim, conv), dtype) if conv else None
    kept = (codes[1].clone(), scales[2].clone())
    for step in range(4):
        x, dt, zz = act(4, dim), rnd(0.5 * f32(4, dim)), act(4, dim) if z else None
        Bt, Ct = act(4, n), act(4, n)
        before = host(m.ssm_state_cache_read(codes, scales))
        cs = host(conv_state)[rows] if conv else None
        pick = lambda v: None if v is None else v[live]  # noqa: E731
        yo, ho, co = oracle.state_update(before[rows], cs, pick(x), pick(dt), A, Bt[live], Ct[live], D,
                                         pick(zz), bias, True, w, wb)
        out = torch.full((4, dim), 5.0, dtype=torch.float32 if dtype == "f32" else torch.bfloat16, device="cuda")
        m.ssm_selective_state_update_cached(
            codes, scales, conv_state, gpu(x, dtype), gpu(dt, dtype), gpu(A, "f32"), gpu(Bt, dtype),
            gpu(Ct, dtype), gpu(D, "f32"), gpu(zz, dtype), gpu(bias, "f32"), True, gpu(w, "f32"),
            gpu(wb, "f32"), slots=slots, out=out)
        assert torch.all(out[1] == 5.0)
        check("dx", host(out)[live], yo, dtype)
        after, top = host(m.ssm_state_cache_read(codes, scales))[rows], np.max(np.abs(ho), -1, keepdims=True)
        assert np.all(np.abs(after - ho) <= top / 254 + 1e-5 * top)
        if conv:
            assert np.array_equal(host(conv_state)[rows], co)
    assert torch.equal(codes[1], kept[0]) and torch.equal(scales[2], kept[1])


@pytest.mark.parametrize("n", [3, 16, 48])
def test_the_largest_state_keeps_its_code(n):
    """Rounding offsets next to 1 on the row's largest state, of either sign: 127 plus the offset
    stays below 128 whatever the fp32 reciprocal does, over many magnitudes. (The step takes the
    quotient within 1e-4: -127 plus such an offset may come out as -127 or -126.)"""
    m = ssm()
    rows = 20000
    g = torch.Generator(device="cuda").manual_seed(2)
    top = torch.exp(torch.rand(rows, 1, generator=g, device="cuda") * 40 - 20)
    for at in (0, n - 1):
        offset = (0xFFFFFFFF - at * 0x9E3779B9) & 0xFFFFFFFF          # state `at` gets the last offset
        rand = torch.full((rows, 1), offset - (1 << 32) if offset >> 31 else offset, dtype=torch.int32, device="cuda")
        for sign in (1.0, -1.0):
            state = 0.3 * top[..., None] * (2 * torch.rand(rows, 1, n, generator=g, device="cuda") - 1)
            state[:, 0, at] = sign * top[:, 0]
            codes = torch.zeros(rows, 1, n, dtype=torch.int8, device="cuda")
            scales = torch.zeros(rows, 1, device="cuda")
            m.ssm_state_cache_write(state, codes, scales, rand=rand)
            want = 127 if sign > 0 else -127
            for _ in range(2):
                assert bool((codes[:, 0, at] == want).all() if sign > 0 else (codes[:, 0, at] <= -126).all())
                zero, bc = torch.zeros(rows, 1, device="cuda"), torch.zeros(rows, n, device="cuda")
                m.ssm_selective_state_update_cached(codes, scales, None, zero, zero, torch.zeros(1, n, device="cuda"),
                                                    bc, bc, dt_softplus=False, rand=rand)


def test_a_state_decays_only_when_dithered():
    """delta A small enough that one token decays a state by less than half a step: rounding
    to the nearest keeps it where it is, dithered rounding loses it at the right rate."""
    m = ssm()
    rows, steps, a = 2048, 50, 0.999
    A = torch.tensor([[0.0, np.log(a) / 0.01]], dtype=torch.float32, device="cuda")
    zero = torch.zeros(rows, 1, device="cuda")
    dt = torch.full((rows, 1), 0.01, device="cuda")
    Bt = torch.zeros(rows, 2, device="cuda")
    state = torch.tensor([127.0, 100.0], device="cuda").repeat(rows, 1, 1)
    g = torch.Generator(device="cuda").manual_seed(1)
    ends = []
    for random in (False, True):
        codes = torch.zeros(rows, 1, 2, dtype=torch.int8, device="cuda")
        scales = torch.zeros(rows, 1, device="cuda")
        m.ssm_state_cache_write(state, codes, scales)
        for _ in range(steps):
            rand = torch.randint(-2 ** 31, 2 ** 31, (rows, 1), generator=g, device="cuda", dtype=torch.int64)
            m.ssm_selective_state_update_cached(codes, scales, None, zero, dt, A, Bt, Bt, dt_softplus=False,
                                                rand=rand.to(torch.int32) if random else None)
        ends.append(float(m.ssm_state_cache_read(codes, scales)[:, 0, 1].mean()))
    assert ends[0] == 100.0
    # 50 steps of variance at most 1/4 each, 2048 rows: standard error at most 0.08
    assert abs(ends[1] - 100.0 * a ** steps) <= 6 * 0.08


def test_prompt_to_tokens():
    """A prompt scanned, its states and conv states put into the cache, tokens decoded on it:
    as the oracle does it with the states rounded the same way."""
    m = ssm()
    r = np.random.default_rng(8)
    B, D, L, N, W = 2, 24, 30, 16, 4
    f32 = lambda *s: r.standard_normal(s).astype(np.float32)  # noqa: E731
    u, dl, z, Bm, Cm = f32(B, D, L), 0.5 * f32(B, D, L), f32(B, D, L), f32(B, N, L), f32(B, N, L)
    A, Dv, bias, w, wb = -np.abs(f32(D, N)) - 0.5, f32(D), f32(D) - 2, 0.5 * f32(D, W), f32(D)
    g = lambda v: gpu(v, "f32")  # noqa: E731
    _, h, cs = m.ssm_selective_scan_fwd(g(u), g(dl), g(A), g(Bm), g(Cm), g(Dv), g(z), g(bias), True, False,
                                        g(w), g(wb), return_final_state=True, return_conv_state=True)
    codes = torch.zeros(3, D, N, dtype=torch.int8, device="cuda")
    scales = torch.zeros(3, D, device="cuda")
    slots = torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    conv = torch.zeros(3, D, W, device="cuda")
    m.ssm_state_cache_write(h, codes, scales, slots=slots)
    conv[[2, 0]] = cs
    for _ in range(3):
        x, dt, zt, Bt, Ct = f32(B, D), 0.5 * f32(B, D), f32(B, D), f32(B, N), f32(B, N)
        held = host(m.ssm_state_cache_read(codes, scales, slots=slots))
        yo, _, _ = oracle.state_update(held, host(conv)[[2, 0]], x, dt, A, Bt, Ct, Dv, zt, bias, True, w, wb)
        y = m.ssm_selective_state_update_cached(codes, scales, conv, g(x), g(dt), g(A), g(Bt), g(Ct), g(Dv),
                                                g(zt), g(bias), True, g(w), g(wb), slots=slots)
        check("y", host(y), yo, "f32")


def test_refusals():
    m = ssm()
    codes = torch.zeros(2, 4, 16, dtype=torch.int8, device="cuda")
    scales = torch.zeros(2, 4, device="cuda")
    state = torch.zeros(3, 4, 16, device="cuda")
    with pytest.raises(m.SSMError) as e:                   # three rows, two slots
        m.ssm_state_cache_write(state, codes, scales)
    assert e.value.name == "SSM_ERR_BAD_SHAPE"
    with pytest.raises(TypeError):
        m.ssm_state_cache_write(state[:2], codes.float(), scales)
    with pytest.raises(TypeError):
        m.ssm_state_cache_read(codes, scales, slots=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        m.ssm_state_cache_write(state[:2], codes, scales[:1])
    with pytest.raises(TypeError):
        m.ssm_checkpoint_pack(torch.zeros(1, 2, 3, dtype=torch.float16, device="cuda"))
    with pytest.raises(ValueError):
        m.ssm_checkpoint_pack(torch.zeros(1, 2, 3))
