"""Padded rows of a call on the 8-bit state cache (a slot outside the cache) are not used: whatever
stands in their places, NaN or rounding bits or nothing finite, the other rows keep their bits and
the padded rows' outputs theirs."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def ssm():
    import mamba_selective_scan_sm_b200 as m
    return m


@pytest.mark.parametrize("random", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dim,n,conv", [(33, 16, 4), (5, 13, 2), (7, 64, 0), (130, 128, 4), (64, 3, 3)])
def test_padded_rows(dim, n, conv, dtype, random):
    m = ssm()
    g = torch.Generator(device="cuda").manual_seed(1)
    r = lambda *s, t=torch.float32: torch.randn(*s, generator=g, device="cuda").to(t)  # noqa: E731
    order = [4, -1, 0, 6, 2, 6, -7]                        # 6 slots: rows 1, 3, 5, 6 are padding
    live = [0, 2, 4]
    slots = torch.tensor(order, dtype=torch.int32, device="cuda")
    B = len(order)
    state, A, D, w = r(B, dim, n), -r(dim, n).abs(), r(dim), r(dim, conv) if conv else None
    x, dt, z = (r(B, dim, t=dtype) for _ in range(3))
    Bt, Ct = r(B, n, t=dtype), r(B, n, t=dtype)
    rand = torch.randint(-2 ** 31, 2 ** 31, (B, dim), generator=g, device="cuda", dtype=torch.int64).to(torch.int32)
    conv0 = r(6, dim, conv, t=dtype) if conv else None

    def tokens(spoil):
        def put(v, bad):
            v = v.clone()
            if spoil:
                v[[i for i in range(B) if i not in live]] = bad
            return v
        nan = float("nan")
        codes, scales = torch.full((6, dim, n), 3, dtype=torch.int8, device="cuda"), torch.ones(6, dim, device="cuda")
        cs = conv0.clone() if conv else None
        bits = put(rand, -1) if random else None
        out = torch.full((B, dim), 7.0, dtype=dtype, device="cuda")
        m.ssm_state_cache_write(put(state, nan), codes, scales, slots=slots, rand=bits)
        for _ in range(2):
            m.ssm_selective_state_update_cached(codes, scales, cs, put(x, nan), put(dt, nan), A, put(Bt, nan),
                                                put(Ct, nan), D, put(z, nan), None, True, w, None, slots=slots,
                                                rand=bits, out=out)
        return [codes, scales, out] + ([cs] if conv else [])
    want, got = tokens(False), tokens(True)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    codes, scales, out = got[:3]
    assert torch.all(out[[1, 3, 5, 6]] == 7.0) and torch.isfinite(out[live].float()).all()
    for slot in (1, 3, 5):
        assert torch.all(codes[slot] == 3) and torch.all(scales[slot] == 1.0)
        assert not conv or torch.equal(got[3][slot], conv0[slot])
