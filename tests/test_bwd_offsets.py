"""Offsets of packed sequences that are out of order or out of range: the scan's gradient gives
that of the cuts they come down to, and touches nothing beside its tensors."""
import numpy as np
import pytest
import torch

from tests import bwd_reference as ref
from tests.bwd_helpers import case, check, gpu, host
from tests.test_gpu_scan_bwd import ssm

L = 80


def since(starts, length):
    """Per position the steps since the start it is given, 0..4: the last of the offsets at or
    before it by a binary search (which needs them in order to mean more than that)."""
    out = np.zeros(length, dtype=int)
    for t in range(length):
        lo, hi = 0, len(starts) - 1
        while hi - lo > 1:
            m = (lo + hi) // 2
            lo, hi = (m, hi) if starts[m] <= t else (lo, m)
        out[t] = min(max(t - starts[lo], 0), 4)
    return out


def cuts(starts, length):
    """Well-formed offsets with the same cuts, if there are any: a start wherever no step lies
    behind; and whether the conv's reach agrees with them."""
    s = since(starts, length)
    at = [int(t) for t in np.flatnonzero(s == 0)]
    clean = [0] + [t for t in at if t > 0] + [length]
    return clean, np.array_equal(since(clean, length), s)


BAD = [[0, 30, 10, 80], [0, 1000000, -7, 80], [0, 50, 20, 60, 80], [0, 40, 40, 39, 80], [0, 10, 2000000000, 80],
       [-5, 2000000000, 3], [5, 9, 80], [0, 40], [0, 16, 32, 16, 48, 80]]


@pytest.mark.parametrize("starts", BAD)
def test_cuts_restated(starts):
    s = since(starts, L)
    assert s.min() >= 0 and s.max() <= 4


@pytest.mark.gpu
@pytest.mark.parametrize("cl", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("segments", [1, 3])
@pytest.mark.parametrize("starts", BAD)
def test_bad_offsets(starts, segments, dtype, cl):
    m, B, D, N, lead = ssm(), 1, 48, 16, 512
    c = case(50, dtype, B, D, L, N, conv=4)
    el = torch.float32 if dtype == "f32" else torch.bfloat16
    bufs = []

    def guarded(n, kind, fill):
        b = torch.full((n + 2 * lead,), fill, dtype=kind, device="cuda")
        bufs.append((b, n, fill))
        return b[lead:lead + n]

    shape, bc = ((B, L, D), (B, L, N)) if cl else ((B, D, L), (B, N, L))
    outs = {k: guarded(D * L, el, 7).view(shape) for k in ("du", "ddelta", "dz")}
    outs |= {k: guarded(N * L, el, 7).view(bc) for k in ("dB", "dC")}
    need = m.ssm_selective_scan_bwd_workspace_size(B, D, L, N, el, conv_width=4, packed_sequences=True,
                                                   channel_last=cl, num_segments=segments)
    ws = guarded(need, torch.uint8, 7)
    st = guarded(len(starts), torch.int32, 7)
    st.copy_(torch.tensor(starts, dtype=torch.int32))
    t = lambda k: gpu(c[k], dtype, cl)  # noqa: E731
    f = lambda k: gpu(c[k], "f32")  # noqa: E731
    g = m.ssm_selective_scan_bwd(t("dout"), t("u"), t("delta"), f("A"), t("B"), t("C"), f("D"), t("z"),
                                 f("delta_bias"), True, False, f("conv_w"), f("conv_b"), seq_starts=st,
                                 channel_last=cl, num_segments=segments, workspace=ws, **outs)
    for b, n, fill in bufs:
        assert torch.all(b[:lead] == fill) and torch.all(b[lead + n:] == fill)
    assert st.tolist() == starts
    clean, same = cuts(starts, L)
    if same:
        want = ref.scan_grads(c["dout"], c["u"], c["delta"], c["A"], c["B"], c["C"], c["D"], c["z"], c["delta_bias"],
                              True, False, c["conv_w"], c["conv_b"], starts=clean)
        for k, o in want.items():
            check(k, host(getattr(g, k), cl and k in ("du", "ddelta", "dz", "dB", "dC")), o, dtype)


def test_some_of_these_have_well_formed_cuts():
    assert sum(cuts(s, L)[1] for s in BAD) >= 4
