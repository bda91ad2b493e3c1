"""The gradients of the selective scan and of the causal conv in numpy, double precision, one
position after the other: what the GPU tests of the backward pass compare with. Written from
the formulas alone; ``test_bwd_reference.py`` holds it against central differences of the
forward oracle. Arrays are (batch, dim, seqlen) / (batch, dstate, seqlen)."""
import numpy as np


def _silu(v):
    return v / (1.0 + np.exp(-v))


def _dsilu(v):
    s = 1.0 / (1.0 + np.exp(-v))
    return s * (1.0 + v * (1.0 - s))


def conv_grads(dout, x, w, bias=None, silu=True, hist=None, starts=None):
    """(dx, dw, dbias, dhist) of act(bias + sum_k w_k x_{t-W+1+k}); ``starts``: offsets of
    packed sequences, before each of which the conv reads nothing."""
    dout, x, w = (np.asarray(v, dtype=np.float64) for v in (dout, x, w))
    B, D, L = x.shape
    W = w.shape[1]
    lead = np.zeros((B, D, W - 1)) if hist is None else np.asarray(hist, dtype=np.float64)
    xp = np.concatenate([lead, x], 2)
    dxp, dw, db = np.zeros_like(xp), np.zeros_like(w), np.zeros(D)
    begin = begins(starts, L)
    for t in range(L):
        taps = [k for k in range(W) if starts is None or t - (W - 1 - k) >= begin[t]]
        pre = np.zeros((B, D)) + (0.0 if bias is None else np.asarray(bias, dtype=np.float64))
        for k in taps:
            pre = pre + w[:, k] * xp[:, :, t + k]
        dp = dout[:, :, t] * (_dsilu(pre) if silu else 1.0)
        db += dp.sum(0)
        for k in taps:
            dxp[:, :, t + k] += w[:, k] * dp
            dw[:, k] += (dp * xp[:, :, t + k]).sum(0)
    return dxp[:, :, W - 1:], dw, db, dxp[:, :, :W - 1]


def begins(starts, L):
    """Per position, where its sequence begins."""
    if starts is None:
        return np.zeros(L, dtype=int)
    out = np.zeros(L, dtype=int)
    for i, j in zip(starts[:-1], starts[1:]):
        out[i:j] = i
    return out


def scan_grads(dout, u, delta, A, B, C, D=None, z=None, delta_bias=None, softplus=True,
               reverse=False, conv_w=None, conv_b=None, dfinal=None, h0=None, hist=None,
               starts=None):
    """Gradients of the selective scan by name, from its inputs. A (dim, dstate) or (heads,)."""
    f = lambda v: None if v is None else np.asarray(v, dtype=np.float64)  # noqa: E731
    dout, u, delta, A, B, C, D, z, delta_bias, conv_w, conv_b, dfinal, h0, hist = map(
        f, (dout, u, delta, A, B, C, D, z, delta_bias, conv_w, conv_b, dfinal, h0, hist))
    flip = (lambda v: v[:, :, ::-1]) if reverse else (lambda v: v)
    dout, x, delta, B, C = (flip(v) for v in (dout, u, delta, B, C))
    z = None if z is None else flip(z)
    nb, dim, L = x.shape
    N = B.shape[1]
    An = np.repeat(A, dim // A.shape[0])[:, None] * np.ones(N) if A.ndim == 1 else A
    begin = begins(starts, L)
    if conv_w is not None:
        W = conv_w.shape[1]
        lead = np.zeros((nb, dim, W - 1)) if hist is None else hist
        xp = np.concatenate([lead, x], 2)
        pre = np.zeros_like(x)
        for t in range(L):
            for k in range(W):
                if starts is None or t - (W - 1 - k) >= begin[t]:
                    pre[:, :, t] += conv_w[:, k] * xp[:, :, t + k]
        pre += 0.0 if conv_b is None else conv_b[:, None]
        x_in, x = x, _silu(pre)
    raw = delta + (0.0 if delta_bias is None else delta_bias[:, None])
    dl = np.logaddexp(0.0, raw) if softplus else raw
    sig = 1.0 / (1.0 + np.exp(-raw)) if softplus else np.ones_like(raw)
    Dv = np.zeros(dim) if D is None else D
    zero = np.zeros((nb, dim, N))
    first = zero if h0 is None else h0
    hs = np.zeros((L, nb, dim, N))
    h = first
    for t in range(L):
        if starts is not None and begin[t] == t:
            h = zero
        h = np.exp(dl[:, :, t, None] * An) * h + (dl[:, :, t] * x[:, :, t])[..., None] * B[:, None, :, t]
        hs[t] = h
    y0 = np.einsum("tbdn,bnt->bdt", hs, C) + Dv[:, None] * x
    g = dout if z is None else dout * _silu(z)
    out = {} if z is None else {"dz": flip(dout * y0 * _dsilu(z))}
    lam = zero.copy() if dfinal is None else dfinal.copy()
    dB, dC, dx, ddl, dA = np.zeros_like(B), np.zeros_like(C), np.zeros_like(x), np.zeros_like(x), zero.copy()
    for t in range(L - 1, -1, -1):
        lam = lam + g[:, :, t, None] * C[:, None, :, t]
        dC[:, :, t] = (g[:, :, t, None] * hs[t]).sum(1)
        dB[:, :, t] = (lam * (dl[:, :, t] * x[:, :, t])[..., None]).sum(1)
        inner = (lam * B[:, None, :, t]).sum(2)
        begins_here = starts is not None and begin[t] == t
        prev = zero if begins_here else (hs[t - 1] if t else first)
        lam = zero if begins_here else lam * np.exp(dl[:, :, t, None] * An)
        q = lam * prev
        dx[:, :, t] = dl[:, :, t] * inner + Dv * g[:, :, t]
        ddl[:, :, t] = x[:, :, t] * inner + (q * An).sum(2)
        dA += q * dl[:, :, t, None]
    ddt = ddl * sig
    dA = dA.sum(0)
    out.update(dB=flip(dB), dC=flip(dC), ddelta=flip(ddt),
               dA=dA if A.ndim == 2 else dA.reshape(A.shape[0], -1).sum(1))
    if D is not None:
        out["dD"] = (g * x).sum((0, 2))
    if delta_bias is not None:
        out["ddelta_bias"] = ddt.sum((0, 2))
    if h0 is not None:
        out["dinitial_state"] = lam
    if conv_w is not None:
        dx, dw, db, dh = conv_grads(dx, x_in, conv_w, conv_b, True, hist, starts)
        out["dconv_weight"] = dw
        if conv_b is not None:
            out["dconv_bias"] = db
        if hist is not None:
            out["dconv_history"] = dh
    out["du"] = flip(dx)
    return out


def pack_reference(x, axis=-1):
    """(codes, scales) of an fp32 array along ``axis``, decided exactly: 127 x / max|x| rounded
    to the nearest integer, ties to even, in rational arithmetic."""
    from fractions import Fraction
    x = np.moveaxis(np.asarray(x, dtype=np.float32), axis, -1)
    flat = x.reshape(-1, x.shape[-1])
    codes, scales = np.zeros(flat.shape, dtype=np.int8), np.zeros(len(flat), dtype=np.float32)
    for i, row in enumerate(flat):
        if not np.all(np.isfinite(row)):
            scales[i] = np.nan
            continue
        top = np.max(np.abs(row)) if row.size else np.float32(0)
        if top < 2.0 ** -100:
            continue
        scales[i] = top / np.float32(127.0)
        codes[i] = [round(Fraction(float(v)) * 127 / Fraction(float(top))) for v in row]
    return np.moveaxis(codes.reshape(x.shape), -1, axis), scales.reshape(x.shape[:-1])
