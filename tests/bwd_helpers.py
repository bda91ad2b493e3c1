"""Inputs and tolerances of the backward-pass GPU tests.

Tolerances. The kernels compute in fp32, the reference in fp64. A decay a = 2^(delta A log2 e)
carries at most about 2^-22 of relative error (2 ulp of the exp, the rounding of its
argument), and a state collects it over its memory, 1 / (1 - a) steps: with the deltas drawn
here at most about 200 steps, 200 * 2^-22 = 5e-5. The sums over states, channels and steps
add less than 64 roundings of 2^-24 (4e-6). So fp32 gradients are held to 1e-4 of
max(|o|, rms(o)), the forward tests' rule; bf16 gradients add their own rounding, 2^-8 |o|.
"""
import numpy as np
import torch

from mamba_selective_scan_sm_b200.synth import round_bf16

F32_TOL, BF16_HALF_STEP = 1e-4, 2.0 ** -8
BF16_NAMES = ("du", "ddelta", "dz", "dB", "dC", "dx", "dconv_history")


def case(seed, dtype, B, D, L, N, heads=0, conv=0, z=True, skip=True, bias=True, h0=False,
         hist=False, dfinal=False):
    """numpy inputs, activations rounded to bf16 where dtype says so."""
    r = np.random.default_rng(seed)
    rnd = round_bf16 if dtype == "bf16" else (lambda v: v)
    act = lambda *s, std=1.0: rnd((std * r.standard_normal(s)).astype(np.float32))  # noqa: E731
    f32 = lambda *s, std=1.0: (std * r.standard_normal(s)).astype(np.float32)  # noqa: E731
    c = {"u": act(B, D, L), "delta": act(B, D, L, std=0.5), "B": act(B, N, L), "C": act(B, N, L),
         "dout": act(B, D, L), "z": act(B, D, L) if z else None, "D": f32(D) if skip else None}
    c["A"] = (-r.uniform(1, 16, heads) if heads else -r.uniform(0.5, 16, (D, N))).astype(np.float32)
    y = np.exp(r.uniform(np.log(5e-3), np.log(0.1), D))
    c["delta_bias"] = np.log(np.expm1(y)).astype(np.float32) if bias else None
    c["conv_w"] = f32(D, conv, std=0.5) if conv else None
    c["conv_b"] = f32(D, std=0.3) if conv else None
    c["h0"] = f32(B, D, N) if h0 else None
    c["hist"] = act(B, D, conv - 1) if hist else None
    c["dfinal"] = f32(B, D, N) if dfinal else None
    return c


def gpu(v, dtype, swap=False):
    """A CUDA tensor of an activation; swap: its last two axes exchanged (channel-last)."""
    if v is None:
        return None
    t = torch.from_numpy(np.ascontiguousarray(v)).cuda()
    t = t.transpose(1, 2).contiguous() if swap else t
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def host(t, swap=False):
    a = t.detach().float().cpu().numpy().astype(np.float64)
    return a.transpose(0, 2, 1) if swap else a


def check(name, got, want, dtype):
    assert got.shape == want.shape, name
    if not want.size:
        return
    assert np.all(np.isfinite(got)), f"{name}: not finite"
    rms = float(np.sqrt(np.mean(want ** 2)))
    err = np.abs(got - want)
    if dtype == "bf16" and name in BF16_NAMES:
        err = np.maximum(err - BF16_HALF_STEP * np.abs(want), 0.0)
    worst = float(np.max(err / np.maximum(np.maximum(np.abs(want), rms), 1e-30)))
    assert worst <= F32_TOL, f"{name}: {worst:.3e} > {F32_TOL}"
