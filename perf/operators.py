"""The operators for training a selective scan and for serving it from an 8-bit state cache,
each in its plain form (elementary torch operations, fp32) and as the library's calls.

* scan_bwd: the gradients of the selective scan (conv + SiLU, softplus delta, diagonal
  recurrence, readout, gate) with respect to every input, from the inputs alone or (packed8)
  from activations kept in 8 bits between the forward and the backward pass.
* conv_bwd: the gradients of the standalone causal conv + SiLU.
* pack: an activation packed to int8 with one scale per 64 positions of a channel, and read
  back.
* decode8: prompts' states written to an 8-bit state cache, decode steps on it, read back.
"""
import torch

own = False

BLOCK = 64                       # positions per scale of a packed activation
TINY = 2.0 ** -100               # a block or row whose largest magnitude is below this is zero
GOLDEN = 0x9E3779B9              # step of the rounding offsets within a state row


# ------------------------------------------------------------------------- cases --

def _scan(name, batch, dim, seqlen, dstate, dtype, conv=0, heads=0, z=True, states=False,
          reverse=False, channel_last=False, seqs=0, packed8=False):
    return {"name": name, "op": "scan_bwd", "batch": batch, "dim": dim, "seqlen": seqlen,
            "dstate": dstate, "dtype": dtype, "conv": conv, "heads": heads, "z": z,
            "states": states, "reverse": reverse, "channel_last": channel_last, "seqs": seqs,
            "packed8": packed8}


def listed():
    return [
        # one short sequence of a small fp32 block, where launch latency counts
        _scan("scan_bwd_tiny", 1, 64, 256, 16, "f32"),
        # a training step's layer of the 130M block: bf16, fused conv, gate
        _scan("scan_bwd_m130", 8, 1536, 2048, 16, "bf16", conv=4),
        # one long sequence of the 2.8B block, continued from a state, its last state used
        _scan("scan_bwd_long", 1, 5120, 16384, 16, "bf16", states=True),
        # A one scalar per head, d_state 128
        _scan("scan_bwd_heads128", 2, 1536, 2048, 128, "bf16", conv=4, heads=24),
        # documents of unequal length packed along one row, in the projections' own layout
        _scan("scan_bwd_packed_cl", 1, 1536, 32768, 16, "bf16", conv=4, channel_last=True, seqs=42),
        # the backward pass of a layer whose activations were kept in 8 bits
        _scan("scan_bwd_kept8", 4, 1536, 2048, 16, "bf16", conv=4, packed8=True),
        # the conv of that layer on its own
        {"name": "conv_bwd_m130", "op": "conv_bwd", "batch": 8, "dim": 1536, "seqlen": 2048,
         "width": 4, "silu": True, "bias": True, "dtype": "bf16"},
        # a small fp32 conv of odd sizes without SiLU
        {"name": "conv_bwd_odd", "op": "conv_bwd", "batch": 3, "dim": 101, "seqlen": 333,
         "width": 3, "silu": False, "bias": True, "dtype": "f32"},
        # one activation of the 130M layer kept in 8 bits and read back
        {"name": "pack_m130", "op": "pack", "batch": 8, "dim": 1536, "seqlen": 2048,
         "dtype": "bf16", "channel_last": False},
        # half of an in_proj output, odd length, in the projections' own layout
        {"name": "pack_cl_odd", "op": "pack", "batch": 2, "dim": 768, "seqlen": 1001,
         "dtype": "f32", "channel_last": True},
        # a full serving batch of the 2.8B block: prompts' states in, eight tokens, states back
        {"name": "decode8_b256", "op": "decode8", "batch": 256, "pad": 0, "dim": 5120, "dstate": 16,
         "heads": 0, "conv": 4, "steps": 8, "dtype": "bf16", "dither": True},
        # a few users of a per-head block, one token, the batch padded
        {"name": "decode8_small", "op": "decode8", "batch": 5, "pad": 2, "dim": 1536, "dstate": 128,
         "heads": 24, "conv": 4, "steps": 1, "dtype": "f32", "dither": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    kind = rng.choice(["scan_bwd", "scan_bwd", "scan_bwd", "conv_bwd", "pack", "decode8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if kind == "scan_bwd":
        packed = rng.random() < 0.25
        dstate = rng.choice([1, 5, 8, 16, 16, 16, 24, 64, 128])
        heads = 0 if packed or rng.random() < 0.6 else rng.choice([1, 3, 8])
        dim = _log(rng, 24, 2048)
        dim += -dim % heads if heads else 0
        batch = 1 if packed else _log(rng, 1, 8)
        seqlen = _log(rng, 1, max(1, min(16384, (1 << 28) // (batch * dim * max(dstate, 8)))))
        case = _scan("", batch, dim, seqlen, dstate, dtype, conv=rng.choice([0, 2, 3, 4, 4]),
                     heads=heads, z=rng.random() < 0.8,
                     channel_last=rng.random() < 0.4, packed8=rng.random() < 0.25)
        if packed:
            case["seqs"] = rng.randint(1, 9)
        elif rng.random() < 0.3:
            case["states"] = True
        elif rng.random() < 0.3:
            case["reverse"] = True
    elif kind == "conv_bwd":
        case = {"op": kind, "batch": _log(rng, 1, 8), "dim": _log(rng, 16, 2048),
                "seqlen": _log(rng, 1, 2048), "width": rng.randint(1, 4),
                "silu": rng.random() < 0.7, "bias": rng.random() < 0.7, "dtype": dtype}
    elif kind == "pack":
        case = {"op": kind, "batch": _log(rng, 1, 8), "dim": _log(rng, 16, 2048),
                "seqlen": _log(rng, 1, 2048), "dtype": dtype, "channel_last": rng.random() < 0.5}
    else:
        dstate = rng.choice([1, 12, 16, 16, 16, 48, 64, 128])
        heads = rng.choice([0, 0, 4, 8])
        dim = _log(rng, 32, 4096)
        dim += -dim % heads if heads else 0
        case = {"op": kind, "batch": _log(rng, 1, max(1, min(256, (1 << 24) // (dim * dstate)))),
                "pad": rng.choice([0, 0, 3]), "dim": dim, "dstate": dstate, "heads": heads,
                "conv": rng.choice([0, 2, 4, 4]), "steps": 1 if dtype == "f32" else rng.randint(1, 8),
                "dtype": dtype, "dither": rng.random() < 0.5}
    case.pop("name", None)
    return case


def work(case):
    es = 2 if case["dtype"] == "bf16" else 4
    b, d = case["batch"], case["dim"]
    if case["op"] == "scan_bwd":
        n, length = case["dstate"], case["seqlen"]
        kept = 1 + 4 / BLOCK if case["packed8"] else es
        streams = 3 if case["z"] else 2                         # u, delta(, z) and their gradients
        bytes_ = b * d * length * (streams * (kept + es) + es)  # and dout
        bytes_ += 4 * b * n * length * es                       # B, C and their gradients
        bytes_ += 8 * d * (n + 4 + case["conv"])                # parameters and their gradients
        # per (position, channel, state): a = exp(delta A), h, lambda, the two outer sums
        # (dB, dC), the three inner sums and dA
        return {"bytes": bytes_, "flops": 20 * b * d * length * n}
    if case["op"] == "conv_bwd":
        n = b * d * case["seqlen"]
        return {"bytes": 3 * n * es + 8 * d * (case["width"] + 1), "flops": n * (6 * case["width"] + 12)}
    if case["op"] == "pack":
        n = b * d * case["seqlen"]
        return {"bytes": n * (2 * es + 2 + 8 / BLOCK), "flops": 5 * n}
    n, t, w = case["dstate"], case["steps"], case["conv"]
    row = 4 * n + n + 4 + es * w * 2 + n + 4 + es * n           # write, conv state, read back
    row += t * (2 * (n + 4) + es * (4 + 2 * w) + (4 if case["dither"] else 0))
    return {"bytes": b * d * row + 4 * d * (n + 4 + w), "flops": b * d * (t * n * 12 + 4 * n)}


# ------------------------------------------------------------------------ inputs --

def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    t = _dtype(case)

    def normal(*shape, std=1.0, dtype=t):
        return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(*shape, generator=g, device="cuda") * (hi - lo) + lo

    f32 = torch.float32
    b, d = case["batch"], case["dim"]
    s = {"case": case}
    if case["op"] in ("scan_bwd", "decode8"):
        n = case["dstate"]
        s["A"] = (-uniform(case["heads"], lo=1.0, hi=16.0) if case["heads"] else
                  -torch.arange(1, n + 1, device="cuda", dtype=f32).repeat(d, 1).mul_(uniform(d, 1, lo=0.5, hi=1.5)))
        s["D"] = normal(d, dtype=f32)
        y = torch.exp(uniform(d, lo=-6.9, hi=-2.3))              # softplus(bias) in [1e-3, 0.1]
        s["bias"] = torch.log(torch.expm1(y))
        s["w"] = normal(d, case["conv"], std=0.5, dtype=f32) if case["conv"] else None
        s["cb"] = normal(d, std=0.1, dtype=f32) if case["conv"] else None
    if case["op"] == "scan_bwd":
        length, cl = case["seqlen"], case["channel_last"]
        if cl:                                                   # views of the projections
            xz, bc = normal(b, length, 2 * d), normal(b, length, 48 + 2 * n)
            s["u"], z = xz[..., :d], xz[..., d:]
            s["B"], s["C"] = bc[..., 48:48 + n], bc[..., 48 + n:]
            s["delta"], s["dout"] = normal(b, length, d, std=0.5), normal(b, length, d)
        else:
            s["u"], z = normal(b, d, length), normal(b, d, length)
            s["B"], s["C"] = normal(b, n, length), normal(b, n, length)
            s["delta"], s["dout"] = normal(b, d, length, std=0.5), normal(b, d, length)
        s["z"] = z if case["z"] else None
        s["h0"] = normal(b, d, n, dtype=f32) if case["states"] else None
        s["dhl"] = normal(b, d, n, dtype=f32) if case["states"] else None
        s["hist"] = normal(b, d, case["conv"] - 1) if case["states"] and case["conv"] > 1 else None
        s["starts"] = None
        if case["seqs"]:
            cuts = (uniform(case["seqs"] - 1) * (length + 1)).floor().clamp_(0, length).to(torch.int32)
            s["starts"] = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), cuts.sort().values,
                                     torch.full((1,), length, dtype=torch.int32, device="cuda")])
        if case["packed8"]:                                      # what the forward pass kept
            for k in ("u", "delta", "z"):
                if s[k] is not None:
                    s[k] = _keep8(s[k], cl)
    elif case["op"] == "conv_bwd":
        s["x"], s["dout"] = normal(b, d, case["seqlen"]), normal(b, d, case["seqlen"])
        s["w"] = normal(d, case["width"], std=0.5, dtype=f32)
        s["cb"] = normal(d, std=0.1, dtype=f32) if case["bias"] else None
    elif case["op"] == "pack":
        length = case["seqlen"]
        s["x"] = (normal(b, length, 2 * d)[..., :d] if case["channel_last"] else normal(b, d, length))
    else:
        live, rows, steps = b, b + case["pad"], case["steps"]
        slots = live + 3
        order = torch.randperm(slots, generator=g, device="cuda")[:live]
        s["live"] = order
        s["slots"] = torch.cat([order.to(torch.int32),
                                torch.full((case["pad"],), -1, dtype=torch.int32, device="cuda")])
        s["state"] = normal(rows, d, n, dtype=f32)
        s["conv0"] = normal(live, d, case["conv"]) if case["conv"] else None
        s["conv_state"] = torch.zeros(slots, d, case["conv"], dtype=t, device="cuda") if case["conv"] else None
        s["codes"] = torch.zeros(slots, d, n, dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(slots, d, device="cuda")
        for k, std in (("x", 1.0), ("dt", 0.5), ("z", 1.0)):
            s[k] = normal(steps, rows, d, std=std)
        s["B"], s["C"] = normal(steps, rows, n), normal(steps, rows, n)
        s["rand"] = (torch.randint(-2 ** 31, 2 ** 31, (steps + 1, rows, d), generator=g, device="cuda",
                                   dtype=torch.int64).to(torch.int32) if case["dither"] else None)
        s["out"] = torch.zeros(steps, rows, d, dtype=t, device="cuda")
        s["back"] = torch.zeros(rows, d, n, dtype=torch.bfloat16, device="cuda")
    return s


def _blocks(x, channel_last):
    """(batch, channel, block, 64) view of an activation, its last block filled with zeros."""
    x = x.transpose(1, 2) if channel_last else x
    pad = -x.shape[2] % BLOCK
    return torch.nn.functional.pad(x, (0, pad)).unflatten(2, (-1, BLOCK))


def _codes(x, rand=None):
    """int8 codes and fp32 scale of the last axis of fp32 values: code = round(127 x / max|x|),
    decided in fp64 (in fp32 a quotient next to a border would fall on either side of it)."""
    top = x.abs().amax(-1)
    zero = top < TINY
    scale = torch.where(zero, 0.0, top / 127.0)
    r = x.double() * 127.0 / torch.where(zero, 1.0, top.double()).unsqueeze(-1)
    r = torch.where(zero.unsqueeze(-1), 0.0, r)
    if rand is None:
        q = torch.round(r)
    else:                                                        # offset in [0, 1) per element
        k = torch.arange(x.shape[-1], device=x.device)
        bits = (rand.to(torch.int64).unsqueeze(-1) + k * GOLDEN) & 0xFFFFFFFF
        q = torch.floor(r + (bits >> 8).double() * 2.0 ** -24)
    return q.clamp(-127, 127).to(torch.int8), scale


def _keep8(x, channel_last):
    q, scale = _codes(_blocks(x.float(), channel_last))
    q = q.flatten(2)[..., :x.shape[1] if channel_last else x.shape[2]]
    return (q.transpose(1, 2).contiguous(), scale.transpose(1, 2).contiguous()) if channel_last else (q.contiguous(), scale)


def _read8(kept, channel_last, t):
    q, scale = kept
    q, scale = (q.transpose(1, 2), scale.transpose(1, 2)) if channel_last else (q, scale)
    v = q.to(t) * scale.to(t).repeat_interleave(BLOCK, 2)[..., :q.shape[2]]
    return v.transpose(1, 2) if channel_last else v


# --------------------------------------------------------------------------- runs --

def run(state):
    if own:
        import mamba_selective_scan_sm_b200 as ssm
        return {"scan_bwd": _own_scan, "conv_bwd": _own_conv, "pack": _own_pack,
                "decode8": _own_decode}[state["case"]["op"]](ssm, state)
    return {"scan_bwd": _plain_scan, "conv_bwd": _plain_conv, "pack": _plain_pack,
            "decode8": _plain_decode}[state["case"]["op"]](state)


def _own_scan(ssm, s):
    c = s["case"]
    u, delta, z = s["u"], s["delta"], s["z"]
    if c["packed8"]:
        u, delta, z = (None if k is None else ssm.Packed8(*k) for k in (u, delta, z))
    g = ssm.ssm_selective_scan_bwd(
        s["dout"], u, delta, s["A"], s["B"], s["C"], s["D"], z, s["bias"], True, c["reverse"],
        s["w"], s["cb"], dfinal_state=s["dhl"], initial_state=s["h0"], conv_history=s["hist"],
        seq_starts=s["starts"], channel_last=c["channel_last"])
    return {k: v for k, v in g._asdict().items() if v is not None}


def _own_conv(ssm, s):
    g = ssm.ssm_causal_conv1d_bwd(s["dout"], s["x"], s["w"], s["cb"], s["case"]["silu"])
    return {k: v for k, v in g._asdict().items() if v is not None}


def _own_pack(ssm, s):
    cl = s["case"]["channel_last"]
    kept = ssm.ssm_checkpoint_pack(s["x"], channel_last=cl)
    return {"values": ssm.ssm_checkpoint_unpack(kept, s["x"].dtype, channel_last=cl),
            "scales": kept.scales}


def _own_decode(ssm, s):
    c, rand = s["case"], s["rand"]
    ssm.ssm_state_cache_write(s["state"], s["codes"], s["scales"], slots=s["slots"],
                              rand=None if rand is None else rand[0])
    if c["conv"]:
        s["conv_state"].index_copy_(0, s["live"], s["conv0"])
    for t in range(c["steps"]):
        ssm.ssm_selective_state_update_cached(
            s["codes"], s["scales"], s["conv_state"], s["x"][t], s["dt"][t], s["A"], s["B"][t], s["C"][t],
            s["D"], s["z"][t], s["bias"], True, s["w"], s["cb"], slots=s["slots"],
            rand=None if rand is None else rand[t + 1], out=s["out"][t])
    ssm.ssm_state_cache_read(s["codes"], s["scales"], slots=s["slots"], out=s["back"])
    return {"out": s["out"], "state": s["back"], "conv_state": s["conv_state"]}


# -------------------------------------------------------------------- plain forms --

def _recur(a, b):
    """h_t = a_t h_{t-1} + b_t along axis 2 from zero, by doubling the span of each pair."""
    k, length = 1, b.shape[2]
    while k < length:
        b = torch.cat([b[:, :, :k], torch.addcmul(b[:, :, k:], a[:, :, k:], b[:, :, :-k])], 2)
        a = torch.cat([a[:, :, :k], a[:, :, k:] * a[:, :, :-k]], 2)
        k *= 2
    return b


def _windows(x, hist, width):
    """The conv's inputs (batch, channel, position, tap), zeros or the history before 0."""
    lead = hist if hist is not None else x.new_zeros(x.shape[0], x.shape[1], width - 1)
    return torch.cat([lead.to(x.dtype), x], 2).unfold(2, width, 1)


def _conv_grads(win, w, cb, keep, silu, du):
    """Gradients of act(cb + sum_k w_k x_{t-W+1+k}): of the padded input, the taps, the bias."""
    width = w.shape[1]
    win = win * keep if keep is not None else win
    if silu:
        pre = (win * w[:, None, :]).sum(-1) + (0.0 if cb is None else cb[:, None])
        sg = torch.sigmoid(pre)
        du = du * sg * (1 + pre * (1 - sg))
    g = du.unsqueeze(-1) * w[:, None, :]
    g = g * keep if keep is not None else g
    dxp = sum(torch.nn.functional.pad(g[..., k], (k, width - 1 - k)) for k in range(width))
    return dxp, (du.unsqueeze(-1) * win).sum((0, 2)), du.sum((0, 2))


def _starts(starts, length):
    """Position within its sequence, of each position of the packed row."""
    t = torch.arange(length, device=starts.device)
    begin = starts[torch.searchsorted(starts[:-1].contiguous(), t.to(torch.int32), right=True) - 1]
    return t - begin


def _plain_scan(s):
    c, f = s["case"], torch.float32
    t, n, cl = _dtype(c), c["dstate"], c["channel_last"]
    length = c["seqlen"]
    fwd = lambda v: v.flip(2) if c["reverse"] else v  # noqa: E731
    take = lambda v: None if v is None else fwd((v.transpose(1, 2) if cl else v).float())  # noqa: E731
    give = lambda v: (fwd(v).transpose(1, 2) if cl else fwd(v)).to(t)  # noqa: E731
    kept = {k: s[k] if s[k] is None or not c["packed8"] else _read8(s[k], cl, f) for k in ("u", "delta", "z")}
    x, dt, z, dy = (take(v) for v in (kept["u"], kept["delta"], kept["z"], s["dout"]))
    Bm, Cm = take(s["B"]).transpose(1, 2)[:, None], take(s["C"]).transpose(1, 2)[:, None]   # (b, 1, L, n)
    pos = None if s["starts"] is None else _starts(s["starts"], length)
    keep = None
    u = x
    if c["conv"]:
        width = c["conv"]
        win = _windows(x, s["hist"], width)
        if pos is not None:
            keep = (pos[:, None] >= width - 1 - torch.arange(width, device=pos.device)).to(f)
        pre = ((win * keep if keep is not None else win) * s["w"][:, None, :]).sum(-1) + s["cb"][:, None]
        u = pre * torch.sigmoid(pre)
    raw = dt + s["bias"][:, None]
    delta = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20.0))))
    A = s["A"].repeat_interleave(c["dim"] // c["heads"])[:, None].expand(-1, n) if c["heads"] else s["A"]
    a = torch.exp(delta.unsqueeze(-1) * A[:, None, :])           # (b, d, L, n)
    if pos is not None:
        a = a * (pos > 0).to(f)[:, None]
    bu = (delta * u).unsqueeze(-1) * Bm
    if s["h0"] is not None:
        bu[:, :, 0] += a[:, :, 0] * s["h0"]
    h = _recur(a, bu)
    y0 = (h * Cm).sum(-1) + s["D"][:, None] * u
    g, out = dy, {}
    if z is not None:
        sg = torch.sigmoid(z)
        g = dy * z * sg
        out["dz"] = give(dy * y0 * sg * (1 + z * (1 - sg)))
    out["dC"] = (g.unsqueeze(-1) * h).sum(1)
    src = g.unsqueeze(-1) * Cm
    if s["dhl"] is not None:
        src[:, :, -1] += s["dhl"]
    back = torch.cat([a[:, :, 1:], torch.zeros_like(a[:, :, :1])], 2).flip(2)   # a_{t+1}, backwards
    lam = _recur(back, src.flip(2)).flip(2)
    del src, back
    out["dB"] = (lam * (delta * u).unsqueeze(-1)).sum(1)
    inner = (lam * Bm).sum(-1)
    first = s["h0"].unsqueeze(2) if s["h0"] is not None else torch.zeros_like(h[:, :, :1])
    q = lam * a * torch.cat([first, h[:, :, :-1]], 2)
    if s["h0"] is not None:
        out["dinitial_state"] = lam[:, :, 0] * a[:, :, 0]
    ddelta = u * inner + (q * A[:, None, :]).sum(-1)
    dA = (q * delta.unsqueeze(-1)).sum((0, 2))
    out["dA"] = dA.reshape(c["heads"], -1).sum(1) if c["heads"] else dA
    ddt = ddelta * torch.sigmoid(raw)
    out["ddelta"], out["ddelta_bias"] = give(ddt), ddt.sum((0, 2))
    out["dD"] = (g * u).sum((0, 2))
    du = delta * inner + s["D"][:, None] * g
    if c["conv"]:
        dxp, out["dconv_weight"], out["dconv_bias"] = _conv_grads(win, s["w"], s["cb"], keep, True, du)
        du = dxp[..., c["conv"] - 1:]
        if s["hist"] is not None:
            out["dconv_history"] = dxp[..., :c["conv"] - 1].to(t)
    out["du"] = give(du)
    for k in ("dB", "dC"):
        v = fwd(out[k].transpose(1, 2))
        out[k] = (v.transpose(1, 2) if cl else v).to(t)
    return out


def _plain_conv(s):
    c = s["case"]
    win = _windows(s["x"].float(), None, c["width"])
    dxp, dw, db = _conv_grads(win, s["w"], s["cb"], None, c["silu"], s["dout"].float())
    out = {"dx": dxp[..., c["width"] - 1:].to(s["x"].dtype), "dw": dw}
    if s["cb"] is not None:
        out["dbias"] = db
    return out


def _plain_pack(s):
    cl = s["case"]["channel_last"]
    kept = _keep8(s["x"], cl)
    return {"values": _read8(kept, cl, torch.float32).to(s["x"].dtype), "scales": kept[1]}


def _plain_decode(s):
    c, rand, rows = s["case"], s["rand"], s["live"]
    live = c["batch"]
    n, w = c["dstate"], c["conv"]
    A = s["A"].repeat_interleave(c["dim"] // c["heads"])[:, None].expand(-1, n) if c["heads"] else s["A"]
    codes, scales = _codes(s["state"][:live], None if rand is None else rand[0, :live])
    if w:
        s["conv_state"].index_copy_(0, rows, s["conv0"])
    for t in range(c["steps"]):
        u = s["x"][t, :live].float()
        if w:
            win = torch.cat([s["conv_state"][rows][..., 1:], s["x"][t, :live].unsqueeze(-1)], -1)
            s["conv_state"].index_copy_(0, rows, win)
            pre = (win.float() * s["w"]).sum(-1) + s["cb"]
            u = pre * torch.sigmoid(pre)
        raw = s["dt"][t, :live].float() + s["bias"]
        delta = torch.where(raw > 20, raw, torch.log1p(torch.exp(raw.clamp(max=20.0))))
        h = torch.exp(delta.unsqueeze(-1) * A) * (codes * scales.unsqueeze(-1))
        h = h + (delta * u).unsqueeze(-1) * s["B"][t, :live, None].float()
        z = s["z"][t, :live].float()
        y = (h * s["C"][t, :live, None].float()).sum(-1) + s["D"] * u
        s["out"][t, :live] = (y * z * torch.sigmoid(z)).to(s["out"].dtype)
        codes, scales = _codes(h, None if rand is None else rand[t + 1, :live])
    s["codes"].index_copy_(0, rows, codes)
    s["scales"].index_copy_(0, rows, scales)
    s["back"][:live] = (codes * scales.unsqueeze(-1)).to(torch.bfloat16)
    return {"out": s["out"], "state": s["back"], "conv_state": s["conv_state"]}


# -------------------------------------------------------------- the definition, fp64 --

def exact(case, seed):
    s = prepare(case, seed)
    return {"scan_bwd": _exact_scan, "conv_bwd": _exact_conv, "pack": _exact_pack,
            "decode8": _exact_decode}[case["op"]](s)


def _exact_scan(s):
    """The recurrence one position after the other, then its adjoint backwards."""
    c, f = s["case"], torch.float64
    b, d, n, length, cl, w = c["batch"], c["dim"], c["dstate"], c["seqlen"], c["channel_last"], c["conv"]

    def steps(v, kept=False):                                    # (position, batch, channel)
        if v is None:
            return None
        v = _read8(v, cl, f) if kept else v.to(f)
        v = v.permute(1, 0, 2) if cl else v.permute(2, 0, 1)
        return v.flip(0) if c["reverse"] else v

    def back(v):
        v = v.flip(0) if c["reverse"] else v
        return v.permute(1, 0, 2) if cl else v.permute(1, 2, 0)

    x, dt, z = (steps(s[k], c["packed8"]) for k in ("u", "delta", "z"))
    dy, Bm, Cm = (steps(s[k]) for k in ("dout", "B", "C"))
    begin = [False] * length
    since = torch.arange(length, device=x.device) + (w if s["hist"] is not None or w == 0 else 0)
    if s["starts"] is not None:
        at = s["starts"].tolist()
        for i, j in zip(at[:-1], at[1:]):
            if j > i:
                begin[i] = True
                since[i:j] = torch.arange(j - i, device=x.device)
    u = x
    if w:
        taps, shifted = s["w"].to(f), []
        pre = s["cb"].to(f).expand(length, b, d).clone()
        for k in range(w):
            lag = w - 1 - k
            v = torch.zeros_like(x)
            v[lag:] = x[:length - lag] if lag else x
            if s["hist"] is not None and lag:
                m = min(lag, length)
                v[:m] = s["hist"].to(f).permute(2, 0, 1)[w - 1 - lag:w - 1 - lag + m]
            v = v * (since >= lag).to(f)[:, None, None]
            shifted.append(v)
            pre += taps[:, k] * v
        u = pre / (1 + torch.exp(-pre))
    raw = dt + s["bias"].to(f)
    delta = torch.nn.functional.relu(raw) + torch.log1p(torch.exp(-raw.abs()))
    A = s["A"].to(f)
    A = A.repeat_interleave(d // c["heads"])[:, None].expand(d, n) if c["heads"] else A
    g = dy if z is None else dy * z / (1 + torch.exp(-z))
    D = s["D"].to(f)
    zero = torch.zeros(b, d, n, dtype=f, device=x.device)
    start = zero if s["h0"] is None else s["h0"].to(f)
    hs, h = torch.empty(length, b, d, n, dtype=f, device=x.device), start
    y0 = torch.empty_like(dy)
    for i in range(length):
        h = zero if begin[i] else h
        h = torch.exp(delta[i].unsqueeze(-1) * A) * h + (delta[i] * u[i]).unsqueeze(-1) * Bm[i][:, None]
        hs[i] = h
        y0[i] = (h * Cm[i][:, None]).sum(-1) + D * u[i]
    lam = zero if s["dhl"] is None else s["dhl"].to(f)
    dB, dC = torch.empty_like(Bm), torch.empty_like(Cm)
    inner, through, dA = torch.empty_like(dy), torch.empty_like(dy), zero.clone()
    for i in range(length - 1, -1, -1):
        lam = lam + g[i].unsqueeze(-1) * Cm[i][:, None]
        dC[i] = (g[i].unsqueeze(-1) * hs[i]).sum(1)
        dB[i] = (lam * (delta[i] * u[i]).unsqueeze(-1)).sum(1)
        inner[i] = (lam * Bm[i][:, None]).sum(-1)
        before = zero if begin[i] else hs[i - 1] if i else start
        lam = lam * torch.exp(delta[i].unsqueeze(-1) * A) if not begin[i] else zero
        q = lam * before
        through[i] = (q * A).sum(-1)
        dA += q * delta[i].unsqueeze(-1)
    del hs
    out = {"dA": dA.sum(0)}
    if c["heads"]:
        out["dA"] = out["dA"].reshape(c["heads"], -1).sum(1)
    if s["h0"] is not None:
        out["dinitial_state"] = lam
    if z is not None:
        sg = 1 / (1 + torch.exp(-z))
        out["dz"] = back(dy * y0 * (sg + z * sg * (1 - sg)))
    du = delta * inner + D * g
    ddt = (u * inner + through) / (1 + torch.exp(-raw))
    out |= {"dB": back(dB), "dC": back(dC), "dD": (g * u).sum((0, 1)), "ddelta": back(ddt),
            "ddelta_bias": ddt.sum((0, 1))}
    if w:
        sg = 1 / (1 + torch.exp(-pre))
        dp = du * (sg + pre * sg * (1 - sg))
        out["dconv_bias"] = dp.sum((0, 1))
        out["dconv_weight"] = torch.stack([(dp * v).sum((0, 1)) for v in shifted], 1)
        wide = torch.zeros(length + w - 1, b, d, dtype=f, device=x.device)
        for k in range(w):
            wide[k:k + length] += taps[:, k] * dp * (since >= w - 1 - k).to(f)[:, None, None]
        du = wide[w - 1:]
        if s["hist"] is not None:
            out["dconv_history"] = wide[:w - 1].permute(1, 2, 0)
    out["du"] = back(du)
    return out


def _exact_conv(s):
    c, f = s["case"], torch.float64
    x, dy, w, width, length = s["x"].to(f), s["dout"].to(f), s["w"].to(f), c["width"], c["seqlen"]
    lead = torch.zeros(c["batch"], c["dim"], width - 1, dtype=f, device=x.device)
    xp = torch.cat([lead, x], 2)
    if c["silu"]:
        pre = sum(w[:, k, None] * xp[..., k:k + length] for k in range(width))
        pre = pre if s["cb"] is None else pre + s["cb"].to(f)[:, None]
        sg = 1 / (1 + torch.exp(-pre))
        dy = dy * (sg + pre * sg * (1 - sg))
    dxp = torch.zeros_like(xp)
    for k in range(width):
        dxp[..., k:k + length] += w[:, k, None] * dy
    out = {"dx": dxp[..., width - 1:],
           "dw": torch.stack([(dy * xp[..., k:k + length]).sum((0, 2)) for k in range(width)], 1)}
    if s["cb"] is not None:
        out["dbias"] = dy.sum((0, 2))
    return out


def _exact_pack(s):
    cl, x = s["case"]["channel_last"], s["x"].to(torch.float64)
    blocks = _blocks(x, cl)
    scale = blocks.abs().amax(-1) / 127
    v = torch.round(blocks / scale.clamp(min=1e-300).unsqueeze(-1)) * scale.unsqueeze(-1)
    v = v.flatten(2)[..., :s["case"]["seqlen"]]
    return {"values": v.transpose(1, 2) if cl else v, "scales": scale.transpose(1, 2) if cl else scale}


def _exact_decode(s):
    c, f, live, n, w = s["case"], torch.float64, s["case"]["batch"], s["case"]["dstate"], s["case"]["conv"]
    A = s["A"].to(f)
    A = A.repeat_interleave(c["dim"] // c["heads"])[:, None].expand(-1, n) if c["heads"] else A

    def stored(h, step):
        scale = h.abs().amax(-1, keepdim=True) / 127
        r = h / scale.clamp(min=1e-300)
        if s["rand"] is None:
            return torch.round(r) * scale
        k = torch.arange(n, device=h.device)
        bits = (s["rand"][step, :live].to(torch.int64).unsqueeze(-1) + k * GOLDEN) & 0xFFFFFFFF
        return torch.floor(r + (bits >> 8).to(f) / 2.0 ** 24).clamp(-127, 127) * scale

    h = stored(s["state"][:live].to(f), 0)
    window = None if w == 0 else s["conv0"].to(f)
    out = torch.zeros(s["out"].shape, dtype=f, device=h.device)
    for t in range(c["steps"]):
        u = s["x"][t, :live].to(f)
        if w:
            window = torch.cat([window[..., 1:], u.unsqueeze(-1)], -1)
            pre = (window * s["w"].to(f)).sum(-1) + s["cb"].to(f)
            u = pre / (1 + torch.exp(-pre))
        raw = s["dt"][t, :live].to(f) + s["bias"].to(f)
        delta = torch.nn.functional.relu(raw) + torch.log1p(torch.exp(-raw.abs()))
        h = torch.exp(delta.unsqueeze(-1) * A) * h + (delta * u).unsqueeze(-1) * s["B"][t, :live, None].to(f)
        z = s["z"][t, :live].to(f)
        out[t, :live] = ((h * s["C"][t, :live, None].to(f)).sum(-1) + s["D"].to(f) * u) * z / (1 + torch.exp(-z))
        h = stored(h, t + 1)
    state = torch.zeros(s["back"].shape, dtype=f, device=h.device)
    state[:live] = h
    conv = None
    if w:
        conv = s["conv_state"].to(f)
        conv[s["live"]] = window
    return {"out": out, "state": state, "conv_state": conv}
