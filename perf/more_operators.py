"""Measured cases of what the decoder stack adds to keep its activations in 8 bits between the forward and the backward:
the checkpoint format itself (act8_quantize, act8_dequantize), the SiLU product with checkpoints of its inputs
(silu_mul_fwd_act8, silu_mul_act8, silu_mul_bwd_act8), the LoRA linear's backward from a checkpoint
(lora_linear_bwd_act8, lora_linear_bwd_bf16_act8), and the residual add fused with the norms around a block, its gate
and its scale, forward and backward (residual_norm_fwd, residual_norm_bwd).

Where ``own`` is false, ``run`` computes the plain form in torch; where it is true, the framework's kernels. ``exact``
gives the same outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
RANK, ALPHA = 16, 32.0
# hidden, query, kv and intermediate widths of the stacks this repository measures
WIDTHS = {"tiny": (128, 128, 32, 256), "7b": (3584, 3584, 512, 18944), "32b": (5120, 5120, 1024, 27648),
          "72b": (8192, 8192, 1024, 29568)}


def _proj(stack, proj):
    """(N, K) of a projection."""
    h, q, kv, i = WIDTHS[stack]
    return {"q": (q, h), "k": (kv, h), "v": (kv, h), "o": (h, q), "gate": (i, h), "up": (i, h), "down": (h, i)}[proj]


def _named(name, case):
    return dict(case, name=name) if name else case


def _act8(name, t, c):
    return _named(name, {"op": "act8", "t": t, "c": c})


def _mlp(name, t, f):
    return _named(name, {"op": "mlp", "t": t, "c": f})


def _linear(name, stack, proj, t, dense=False):
    n, k = _proj(stack, proj)
    return _named(name, {"op": "linear", "t": t, "n": n, "k": k, "dense": dense})


def _norm(name, op, t, h, block, post=False, gate="none", scale=1.0, gain=False, offset=0.0, act8=False, dns=1):
    """block: whether a block's output is added; act8: the forward writes the checkpoint of n, or the backward reads it."""
    return _named(name, {"op": op, "t": t, "c": h, "block": block, "post": post, "gate": gate, "scale": scale,
                         "gain": gain, "offset": offset, "act8": act8, "dns": dns})


def listed():
    return [
        # one token's normalised row, written and read back: latency alone
        _act8("act8_7b_1", 1, 3584),
        # the widest activation of a long sequence
        _act8("act8_72b_8192", 8192, 29568),
        # the small stack that the tests drive
        _mlp("mlp_tiny_40", 40, 256),
        # the layer benchmark's tokens: the MLP activation of an ordinary step, forward, rebuilt, backward
        _mlp("mlp_7b_512", 512, 18944),
        # a long sequence on the 72B widths
        _mlp("mlp_72b_8192", 8192, 29568),
        # a few odd rows of a width that no vector load fits
        _norm("norm_fwd_odd_33", "norm_fwd", 33, 1001, True, gain=True),
        # everything at once on a long sequence: norms on both sides, a gate a channel, a scaled branch, the checkpoint
        _norm("norm_fwd_72b_8192", "norm_fwd", 8192, 8192, True, True, "channel", 0.5, True, 1.0, act8=True),
        # the stack's own backward of its second norm: two projections' gradients, n from its checkpoint
        _norm("norm_bwd_7b_512", "norm_bwd", 512, 3584, False, act8=True, dns=2),
        # trained gains and a gate a token, ragged length
        _norm("norm_bwd_32b_2731", "norm_bwd", 2731, 5120, True, True, "token", 0.25, True, dns=3),
        # one token through the query projection's backward: latency and the weight's bytes
        _linear("linear_7b_q_1", "7b", "q", 1),
        # the layer benchmark's largest projection
        _linear("linear_7b_gate_512", "7b", "gate", 512),
        # a ragged batch through the dense base
        _linear("linear_32b_q_1291_dense", "32b", "q", 1291, True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["act8", "mlp", "mlp", "linear", "linear", "norm_fwd", "norm_fwd", "norm_bwd", "norm_bwd"])
    t = _log_int(rng, 1, 8192)
    if op in ("act8", "mlp"):
        return {"act8": _act8, "mlp": _mlp}[op](None, t, 64 * _log_int(rng, 1, 462))
    if op == "linear":
        stack = rng.choice(["tiny", "7b", "7b", "32b"])
        proj = rng.choice(["q", "k", "o", "gate", "down"])
        n, k = _proj(stack, proj)
        most = min(2048, int(512 * 18944 * 3584 / (n * k)))  # no more work than the largest listed projection
        return _linear(None, stack, proj, _log_int(rng, 1, max(1, most)), rng.random() < 0.3)
    h = rng.choice([128, 3584, 5120, 8192, 64 * _log_int(rng, 1, 128), _log_int(rng, 32, 8192)])
    block = rng.random() < 0.75
    post, gate = block and rng.random() < 0.5, rng.choice(["none", "channel", "token"]) if block else "none"
    scale = rng.choice([1.0, 0.5, 0.22]) if block else 1.0
    gain = rng.random() < 0.6
    act8 = h % 64 == 0 and rng.random() < 0.5 and (op == "norm_fwd" or not gain)
    return _norm(None, op, t, h, block, post, gate, scale, gain, rng.choice([0.0, 1.0]) if gain or post else 0.0, act8,
                 rng.choice([1, 2, 3]) if op == "norm_bwd" else 1)


# ------------------------------------------------------------------ the formats, in torch

def _quantized(x):
    """x [T, C] -> (codes uint8 [T, C], scale float32 [T, C / 64])."""
    b = x.float().view(x.shape[0], -1, 64)
    top = b.abs().amax(-1, keepdim=True)
    small = torch.where(top < 2.0 ** -64, 2.0 ** 64, 1.0)
    inv = torch.where(top > 0, 127.0 / (top * small), torch.zeros_like(top))
    # a product next to a half has to be whole: 8 and 24 bits of significand
    codes = ((b * small).double() * inv.double()).round_() + 128.0
    scale = top / 127.0
    bad = ~torch.isfinite(b).all(-1, keepdim=True)
    codes = torch.where(bad, 128.0, codes).to(torch.uint8)
    return codes.view(x.shape), torch.where(bad, math.nan, scale).squeeze(-1)


def _values(codes, scale):
    """What a checkpoint stands for, float32 [T, C]."""
    b = codes.view(codes.shape[0], -1, 64).float() - 128.0
    return (b * scale.unsqueeze(-1)).view(codes.shape)


def _levels(device):
    """The 16 levels of the 4-bit base: normal quantiles on two even grids, scaled to [-1, 1]."""
    edge = ((1 - 1 / 30) + (1 - 1 / 32)) / 2
    p = [edge - (edge - 0.5) * i / 8 for i in range(8)] + [0.5]
    m = [edge - (edge - 0.5) * i / 7 for i in range(7)]

    def quantile(v):
        return torch.erfinv(2 * torch.tensor(v, dtype=F64) - 1)

    up, down = quantile(p), -quantile(m)
    return (torch.cat([down, up.flip(0)]) / up[0]).to(device)


def _base(w):
    """A bf16 weight [N, K] as the 4-bit base: packed codes uint8 [N, K / 2], absmax float32 [N, K / 64]."""
    levels = _levels(w.device)
    mid = ((levels[1:] + levels[:-1]) / 2).float()
    b = w.float().view(-1, 64)
    top = b.abs().amax(-1, keepdim=True)
    codes = torch.bucketize((b / top).view(-1, 2), mid, out_int32=True).to(torch.uint8)
    return (codes[:, 0] | (codes[:, 1] << 4)).view(w.shape[0], -1), top.view(w.shape[0], -1)


def _base_values(codes, absmax):
    levels = _levels(codes.device).float()
    c = torch.stack([codes & 15, codes >> 4], -1).view(codes.shape[0], -1, 64)
    return (levels[c.int()] * absmax.unsqueeze(-1)).view(codes.shape[0], -1).to(BF16)


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)

    def empty(*shape, dtype=BF16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def spread(c):
        """Channels of trained networks differ in size."""
        return torch.exp(0.7 * torch.randn(c, generator=g, device="cuda"))

    op, t = case["op"], case["t"]
    s = {"case": case}
    if op == "linear":
        n, k, r = case["n"], case["k"], RANK
        w = normal(n, k, std=0.02)
        x = normal(t, k)
        s["A"] = ((torch.rand(r, k, generator=g, device="cuda") * 2 - 1) / k ** 0.5).to(BF16)
        s["B"] = normal(n, r, std=0.01)
        s["u"] = x.float() @ s["A"].float().t()
        s["dy"] = normal(t, n, std=0.05)
        s["x8"], s["x8s"] = _quantized(x)
        if case["dense"]:
            s["w"] = w
        else:
            s["codes"], s["absmax"] = _base(w)
        s.update(dx=empty(t, k), dA=empty(r, k, dtype=F32), dB=empty(n, r, dtype=F32))
        return s
    c = case["c"]
    if op == "act8":
        s.update(x=(torch.randn(t, c, generator=g, device="cuda") * spread(c)).to(BF16), out=empty(t, c))
        s.update(codes=empty(t, c, dtype=torch.uint8), scale=empty(t, c // 64, dtype=F32))
        return s
    if op == "mlp":
        s.update(gate=normal(t, c, std=1.5), up=normal(t, c), dm=normal(t, c, std=0.02))
        s.update({n: empty(t, c) for n in ("m", "m_again", "dgate", "dup")})
        for n in ("gate8", "up8"):
            s[n], s[n + "s"] = empty(t, c, dtype=torch.uint8), empty(t, c // 64, dtype=F32)
        return s
    s["h"] = (torch.randn(t, c, generator=g, device="cuda") * spread(c)).to(BF16)
    s["o"] = normal(t, c, std=1.5) if case["block"] else None
    # with an offset of 1 the trained gains lie around 0
    s["post_gain"] = (normal(c, std=0.2) + (1 - case["offset"])).to(BF16) if case["post"] else None
    s["gain"] = (normal(c, std=0.2) + (1 - case["offset"])).to(BF16) if case["gain"] else None
    s["gate"] = {"none": None, "channel": (c,), "token": (t, c)}[case["gate"]]
    if s["gate"]:
        s["gate"] = normal(*s["gate"], std=0.7)
    if op == "norm_fwd":
        s.update(h_out=empty(t, c) if case["block"] else None, n=empty(t, c))
        if case["act8"]:
            s.update(n8=empty(t, c, dtype=torch.uint8), n8s=empty(t, c // 64, dtype=F32), n_back=empty(t, c))
        return s
    s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + 1e-6)
    if case["post"]:
        s["rstd_o"] = torch.rsqrt(s["o"].float().square().mean(-1) + 1e-6)
    if case["act8"]:
        s["n8"], s["n8s"] = _quantized((s["h"].float() * s["rstd"][:, None]).to(BF16))
    s["dn"] = [normal(t, c, std=0.05) for _ in range(case["dns"])]
    s["dres"] = normal(t, c, std=0.05)
    return s


# ------------------------------------------------------------------ plain forms, in 32 bits

def _plain_act8(s):
    return _values(*_quantized(s["x"])).to(BF16)


def _plain_mlp(s):
    gate, up = s["gate"].float(), s["up"].float()
    m = (gate / (1 + torch.exp(-gate)) * up).to(BF16)
    gate, up = _values(*_quantized(s["gate"])), _values(*_quantized(s["up"]))
    sig = 1 / (1 + torch.exp(-gate))
    silu = gate * sig
    dm = s["dm"].float()
    return {"m": m, "m_again": (silu * up).to(BF16),
            "dgate": (dm * up * sig * (1 + gate * (1 - sig))).to(BF16), "dup": (dm * silu).to(BF16)}


def _plain_linear(s):
    c, f = s["case"], ALPHA / RANK
    w = (s["w"] if c["dense"] else _base_values(s["codes"], s["absmax"])).float()
    x = _values(s["x8"], s["x8s"]).to(BF16).float()
    dy, a, b = s["dy"].float(), s["A"].float(), s["B"].float()
    g = dy @ b
    return {"dx": (dy @ w + f * (g @ a)).to(BF16), "dA": f * (g.t() @ x), "dB": f * (dy.t() @ s["u"])}


def _gain(s, name):
    return 1.0 if s[name] is None else s[name].float() + s["case"]["offset"]


def _plain_norm_fwd(s):
    c = s["case"]
    x, out = s["h"].float(), {}
    if c["block"]:
        v = s["o"].float()
        if c["post"]:
            out["rstd_o"] = torch.rsqrt(v.square().mean(-1) + 1e-6)
            v = v * out["rstd_o"][:, None] * _gain(s, "post_gain")
        x = x + c["scale"] * (v if s["gate"] is None else s["gate"].float() * v)
        out["h"] = x.to(BF16)
    out["rstd"] = torch.rsqrt(x.square().mean(-1) + 1e-6)
    out["n"] = (x * out["rstd"][:, None] * _gain(s, "gain")).to(BF16)
    if c["act8"]:
        out["n_back"] = _values(*_quantized(out["n"])).to(BF16)
    return out


def _plain_norm_bwd(s):
    c = s["case"]
    rstd = s["rstd"][:, None]
    b = _values(s["n8"], s["n8s"]) if c["act8"] else s["h"].float() * rstd
    g = sum(d.float() for d in s["dn"])
    w = g * _gain(s, "gain")
    ds = s["dres"].float() + rstd * (w - b * (w * b).mean(-1, keepdim=True))
    out = {"dh": ds.to(BF16)}
    if c["gain"]:
        out["dgain"] = (g * b).sum(0)
    if not c["block"]:
        return out
    unit = s["o"].float() * (s["rstd_o"][:, None] if c["post"] else 1.0)
    v = unit * _gain(s, "post_gain")
    dv = c["scale"] * ds
    if s["gate"] is not None:
        dgate = dv * v
        out["dgate"] = dgate.sum(0) if c["gate"] == "channel" else dgate.to(BF16)
        dv = dv * s["gate"].float()
    if c["post"]:
        out["dpost_gain"] = (dv * unit).sum(0)
        p = dv * _gain(s, "post_gain")
        dv = s["rstd_o"][:, None] * (p - unit * (p * unit).mean(-1, keepdim=True))
    out["do"] = dv.to(BF16)
    return out


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"act8": _plain_act8, "mlp": _plain_mlp, "linear": _plain_linear, "norm_fwd": _plain_norm_fwd,
                "norm_bwd": _plain_norm_bwd}[op](s)
    from nf4_weight_streamed_amd import lib
    if op == "act8":
        return lib.act8_dequantize(lib.act8_quantize(s["x"], out=lib.Act8(s["codes"], s["scale"])), out=s["out"])
    if op == "mlp":
        gate8, up8 = lib.Act8(s["gate8"], s["gate8s"]), lib.Act8(s["up8"], s["up8s"])
        lib.silu_mul_fwd_act8(s["gate"], s["up"], out=s["m"], gate8=gate8, up8=up8)
        lib.silu_mul_act8(gate8, up8, out=s["m_again"])
        lib.silu_mul_bwd_act8(gate8, up8, s["dm"], dgate=s["dgate"], dup=s["dup"])
        return {n: s[n] for n in ("m", "m_again", "dgate", "dup")}
    if op == "linear":
        x8, to = lib.Act8(s["x8"], s["x8s"]), {n: s[n] for n in ("dx", "dA", "dB")}
        if c["dense"]:
            lib.lora_linear_bwd_bf16_act8(s["w"], x8, s["u"], s["dy"], s["A"], s["B"], ALPHA, **to)
        else:
            lib.lora_linear_bwd_act8(s["codes"], s["absmax"], x8, s["u"], s["dy"], s["A"], s["B"], ALPHA, **to)
        return to
    if op == "norm_fwd":
        n8 = lib.Act8(s["n8"], s["n8s"]) if c["act8"] else None
        r = lib.residual_norm_fwd(s["h"], s["o"], post_norm=c["post"], post_gain=s["post_gain"], gate=s["gate"],
                                  scale=c["scale"], gain=s["gain"], gain_offset=c["offset"], h_out=s["h_out"], n=s["n"],
                                  n8=n8)
        out = {"n": r.n, "rstd": r.rstd}
        if c["block"]:
            out["h"] = r.h
        if c["post"]:
            out["rstd_o"] = r.rstd_o
        if c["act8"]:
            out["n_back"] = lib.act8_dequantize(n8, out=s["n_back"])
        return out
    r = lib.residual_norm_bwd(s["dn"], s["rstd"], h=None if c["act8"] else s["h"],
                              n8=lib.Act8(s["n8"], s["n8s"]) if c["act8"] else None, dres=s["dres"], o=s["o"],
                              post_norm=c["post"], rstd_o=s.get("rstd_o"), post_gain=s["post_gain"], gate=s["gate"],
                              scale=c["scale"], gain=s["gain"], gain_offset=c["offset"])
    out = {"dh": r.dh, "do": r.do, "dgate": r.dgate, "dpost_gain": r.dpost_gain, "dgain": r.dgain}
    return {n: x for n, x in out.items() if x is not None}


def work(case):
    t = case["t"]
    if case["op"] == "linear":
        n, k, r = case["n"], case["k"], RANK
        weight = n * k * (2 if case["dense"] else 0.5625)
        return {"bytes": weight + 2 * t * n + 1.0625 * t * k + 2 * t * k + 4 * t * r + 6 * r * (n + k),
                "flops": 2 * t * n * k + 4 * t * r * (n + k)}
    c = case["c"]
    e = t * c
    if case["op"] == "act8":  # the checkpoint is written and read
        return {"bytes": (2 + 1.0625 + 1.0625 + 2) * e, "flops": 4 * e}
    if case["op"] == "mlp":  # two checkpoints, written once and read twice: the down projection's backward lies between
        return {"bytes": (3 * 2 + 4 * 2 + 3 * 2.125) * e, "flops": 28 * e}
    gate = {"none": 0, "channel": 2 * c, "token": 2 * e}[case["gate"]]
    params = 2 * c * (case["gain"] + case["post"])
    if case["op"] == "norm_fwd":
        b = 2 * e + 2 * e + (4 * e if case["block"] else 0) + (4.125 * e if case["act8"] else 0)
        return {"bytes": b + gate + params + 4 * t * (1 + case["post"]), "flops": 10 * e}
    b = 2 * e * case["dns"] + 2 * e + (1.0625 * e if case["act8"] else 2 * e) + 2 * e + (4 * e if case["block"] else 0)
    return {"bytes": b + 2 * gate + 3 * params + 4 * t * (1 + case["post"]), "flops": 24 * e}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def _exact_checkpoint(x):
    """The nearest of 255 even steps between minus and plus the largest of each 64, in 64 bits."""
    b = x.double().reshape(-1, 64)
    step = b.abs().max(dim=1, keepdim=True).values / 127
    return torch.where(step > 0, torch.round(b / step) * step, torch.zeros_like(b)).reshape(x.shape)


def exact(case, seed):
    s = prepare(case, seed)
    op, t = case["op"], case["t"]
    if op == "act8":
        return _exact_checkpoint(s["x"])
    if op == "mlp":
        out = {"m": torch.nn.functional.silu(s["gate"].double()) * s["up"].double()}
        gate, up = _exact_checkpoint(s["gate"]).requires_grad_(), _exact_checkpoint(s["up"]).requires_grad_()
        again = torch.nn.functional.silu(gate) * up
        dgate, dup = torch.autograd.grad(again, (gate, up), s["dm"].double())
        return dict(out, m_again=again.detach(), dgate=dgate, dup=dup)
    if op == "linear":
        if case["dense"]:
            w = s["w"].double()
        else:
            low, high = (s["codes"] % 16).long(), (s["codes"] // 16).long()
            level = _levels("cuda").float()[torch.stack((low, high), 2).flatten(1)]
            w = (level * s["absmax"].repeat_interleave(64, 1)).bfloat16().double()
            del low, high, level
        x = (s["x8"].double() - 128) * s["x8s"].double().repeat_interleave(64, 1)
        x = x.float().bfloat16().double()  # an operand of the products is a bf16 value
        dy, lora = s["dy"].double(), s["B"].double() @ s["A"].double() * (ALPHA / RANK)
        return {"dx": dy @ (w + lora), "dA": s["B"].double().t() @ (dy.t() @ x) * (ALPHA / RANK),
                "dB": dy.t() @ s["u"].double() * (ALPHA / RANK)}
    leaf = {n: s[n].double().requires_grad_() for n in ("h", "o", "post_gain", "gain", "gate") if s[n] is not None}

    def unit(x, r=None):
        return x / torch.sqrt(x.pow(2).mean(1, keepdim=True) + 1e-6) if r is None else x * r

    def weight(name):
        return leaf[name] + case["offset"] if name in leaf else 1.0

    if op == "norm_fwd":
        with torch.no_grad():
            x, out = leaf["h"], {}
            if case["block"]:
                v = leaf["o"]
                if case["post"]:
                    out["rstd_o"] = 1 / torch.sqrt(v.pow(2).mean(1) + 1e-6)
                    v = unit(v) * weight("post_gain")
                x = x + case["scale"] * leaf.get("gate", 1.0) * v
                out["h"] = x
            out["rstd"] = 1 / torch.sqrt(x.pow(2).mean(1) + 1e-6)
            out["n"] = unit(x) * weight("gain")
            if case["act8"]:
                out["n_back"] = _exact_checkpoint(out["n"].float().bfloat16())
            return out
    # the statistics are the caller's: their derivative is put in by hand
    g = sum(d.double() for d in s["dn"])
    r = s["rstd"].double()[:, None]
    if case["act8"]:
        b = (s["n8"].double() - 128) * s["n8s"].double().repeat_interleave(64, 1)
    else:
        b = leaf["h"].detach() * r
    c = b.shape[1]
    weighted = g * (weight("gain").detach() if case["gain"] else 1.0)
    ds = s["dres"].double() + r * weighted - r * b * ((weighted * b).sum(1, keepdim=True) / c)
    out = {"dh": ds}
    if case["gain"]:
        out["dgain"] = torch.einsum("tc,tc->c", g, b)
    if not case["block"]:
        return out
    r_o = s["rstd_o"].double()[:, None] if case["post"] else None
    branch = unit(leaf["o"], r_o if case["post"] else 1.0) * weight("post_gain")
    branch = case["scale"] * leaf.get("gate", 1.0) * branch
    names = [n for n in ("o", "gate", "post_gain") if n in leaf]
    grads = dict(zip(names, torch.autograd.grad(branch, [leaf[n] for n in names], ds)))
    do = grads["o"]
    if case["post"]:
        bo = leaf["o"].detach() * r_o
        do = do - r_o * bo * ((do / r_o * bo).sum(1, keepdim=True) / c)
    out["do"] = do
    if "gate" in grads:
        out["dgate"] = grads["gate"]
    if case["post"]:
        out["dpost_gain"] = grads["post_gain"]
    return out
