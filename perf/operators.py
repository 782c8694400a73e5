"""Measured cases of the operators that a decoder layer's training step adds to the NF4-LoRA linear: rotary positions
(nf4_rope), grouped-query attention with packed sequences forward and backward (nf4_attn_fwd, nf4_attn_bwd), and the
global gradient norm with clipping over many tensors (nf4_grad_clip).

Where ``own`` is false, ``run`` computes the plain form in torch; where it is true, the framework's kernels. ``exact``
gives the same outputs from the definitions in 64 bits.
"""

import math

import torch

own = False

BF16 = torch.bfloat16
# (query heads, kv heads, head width, hidden, intermediate, layers) of the stacks this repository measures
HEADS = {"tiny": (4, 1, 32), "7b": (28, 4, 128), "32b": (40, 8, 128), "72b": (64, 8, 128), "mha64": (16, 16, 64),
         "gqa64": (14, 2, 64)}
WIDTHS = {"tiny": (128, 128, 32, 256, 3), "7b": (3584, 3584, 512, 18944, 28), "32b": (5120, 5120, 1024, 27648, 64),
          "72b": (8192, 8192, 1024, 29568, 80)}


def _attn(name, op, heads, lens, causal=True):
    hq, hkv, d = HEADS[heads]
    c = {"op": op, "hq": hq, "hkv": hkv, "d": d, "lens": lens, "causal": causal}
    return dict(c, name=name) if name else c


def _rope(name, heads, t, sections, inverse=False):
    hq, hkv, d = HEADS[heads]
    c = {"op": "rope", "hq": hq, "hkv": hkv, "d": d, "t": t, "sections": sections, "inverse": inverse}
    return dict(c, name=name) if name else c


def _clip(name, stack, layers, rank, dtype, in_place):
    hidden, q, kv, inter, _ = WIDTHS[stack]
    c = {"op": "clip", "hidden": hidden, "q": q, "kv": kv, "inter": inter, "layers": layers, "rank": rank,
         "dtype": dtype, "in_place": in_place}
    return dict(c, name=name) if name else c


def listed():
    return [
        # a 40-token step of the small stack that the tests drive: latency alone
        _attn("fwd_tiny_40", "attn_fwd", "tiny", "40"),
        # the layer benchmark's tokens on the 7B widths: the ordinary streamed training step
        _attn("fwd_7b_512", "attn_fwd", "7b", "512"),
        # several samples of odd lengths packed into one batch, 32B widths
        _attn("fwd_32b_packed", "attn_fwd", "32b", "1,733,64,1291,17,1025,965"),
        # a long sequence on the 72B widths
        _attn("fwd_72b_8192", "attn_fwd", "72b", "8192"),
        # the backward of the ordinary step
        _attn("bwd_7b_512", "attn_bwd", "7b", "512"),
        # without a causal mask, 64-wide heads, one kv head a query head, packed and ragged
        _attn("bwd_mha64_packed_full", "attn_bwd", "mha64", "511,130,1407", False),
        # the long sequence's backward: the largest case
        _attn("bwd_72b_8192", "attn_bwd", "72b", "8192"),
        # one new token's q and k
        _rope("rope_7b_1", "7b", 1, "64"),
        # a long mixed sequence with time, height and width positions, 72B widths, the gradient's direction
        _rope("rope_72b_8192_axes3", "72b", 8192, "16,24,24", True),
        # the adapters' gradients of one 7B layer in bf16: 14 tensors, latency
        _clip("clip_7b_layer_bf16", "7b", 1, 16, "bfloat16", False),
        # the ordinary step of a 7B stack whose norm is below the bound: nothing to scale, in place
        _clip("clip_7b_stack_below", "7b", 28, 16, "float32", True),
        # a 72B stack's 1120 gradient tensors, scaled
        _clip("clip_72b_stack", "72b", 80, 16, "float32", False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "rope", "clip"])
    if op == "rope":
        heads = rng.choice(sorted(HEADS))
        half = HEADS[heads][2] // 2
        a = rng.randrange(1, half - 1)
        b = rng.randrange(1, half - a)
        sections = rng.choice(["%d" % half, "%d,%d" % (a, half - a), "%d,%d,%d" % (a, b, half - a - b)])
        return _rope(None, heads, _log_int(rng, 1, 8192), sections, rng.random() < 0.5)
    if op == "clip":
        stack = rng.choice(sorted(WIDTHS))
        return _clip(None, stack, _log_int(rng, 1, WIDTHS[stack][4]), rng.choice([1, 5, 8, 16]),
                     rng.choice(["float32", "bfloat16"]), rng.random() < 0.3)
    heads = rng.choice(sorted(HEADS))
    causal = rng.random() < 0.75
    t = _log_int(rng, 1, 8192 if causal else 5000)
    n = rng.choice([1, 1, 1, 2, 3, 8])
    cuts = sorted(rng.randrange(0, t + 1) for _ in range(n - 1))  # a sequence may come out empty
    lens = [b - a for a, b in zip([0] + cuts, cuts + [t])]
    return _attn(None, op, heads, ",".join(map(str, lens)), causal)


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def _sections(case):
    return [int(v) for v in case["sections"].split(",")]


def _grad_sizes(case):
    """Elements of each gradient tensor, dA [r, K] and dB [N, r] of the seven projections, layer after layer."""
    h, q, kv, i, r = case["hidden"], case["q"], case["kv"], case["inter"], case["rank"]
    shapes = [(q, h), (kv, h), (kv, h), (h, q), (i, h), (i, h), (h, i)]
    return [r * v for _ in range(case["layers"]) for n, k in shapes for v in (k, n)]


MAX_NORM = 1.0


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(BF16)

    s = {"case": case}
    if case["op"] == "clip":
        sizes = _grad_sizes(case)
        # per-element spreads of trained adapters' gradients; below the bound where nothing is to be scaled
        std = (0.1 if case["in_place"] else 30.0) / math.sqrt(sum(sizes))
        flat = torch.randn(sum(sizes), generator=g, device="cuda").mul_(std).to(getattr(torch, case["dtype"]))
        out = flat if case["in_place"] else torch.empty_like(flat)
        s.update(flat=flat, out=out)
        if own:  # the handle that a training program makes once over its gradient buffers
            from nf4_weight_streamed_amd import lib
            s["grads"] = lib.GradList(list(flat.split(sizes)), list(out.split(sizes)))
        return s
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        t, sections = case["t"], _sections(case)
        i = torch.arange(t, device="cuda") + int(torch.randint(0, 100000, (1,), generator=g, device="cuda"))
        # text counts on; images and video count frames of 32 x 24 patches, their rows and columns
        pos = [i] if len(sections) == 1 else [i // 768, i // 24 % 32, i % 24][:len(sections)]
        s.update(q=normal(t, hq * d), k=normal(t, hkv * d), pos=torch.stack(pos).to(torch.int32).contiguous(),
                 inv_freq=1e6 ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d), sections=sections)
        s.update(q_out=torch.empty_like(s["q"]), k_out=torch.empty_like(s["k"]))
        return s
    lens = _lens(case)
    t = sum(lens)
    s.update(q=normal(t, hq * d, std=2.0), k=normal(t, hkv * d), v=normal(t, hkv * d), cu=None)
    seq = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).cuda()
    s["seq"] = seq  # which sequence a row belongs to: the plain form's mask
    if len(lens) > 1:
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32).cuda()
    s.update(o=torch.empty_like(s["q"]), lse=torch.empty(hq, t, device="cuda"))
    if case["op"] == "attn_bwd":
        s["o"], s["lse"] = _plain_attn_fwd(s)
        s.update(do=normal(t, hq * d), dq=torch.empty_like(s["q"]), dk=torch.empty_like(s["k"]),
                 dv=torch.empty_like(s["v"]))
    return s


# ------------------------------------------------------------------ plain forms, in 32 bits

def _heads(x, hkv, d):
    """[T, heads * d] -> float32 [kv heads, heads a kv head, T, d]."""
    t = x.shape[0]
    return x.float().view(t, hkv, -1, d).permute(1, 2, 0, 3).contiguous()


def _rows(x):
    """The way back: [kv heads, group, T, d] -> [T, heads * d]."""
    return x.permute(2, 0, 1, 3).reshape(x.shape[2], -1)


def _plain_scores(s):
    c = s["case"]
    q, k = _heads(s["q"], c["hkv"], c["d"]), _heads(s["k"], c["hkv"], c["d"])
    scores = torch.matmul(q, k.transpose(-1, -2).contiguous()).mul_(1.0 / math.sqrt(c["d"]))
    t = q.shape[2]
    off = s["seq"][:, None] != s["seq"][None, :]
    if c["causal"]:
        off |= torch.ones(t, t, dtype=torch.bool, device=q.device).triu_(1)
    return scores.masked_fill_(off, -math.inf)


def _plain_attn_fwd(s):
    c = s["case"]
    p = _plain_scores(s)
    top = p.amax(-1, keepdim=True)
    p = p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, _heads(s["v"], c["hkv"], c["d"])) / total
    return _rows(o).to(BF16), (top + total.log()).view(c["hq"], -1)


def _plain_attn_bwd(s):
    c = s["case"]
    hkv, d = c["hkv"], c["d"]
    q, k, v = (_heads(s[n], hkv, d) for n in ("q", "k", "v"))
    do, o = _heads(s["do"], hkv, d), _heads(s["o"], hkv, d)
    lse = s["lse"].view(hkv, -1, q.shape[2], 1)
    p = _plain_scores(s).sub_(lse).exp_()
    dv = torch.matmul(p.transpose(-1, -2), do).sum(1, keepdim=True)
    dp = torch.matmul(do, v.transpose(-1, -2).contiguous())
    ds = p.mul_(dp.sub_((do * o).sum(-1, keepdim=True))).mul_(1.0 / math.sqrt(d))
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(1, keepdim=True)
    return _rows(dq).to(BF16), _rows(dk).to(BF16), _rows(dv).to(BF16)


def _plain_rope(s):
    c = s["case"]
    d = c["d"]
    axis = torch.repeat_interleave(torch.arange(len(s["sections"])), torch.tensor(s["sections"])).to(s["pos"].device)
    angle = s["pos"].double()[axis].t() * s["inv_freq"]  # [T, d / 2]; far positions lose their fraction in 32 bits
    sign = -1.0 if c["inverse"] else 1.0
    cos, sin = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :] * sign
    out = []
    for x in (s["q"], s["k"]):
        lo, hi = x.float().view(x.shape[0], -1, 2, d // 2).unbind(2)
        out.append(torch.stack([lo * cos - hi * sin, hi * cos + lo * sin], 2).view(x.shape).to(BF16))
    return tuple(out)


def _plain_clip(s):
    flat = s["flat"]
    norm = flat.float().square().sum(dtype=torch.float64).sqrt().float().view(1)
    scale = (MAX_NORM / (norm + 1e-6)).clamp(max=1.0)
    if s["out"] is flat:
        return norm, flat.mul_(scale)
    return norm, (flat.float() * scale).to(flat.dtype)


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"attn_fwd": _plain_attn_fwd, "attn_bwd": _plain_attn_bwd, "rope": _plain_rope,
                "clip": _plain_clip}[op](s)
    from nf4_weight_streamed_amd import lib
    if op == "attn_fwd":
        return lib.attn_fwd(s["q"], s["k"], s["v"], c["d"], cu_seqlens=s["cu"], causal=c["causal"], o=s["o"],
                            lse=s["lse"])
    if op == "attn_bwd":
        return lib.attn_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], c["d"], cu_seqlens=s["cu"],
                            causal=c["causal"], dq=s["dq"], dk=s["dk"], dv=s["dv"])
    if op == "rope":
        return lib.rope(s["q"], s["k"], c["d"], s["pos"], s["inv_freq"], sections=s["sections"],
                        inverse=c["inverse"], q_out=s["q_out"], k_out=s["k_out"])
    return s["grads"].clip(MAX_NORM), s["out"]


def work(case):
    if case["op"] == "clip":
        n, size = sum(_grad_sizes(case)), 4 if case["dtype"] == "float32" else 2
        return {"bytes": n * size * (1 if case["in_place"] else 2) + 4, "flops": 3 * n}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        t = case["t"]
        n = t * (hq + hkv) * d
        return {"bytes": 4 * n + 4 * t * len(_sections(case)) + 4 * d, "flops": 3 * n}
    lens = _lens(case)
    t = sum(lens)
    pairs = sum(n * (n + 1) // 2 if case["causal"] else n * n for n in lens)
    q, kv, lse = 2 * t * hq * d, 2 * t * hkv * d, 4 * t * hq
    if case["op"] == "attn_fwd":
        return {"bytes": 2 * q + 2 * kv + lse, "flops": 4 * d * hq * pairs}
    return {"bytes": 4 * q + 4 * kv + lse, "flops": 10 * d * hq * pairs}


# ------------------------------------------------------------------ from the definitions, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "clip":
        parts = [p.double() for p in s["flat"].split(1 << 26)]
        norm = math.sqrt(math.fsum(float(torch.dot(p, p)) for p in parts))
        scale = min(1.0, MAX_NORM / (norm + 1e-6))
        return torch.tensor([norm], dtype=torch.float64), torch.cat([p * scale for p in parts])
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    if case["op"] == "rope":
        t, half = case["t"], d // 2
        out = {"q": s["q"].double().view(t, hq, d), "k": s["k"].double().view(t, hkv, d)}
        turned = {n: torch.empty_like(x) for n, x in out.items()}
        first = 0
        for a, count in enumerate(s["sections"]):
            for i in range(first, first + count):
                phi = s["pos"][a].double() * s["inv_freq"][i] * (-1 if case["inverse"] else 1)
                z = torch.polar(torch.ones_like(phi), phi)[:, None]
                for n, x in out.items():
                    w = torch.complex(x[:, :, i], x[:, :, i + half]) * z
                    turned[n][:, :, i], turned[n][:, :, i + half] = w.real, w.imag
            first += count
        return turned["q"].reshape(t, -1), turned["k"].reshape(t, -1)
    t = sum(_lens(case))
    x = {n: s[n].double().view(t, -1, d) for n in ("q", "k", "v", "o", "do") if n in s}
    fwd = case["op"] == "attn_fwd"
    o, dq = torch.zeros(t, hq, d, dtype=torch.float64, device="cuda"), torch.zeros(t, hq, d, dtype=torch.float64, device="cuda")
    dk, dv = (torch.zeros(t, hkv, d, dtype=torch.float64, device="cuda") for _ in range(2))
    lse = torch.zeros(hq, t, dtype=torch.float64, device="cuda")
    begin = 0
    for n in _lens(case):
        rows = slice(begin, begin + n)
        begin += n
        if n == 0:
            continue
        for h in range(hq):
            j = h // (hq // hkv)
            q, k, v = (x["q"][rows, h].contiguous(), x["k"][rows, j].contiguous(), x["v"][rows, j].contiguous())
            z = q @ k.t().contiguous() / d ** 0.5
            if case["causal"]:
                z = torch.where(torch.ones_like(z, dtype=torch.bool).tril(), z, -math.inf)
            if fwd:
                lse[h, rows] = torch.logsumexp(z, 1)
                o[rows, h] = torch.softmax(z, 1) @ v
                continue
            p = torch.exp(z - s["lse"][h, rows].double()[:, None])
            g = x["do"][rows, h].contiguous()
            e = p * (g @ v.t().contiguous() - (g * x["o"][rows, h]).sum(1)[:, None]) / d ** 0.5
            dv[rows, j] += p.t().contiguous() @ g
            dq[rows, h] = e @ k
            dk[rows, j] += e.t().contiguous() @ q
    if fwd:
        return o.view(t, -1), lse
    return dq.view(t, -1), dk.view(t, -1), dv.view(t, -1)
