"""fp64 CPU oracle of activations kept in 8 bits (the checkpoint format, the SiLU product at its
values) and of the residual add fused with the norms around a block, forward and backward.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): plain numpy from the definitions.

Pins (tests/test_oracle_act8.py): act8_quantize by exact rational arithmetic and by its error
bound; residual_norm_bwd and silu_mul_bwd by central finite differences of their forwards;
decoder_backward_act8, with checkpoints that hold their values exactly, by decoder_backward.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

from .decoder_oracle import attention_bwd, rope
from .nf4_oracle import RMS_EPS, _as_f64, _layer_f64, _lin_bwd, round_bf16, silu, silu_grad

__all__ = ["act8_quantize", "act8_values", "silu_mul", "silu_mul_bwd", "residual_norm_fwd", "residual_norm_bwd",
           "decoder_backward_act8"]

BLOCK = 64


def act8_quantize(x):
    """x [T, C] (bf16 bits or values that bf16 holds) -> (codes uint8 [T, C], scale float32 [T, C/64])."""
    b = _as_f64(x).reshape(-1, BLOCK)
    codes, scale = np.full(b.shape, 128, np.uint8), np.zeros(len(b), np.float32)
    bad = ~np.isfinite(b).all(axis=1)
    scale[bad] = np.nan
    a = np.abs(b).max(axis=1)
    some = ~bad & (a > 0)
    lift = np.where(a < 2.0 ** -64, 2.0 ** 64, 1.0)
    with np.errstate(all="ignore"):
        scale[some] = np.float32(a[some]) / np.float32(127)
        inv = np.float32(127) / np.float32(a * lift)
    # bf16 times fp32: 8 + 24 bits, exact in fp64; rint rounds halves to even
    codes[some] = 128 + np.rint((b * lift[:, None])[some] * inv[some].astype(np.float64)[:, None])
    return codes.reshape(np.shape(x)), scale.reshape(np.shape(x)[0], -1)


def act8_values(codes, scale):
    """float32 [T, C]: what a checkpoint stands for."""
    b = codes.reshape(-1, BLOCK).astype(np.float32) - np.float32(128)
    with np.errstate(all="ignore"):
        return (b * scale.reshape(-1, 1)).reshape(codes.shape)


def exact_code(x: float, a: float) -> int:
    """The code of x in a block whose largest magnitude is a >= 2^-64, in rational arithmetic."""
    p = Fraction(float(x)) * Fraction(float(np.float32(127) / np.float32(a)))
    return 128 + round(p)  # halves to even


def silu_mul(gate, up):
    return silu(_as_f64(gate)) * _as_f64(up)


def silu_mul_bwd(gate, up, dm):
    """(dgate, dup)"""
    gate, up, dm = _as_f64(gate), _as_f64(up), _as_f64(dm)
    return dm * up * silu_grad(gate), dm * silu(gate)


def _factor(gain, offset):
    return 1.0 if gain is None else _as_f64(gain) + offset


def residual_norm_fwd(h, o=None, post_norm=False, post_gain=None, gate=None, scale=1.0, gain=None, offset=0.0, eps=1e-6):
    """-> dict of s (the stream, unrounded), n, rstd_o (or None), rstd."""
    s, rstd_o = _as_f64(h), None
    if o is not None:
        v = _as_f64(o)
        if post_norm:
            rstd_o = 1.0 / np.sqrt(np.mean(v * v, axis=1) + eps)
            v = v * rstd_o[:, None] * _factor(post_gain, offset)
        s = s + scale * (1.0 if gate is None else _as_f64(gate)) * v
    rstd = 1.0 / np.sqrt(np.mean(s * s, axis=1) + eps)
    return {"s": s, "n": s * rstd[:, None] * _factor(gain, offset), "rstd_o": rstd_o, "rstd": rstd}


def residual_norm_bwd(dn, rstd, b, dres=None, o=None, post_norm=False, rstd_o=None, post_gain=None, gate=None, scale=1.0,
                      gain=None, offset=0.0):
    """b: the normalised stream (h rstd, or a checkpoint's values). dn: a list. -> dict of dh, dgain and,
    with o, do, dgate (a row per token), dpost_gain."""
    g = sum(_as_f64(d) for d in dn)
    rstd, b = _as_f64(rstd)[:, None], _as_f64(b)
    w = g * _factor(gain, offset)
    ds = rstd * (w - b * np.mean(w * b, axis=1, keepdims=True))
    if dres is not None:
        ds = ds + _as_f64(dres)
    out = {"dh": ds, "dgain": np.sum(g * b, axis=0)}
    if o is None:
        return out
    u = _as_f64(o) * (_as_f64(rstd_o)[:, None] if post_norm else 1.0)
    dv = scale * ds
    out["dgate"] = dv * u * (_factor(post_gain, offset) if post_norm else 1.0)
    if gate is not None:
        dv = dv * _as_f64(gate)
    out["dpost_gain"] = np.sum(dv * u, axis=0)
    if post_norm:
        p = dv * _factor(post_gain, offset)
        dv = _as_f64(rstd_o)[:, None] * (p - u * np.mean(p * u, axis=1, keepdims=True))
    out["do"] = dv
    return out


def decoder_backward_act8(dh, layers, dims, alpha, saved, pos, inv_freq, lens=None, keep=None):
    """decoder_backward where ha, hm, gate and up are what their 8-bit checkpoints stand for, m is
    formed again from the latter two, and the norms go back through their own results (ha, hm) and
    1 / rms. keep(x) gives a checkpoint's values (default: act8_quantize's)."""
    keep = keep or (lambda x: act8_values(*act8_quantize(x)).astype(np.float64))
    dh, d, grads = _as_f64(dh), dims.head_dim, [None] * len(layers)

    def norm_back(n, h, dres, dys):
        rstd = 1.0 / np.sqrt(np.mean(h * h, axis=1) + RMS_EPS)
        return round_bf16(residual_norm_bwd(dys, rstd, n, dres)["dh"])

    for li in range(len(layers) - 1, -1, -1):
        p, st, g = _layer_f64(layers[li]), saved[li], {}
        ha, hm, gate, up = (keep(st[n]) for n in ("ha", "hm", "gate", "up"))

        def lin(x, name, dy):
            dx, g[name + "_dA"], g[name + "_dB"] = _lin_bwd(x, p[name], alpha, dy)
            return round_bf16(dx)

        dm = lin(round_bf16(silu_mul(gate, up)), "down", dh)
        dgate, dup = (round_bf16(x) for x in silu_mul_bwd(gate, up, dm))
        dhm = [lin(round_bf16(hm), n, dy) for n, dy in (("gate", dgate), ("up", dup))]
        dh1 = norm_back(hm, st["h1"], dh, dhm)
        da = lin(st["a"], "o", dh1)
        dq, dk, dv = (round_bf16(x) for x in attention_bwd(st["q"], st["k"], st["v"], st["a"], st["lse"], da, d, lens))
        dq, dk = (round_bf16(rope(x, d, pos, inv_freq, inverse=True)) for x in (dq, dk))
        dha = [lin(round_bf16(ha), n, dy) for n, dy in (("v", dv), ("q", dq), ("k", dk))]
        # dB's products read u = x A^T of the forward's own x
        for n, x, dy in (("gate", "hm", dgate), ("up", "hm", dup), ("v", "ha", dv), ("q", "ha", dq), ("k", "ha", dk),
                         ("down", "m", dh)):
            g[n + "_dB"] = _lin_bwd(st[x], p[n], alpha, dy)[2]
        dh = norm_back(ha, st["h"], dh1, dha)
        grads[li] = g
    return dh, grads
