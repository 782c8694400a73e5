"""fp64 CPU oracle of the decoder layer's remaining operators: rotary positions, softmax
attention over packed sequences (forward and backward), the gradients' global norm with
clipping, and the decoder stack whose layers mix tokens by that attention.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``): plain numpy from the definitions.

Pins (tests/test_oracle_decoder.py): attention_bwd by central finite differences of
attention_fwd; attention_fwd by a brute-force softmax on small integers and by its limits
(one key, equal keys, a dominating key); rope by the complex product, its inverse and the
dependence of rotated dot products on position differences alone; decoder_backward by
central finite differences of decoder_forward (storage rounding off).
"""

from __future__ import annotations

import numpy as np

from .nf4_oracle import (_as_f64, _layer_f64, _lin, _lin_bwd, rmsnorm_bwd, rmsnorm_fwd, round_bf16, silu, silu_grad)

__all__ = ["attention_fwd", "attention_bwd", "attention_bounds", "rope", "grad_clip", "decoder_forward",
           "decoder_backward"]


def _spans(t, lens):
    """(begin, end) of each sequence; None: one of all rows."""
    if lens is None:
        return [(0, t)]
    ends = np.cumsum(lens)
    return [(int(e - n), int(e)) for e, n in zip(ends, lens)]


def _scores(q, k, scale, causal):
    s = scale * (q @ k.T)
    if causal:
        s = np.where(np.tri(len(q), dtype=bool), s, -np.inf)
    return s


def attention_fwd(q, k, v, head_dim, lens=None, causal=True, scale=None):
    """q [T, hq*D], k, v [T, hkv*D] -> (o [T, hq*D], lse [hq, T]); rows outside the sequences are 0."""
    q, k, v = (_as_f64(x) for x in (q, k, v))
    t, d = q.shape[0], head_dim
    scale = d ** -0.5 if scale is None else scale
    hq, hkv = q.shape[1] // d, k.shape[1] // d
    o, lse = np.zeros_like(q), np.zeros((hq, t))
    for b, e in _spans(t, lens):
        if e == b:
            continue
        for h in range(hq):
            c, ck = slice(h * d, h * d + d), slice(h // (hq // hkv) * d, h // (hq // hkv) * d + d)
            s = _scores(q[b:e, c], k[b:e, ck], scale, causal)
            top = s.max(axis=1, keepdims=True)
            p = np.exp(s - top)
            total = p.sum(axis=1, keepdims=True)
            o[b:e, c] = p @ v[b:e, ck] / total
            lse[h, b:e] = (top + np.log(total))[:, 0]
    return o, lse


def attention_bwd(q, k, v, o, lse, do, head_dim, lens=None, causal=True, scale=None):
    """(dq, dk, dv) from the stored o and lse: P = e^(S - lse), delta = do . o."""
    q, k, v, o, lse, do = (_as_f64(x) for x in (q, k, v, o, lse, do))
    d = head_dim
    scale = d ** -0.5 if scale is None else scale
    hq, hkv = q.shape[1] // d, k.shape[1] // d
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b, e in _spans(q.shape[0], lens):
        if e == b:
            continue
        for h in range(hq):
            c, ck = slice(h * d, h * d + d), slice(h // (hq // hkv) * d, h // (hq // hkv) * d + d)
            p = np.exp(_scores(q[b:e, c], k[b:e, ck], scale, causal) - lse[h, b:e, None])
            g = do[b:e, c]
            ds = p * (g @ v[b:e, ck].T - np.sum(g * o[b:e, c], axis=1, keepdims=True))
            dq[b:e, c] = scale * ds @ k[b:e, ck]
            dk[b:e, ck] += scale * ds.T @ q[b:e, c]
            dv[b:e, ck] += p.T @ g
    return dq, dk, dv


def attention_bounds(q, k, v, o, lse, do, head_dim, lens=None, causal=True, scale=None, ds_unit=2.0 ** -8):
    """How far an fp32 evaluation that rounds P and dS to bf16 for their products may be from
    the exact outputs (before an output's own rounding): {"o", "lse", "dq", "dk", "dv"}.

    With u = 2^-24: a score is a sum of D exact bf16 products in fp32, then one multiply-add
    and an exp2 (2 units), so as an exponent it is off by at most
        e = u (D + 4) max scale sum|q||k| + 3 u max|lse| + 2^-21
    (lse: its own rounding and its product with log2 e), which is P's relative error. Rounding P to bf16 adds at most 2^-8 of P. Sums over n rows
    add n u of the sum of magnitudes. lse: its sum's relative error (e + n u) as an absolute
    one, plus 2^-22 of its own size. dP and delta are D-term sums: off by
    u (D + 1) (|do||v| + |do||o|); dS by P times that, plus |dS| (e + 2u), plus ds_unit of |dS|
    (2^-8 for one bf16 value, 2^-16 for the sum of two).
    Underflow: a P or dS below 2^-126, the least normal value of fp32 and bf16 alike, may
    come out as zero: each is off by at most 2^-126 more (P's times |dP - delta| in dS).
    """
    q, k, v, o, lse, do = (_as_f64(x) for x in (q, k, v, o, lse, do))
    d, u, t = head_dim, 2.0 ** -24, q.shape[0]
    scale = d ** -0.5 if scale is None else scale
    hq, hkv = q.shape[1] // d, k.shape[1] // d
    out = {"o": np.zeros_like(q), "lse": np.zeros((hq, t)), "dq": np.zeros_like(q), "dk": np.zeros_like(k),
           "dv": np.zeros_like(v)}
    rep = hq // hkv
    for b, e_ in _spans(t, lens):
        n = e_ - b
        if n == 0:
            continue
        for h in range(hq):
            c, ck = slice(h * d, h * d + d), slice(h // rep * d, h // rep * d + d)
            qa, ka, va, ga, oa = (np.abs(x[b:e_, s]) for x, s in ((q, c), (k, ck), (v, ck), (do, c), (o, c)))
            e = u * (d + 4) * scale * float((qa @ ka.T).max()) + 2.0 ** -21
            e += 3 * u * float(np.abs(lse[h, b:e_]).max())
            p = np.exp(_scores(q[b:e_, c], k[b:e_, ck], scale, causal) - lse[h, b:e_, None])
            rel = 2.0 ** -8 + 2 * e + 2 * (n + 64) * u
            tiny = 2.0 ** -126
            out["o"][b:e_, c] = (rel * p + tiny) @ va
            out["lse"][h, b:e_] = e + (n + 64) * u + 2.0 ** -22 * (1 + np.abs(lse[h, b:e_]))
            err_dp = u * (d + 1) * (ga @ va.T + np.sum(ga * oa, axis=1, keepdims=True))
            rest = np.abs(do[b:e_, c] @ v[b:e_, ck].T - np.sum(do[b:e_, c] * o[b:e_, c], axis=1, keepdims=True))
            ds = p * rest
            err = p * err_dp * (1 + ds_unit) + ds * (ds_unit + e + 2 * u) + tiny * (1 + rest)
            # sums over n rows (and rep heads) in fp32, and the final scaling
            out["dq"][b:e_, c] = scale * ((err + (n + 64) * u * ds) @ ka)
            out["dk"][b:e_, ck] += scale * ((err + (rep * n + 64) * u * ds).T @ qa)
            out["dv"][b:e_, ck] += ((2.0 ** -8 + e + (rep * n + 64) * u) * p + tiny).T @ ga
    return out


def rope(x, head_dim, pos, inv_freq, sections=None, inverse=False):
    """x [T, heads*D] with pair (i, i + D/2) of each head turned by pos[axis(i)] * inv_freq[i]."""
    x, pos = _as_f64(x), np.atleast_2d(np.asarray(pos))
    half = head_dim // 2
    axis = np.repeat(np.arange(pos.shape[0]), [half] if sections is None else sections)
    phi = (pos[axis].T.astype(np.float64) * np.asarray(inv_freq))[:, None, :] * (-1.0 if inverse else 1.0)
    y = x.reshape(x.shape[0], -1, head_dim)
    lo, hi = y[..., :half], y[..., half:]
    return np.concatenate([lo * np.cos(phi) - hi * np.sin(phi), hi * np.cos(phi) + lo * np.sin(phi)],
                          axis=-1).reshape(x.shape)


def grad_clip(grads, max_norm):
    """(norm, scaled gradients): g * min(1, max_norm / (norm + 1e-6))."""
    norm = float(np.sqrt(sum(np.sum(np.square(np.asarray(g, np.float64))) for g in grads)))
    f = min(1.0, max_norm / (norm + 1e-6))
    return norm, [np.asarray(g, np.float64) * f for g in grads]


def decoder_forward(h0, layers, dims, alpha, pos, inv_freq, lens=None, round_storage=True):
    """The stack of ``stack_forward`` with attention in place of the identity mixing:
    a = attention(rope(q), rope(k), v), causal within each sequence. Storage points in
    addition: rotated q and k, a. (lse is fp32.)"""
    rnd = round_bf16 if round_storage else (lambda z: np.asarray(z, dtype=np.float64))
    h, d, saved = _as_f64(h0), dims.head_dim, []
    for layer in layers:
        p, st = _layer_f64(layer), {"h": h}
        st["ha"] = rnd(rmsnorm_fwd(h))
        for name in ("q", "k", "v"):
            st[name] = rnd(_lin(st["ha"], p[name], alpha)[0])
        for name in ("q", "k"):
            st[name] = rnd(rope(st[name], d, pos, inv_freq))
        a, st["lse"] = attention_fwd(st["q"], st["k"], st["v"], d, lens)
        st["a"] = rnd(a)
        st["h1"] = rnd(h + rnd(_lin(st["a"], p["o"], alpha)[0]))
        st["hm"] = rnd(rmsnorm_fwd(st["h1"]))
        for name in ("gate", "up"):
            st[name] = rnd(_lin(st["hm"], p[name], alpha)[0])
        st["m"] = rnd(silu(st["gate"]) * st["up"])
        h = rnd(st["h1"] + rnd(_lin(st["m"], p["down"], alpha)[0]))
        saved.append(st)
    return h, saved


def decoder_backward(dh, layers, dims, alpha, saved, pos, inv_freq, lens=None, round_storage=True):
    """Backward of ``decoder_forward``: (dh0, grads) with grads[l][name + "_dA" / "_dB"]."""
    rnd = round_bf16 if round_storage else (lambda z: np.asarray(z, dtype=np.float64))
    dh, d, grads = _as_f64(dh), dims.head_dim, [None] * len(layers)
    for li in range(len(layers) - 1, -1, -1):
        p, st, g = _layer_f64(layers[li]), saved[li], {}

        def lin(x, name, dy):
            dx, g[name + "_dA"], g[name + "_dB"] = _lin_bwd(st[x], p[name], alpha, dy)
            return rnd(dx)

        dm = lin("m", "down", dh)
        dhm = rnd(lin("hm", "gate", rnd(dm * st["up"] * silu_grad(st["gate"])))
                  + lin("hm", "up", rnd(dm * silu(st["gate"]))))
        dh1 = rnd(dh + rmsnorm_bwd(st["h1"], dhm))
        da = lin("a", "o", dh1)
        dq, dk, dv = (rnd(x) for x in attention_bwd(st["q"], st["k"], st["v"], st["a"], st["lse"], da, d, lens))
        dq, dk = (rnd(rope(x, d, pos, inv_freq, inverse=True)) for x in (dq, dk))
        dha = rnd(lin("ha", "v", dv) + lin("ha", "q", dq) + lin("ha", "k", dk))
        dh = rnd(dh1 + rmsnorm_bwd(st["h"], dha))
        grads[li] = g
    return dh, grads
