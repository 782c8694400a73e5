"""Pins of the oracle's decoder operators: attention, rotary positions, clipping, and the
attention-mixing stack, against brute force, limits and central finite differences."""

import math

import numpy as np
import pytest

import oracle as O


def test_attention_is_the_softmax_average():
    rng = np.random.default_rng(1)
    t, hq, hkv, d = 5, 4, 2, 3
    q, k, v = (rng.integers(-2, 3, size=(t, h * d)).astype(float) for h in (hq, hkv, hkv))
    o, lse = O.attention_fwd(q, k, v, d, causal=True, scale=0.5)
    for h in range(hq):
        for i in range(t):
            e = [math.exp(0.5 * sum(q[i, h * d + x] * k[j, h // 2 * d + x] for x in range(d))) for j in range(i + 1)]
            assert lse[h, i] == pytest.approx(math.log(sum(e)), rel=1e-12)
            for x in range(d):
                want = sum(e[j] * v[j, h // 2 * d + x] for j in range(i + 1)) / sum(e)
                assert o[i, h * d + x] == pytest.approx(want, rel=1e-12, abs=1e-12)


def test_attention_limits():
    rng = np.random.default_rng(2)
    v = rng.normal(size=(6, 4))
    zero = np.zeros((6, 4))
    o, lse = O.attention_fwd(zero, zero, v, 4, causal=True)          # equal scores: running means
    assert np.allclose(o, np.cumsum(v, 0) / np.arange(1, 7)[:, None]) and np.allclose(lse[0], np.log(np.arange(1, 7)))
    k = np.zeros((6, 4))
    k[0, 0] = 1e6                                                     # one key dominates
    o, _ = O.attention_fwd(np.ones((6, 4)), k, v, 4)
    assert np.allclose(o, v[0])
    a, _ = O.attention_fwd(v, v, v, 4, lens=[1, 0, 5])                # sequences are apart
    b, _ = O.attention_fwd(v[1:], v[1:], v[1:], 4)
    assert np.allclose(a[0], v[0]) and np.array_equal(a[1:], b)


@pytest.mark.parametrize("causal", [True, False])
def test_attention_bwd_finite_differences(causal):
    rng = np.random.default_rng(3)
    t, d, lens = 7, 4, [4, 0, 3]
    x = {"q": rng.normal(size=(t, 4 * d)), "k": rng.normal(size=(t, 2 * d)), "v": rng.normal(size=(t, 2 * d))}
    do = rng.normal(size=(t, 4 * d))
    f = lambda y: float(np.sum(do * O.attention_fwd(y["q"], y["k"], y["v"], d, lens, causal)[0]))
    o, lse = O.attention_fwd(x["q"], x["k"], x["v"], d, lens, causal)
    g = dict(zip("qkv", O.attention_bwd(x["q"], x["k"], x["v"], o, lse, do, d, lens, causal)))
    for name in "qkv":
        step = rng.normal(size=x[name].shape)
        hi, lo = ({**x, name: x[name] + s * 1e-5 * step} for s in (1, -1))
        assert (f(hi) - f(lo)) / 2e-5 == pytest.approx(float(np.sum(g[name] * step)), rel=1e-7, abs=1e-8)


def test_rope_is_a_rotation():
    rng = np.random.default_rng(4)
    d, t = 8, 6
    x = rng.normal(size=(t, 2 * d))
    inv = 1e4 ** (-np.arange(0, d, 2) / d)
    pos = np.stack([rng.integers(-9, 99, t) for _ in range(3)])
    y = O.rope(x, d, pos, inv, [1, 2, 1])
    for h in range(2):
        for i, axis in enumerate([0, 1, 1, 2]):
            z = (x[:, h * d + i] + 1j * x[:, h * d + i + 4]) * np.exp(1j * pos[axis] * inv[i])
            assert np.allclose(y[:, h * d + i], z.real) and np.allclose(y[:, h * d + i + 4], z.imag)
    assert np.allclose(O.rope(y, d, pos, inv, [1, 2, 1], inverse=True), x)
    a, b = rng.normal(size=(2, 1, d))
    dots = [float(np.sum(O.rope(a, d, [p + 5], inv) * O.rope(b, d, [p], inv))) for p in (0, 17, 4000)]
    assert np.allclose(dots, dots[0])


def test_grad_clip_scales_to_the_bound():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    norm, out = O.grad_clip(g, 1.0)
    assert norm == 5.0 and np.allclose(out[0], [3 / (5 + 1e-6), 0]) and np.allclose(out[1], 4 / (5 + 1e-6))
    norm, out = O.grad_clip(g, 5.1)
    assert norm == 5.0 and np.array_equal(out[0], g[0]) and np.array_equal(out[1], g[1])


def test_decoder_stack_finite_differences():
    rng = np.random.default_rng(5)
    dims, alpha, t, lens = O.StackLayerDims(hidden=16, q=16, kv=8, inter=24, head_dim=4), 4.0, 6, [2, 4]
    layers = []
    for _ in range(2):
        layers.append({n: (rng.normal(0, 1 / np.sqrt(k), (m, k)), rng.normal(0, 1 / np.sqrt(k), (2, k)),
                           rng.normal(0, 0.3, (m, 2))) for n, (m, k) in dims.proj_shapes().items()})
    pos, inv = np.array([0, 1, 0, 1, 2, 3]), 100.0 ** (-np.arange(0, 4, 2) / 4)
    h0, dh = rng.normal(size=(2, t, 16))

    def loss(h, ls):
        return float(np.sum(dh * O.decoder_forward(h, ls, dims, alpha, pos, inv, lens, round_storage=False)[0]))

    _, saved = O.decoder_forward(h0, layers, dims, alpha, pos, inv, lens, round_storage=False)
    dh0, grads = O.decoder_backward(dh, layers, dims, alpha, saved, pos, inv, lens, round_storage=False)
    step = rng.normal(size=h0.shape)
    got = (loss(h0 + 1e-5 * step, layers) - loss(h0 - 1e-5 * step, layers)) / 2e-5
    assert got == pytest.approx(float(np.sum(dh0 * step)), rel=1e-6, abs=1e-7)
    for li in range(2):
        for n in dims.proj_shapes():
            for which, key in ((1, "_dA"), (2, "_dB")):
                step = rng.normal(size=layers[li][n][which].shape)
                vals = []
                for s in (1e-5, -1e-5):
                    moved = [dict(l) for l in layers]
                    w = list(moved[li][n])
                    w[which] = w[which] + s * step
                    moved[li][n] = tuple(w)
                    vals.append(loss(h0, moved))
                got = (vals[0] - vals[1]) / 2e-5
                assert got == pytest.approx(float(np.sum(grads[li][n + key] * step)), rel=1e-5, abs=1e-6), (li, n, key)
