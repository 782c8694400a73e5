"""Pins of the oracle of 8-bit checkpoints and fused residual norms."""

import numpy as np
import pytest

import oracle as O
import synthetic_inputs as S


def _bits(a):
    return S.to_bf16_bits(a)


def test_codes_are_the_exact_products_rounded():
    from oracle.act8_oracle import exact_code

    rng = np.random.default_rng(0)
    x = _bits(np.concatenate([rng.normal(size=(6, 64)), rng.standard_cauchy(size=(6, 64)), 2.0 ** rng.integers(-40, 60, (4, 64))]))
    codes, scale = O.act8_quantize(x)
    v = O.bf16_bits_to_f64(x)
    for row, c in zip(v, codes):
        a = np.abs(row).max()
        assert [exact_code(e, a) for e in row] == list(c)
    assert np.array_equal(scale[:, 0], (np.abs(v).max(1).astype(np.float32) / np.float32(127)))


def test_values_are_within_half_a_step():
    """|value - x| <= a / 254, plus three fp32 roundings (127 / a, a / 127, the value) of at most a."""
    rng = np.random.default_rng(1)
    x = _bits(rng.normal(size=(50, 320)) * np.exp(rng.normal(size=320) * 3))
    codes, scale = O.act8_quantize(x)
    v = O.bf16_bits_to_f64(x).reshape(50, 5, 64)
    a = np.abs(v).max(2, keepdims=True)
    err = np.abs(O.act8_values(codes, scale).astype(np.float64).reshape(v.shape) - v)
    assert np.all(err <= a * (1 / 254 + 3 * 2.0 ** -24))
    top = np.abs(codes.astype(int) - 128).reshape(50, 5, 64).max(2)
    assert np.all(top == 127)                                   # the largest has a code at the end of the range


def test_zero_tiny_and_non_finite_blocks():
    x = np.zeros((1, 64 * 5), np.uint16)
    x[0, 64:128] = 1                                            # 2^-133, the smallest bf16
    x[0, 130] = 0x7F80                                          # +inf
    x[0, 200] = 0xFFC1                                          # NaN
    x[0, 256:] = 0x7F7F                                         # the largest finite value
    codes, scale = O.act8_quantize(x)
    assert scale[0, 0] == 0 and np.all(codes[0, :64] == 128)
    assert np.all(codes[0, 64:128] == 255) and scale[0, 1] > 0
    assert np.isnan(scale[0, 2]) and np.isnan(scale[0, 3]) and np.all(codes[0, 128:256] == 128)
    assert np.all(np.isnan(O.act8_values(codes, scale)[0, 128:256]))
    assert np.all(codes[0, 256:] == 255) and np.isfinite(scale[0, 4])


def _differences(f, x, dx, step=1e-6):
    """d f along each of a few random directions of x, against the gradient dx."""
    rng = np.random.default_rng(5)
    for _ in range(3):
        d = rng.normal(size=x.shape)
        want = (f(x + step * d) - f(x - step * d)) / (2 * step)
        assert np.sum(dx * d) == pytest.approx(want, rel=2e-6, abs=1e-8)


def test_silu_mul_backward_by_differences():
    rng = np.random.default_rng(2)
    g, u, dm = (rng.normal(size=(3, 64)) for _ in range(3))
    dg, du = O.silu_mul_bwd(g, u, dm)
    _differences(lambda v: np.sum(O.silu_mul(v, u) * dm), g, dg)
    _differences(lambda v: np.sum(O.silu_mul(g, v) * dm), u, du)


@pytest.mark.parametrize("post,gated,gained", [(False, None, False), (True, "channel", True), (True, "token", False),
                                               (False, "token", True)])
def test_residual_norm_backward_by_differences(post, gated, gained):
    rng = np.random.default_rng(3)
    t, c = 4, 24
    p = {"h": rng.normal(size=(t, c)), "o": rng.normal(size=(t, c))}
    if post:
        p["post_gain"] = rng.normal(size=c)
    if gated:
        p["gate"] = rng.normal(size=c if gated == "channel" else (t, c))
    if gained:
        p["gain"] = rng.normal(size=c)
    dn, dres = [rng.normal(size=(t, c)) for _ in range(2)], rng.normal(size=(t, c))

    def loss(**change):
        f = O.residual_norm_fwd(**dict(p, **change), post_norm=post, scale=0.3, offset=0.5, eps=1e-3)
        return np.sum(f["n"] * sum(dn)) + np.sum(f["s"] * dres)

    f = O.residual_norm_fwd(**p, post_norm=post, scale=0.3, offset=0.5, eps=1e-3)
    got = O.residual_norm_bwd(dn, f["rstd"], f["s"] * f["rstd"][:, None], dres, p["o"], post, f["rstd_o"], p.get("post_gain"),
                              p.get("gate"), 0.3, p.get("gain"), 0.5)
    for name, grad in (("h", "dh"), ("o", "do"), ("post_gain", "dpost_gain"), ("gate", "dgate"), ("gain", "dgain")):
        if name in p:
            d = got[grad].sum(0) if grad == "dgate" and gated == "channel" else got[grad]
            _differences(lambda v: loss(**{name: v}), p[name], d)


def test_stack_backward_with_exact_checkpoints_is_the_plain_one():
    """With checkpoints that keep every value, the stack's backward differs from decoder_backward's only in
    which sums are rounded to bf16 (the projections' gradients before a norm) and in n taken for h / rms
    (its rounding): a few steps of 2^-9 in quadrature on the way through two layers."""
    dims = O.StackLayerDims(128, 128, 32, 256, 32)
    rng = np.random.default_rng(6)
    shapes = {"q": (128, 128), "k": (32, 128), "v": (32, 128), "o": (128, 128), "gate": (256, 128), "up": (256, 128),
              "down": (128, 256)}
    layers = [{n: (_bits(0.08 * rng.normal(size=s)), _bits(rng.normal(size=(8, s[1])) * 0.1), _bits(rng.normal(size=(s[0], 8)) * 0.05))
               for n, s in shapes.items()} for _ in range(2)]
    h0, dh = _bits(rng.normal(size=(9, 128))), _bits(rng.normal(size=(9, 128)))
    pos, inv = np.arange(9), 1e6 ** (-np.arange(0, 32, 2) / 32)
    _, saved = O.decoder_forward(h0, layers, dims, 16.0, pos, inv)
    want, grads = O.decoder_backward(dh, layers, dims, 16.0, saved, pos, inv)
    got, grads8 = O.decoder_backward_act8(dh, layers, dims, 16.0, saved, pos, inv, keep=lambda x: np.asarray(x, np.float64))
    assert O.rel_l2(got, want) <= 8 * 2.0 ** -9
    for a, b in zip(grads8, grads):
        for key in b:
            assert O.rel_l2(a[key], b[key]) <= 8 * 2.0 ** -9, key


@pytest.mark.parametrize("a", [range(0x3F80, 0x4000), range(0x0001, 0x0480)])
def test_values_within_the_stated_bound(a):
    """|value - x| <= a / 254 + 2^-23 |value| over every largest a of one binade beside every bf16 value down to
    code 0, and over every a up to past where the step a / 127 is a normal fp32 number (a = 127 2^-126) beside every
    value below it: there the step's own rounding, by up to 2^-150, adds at most 127 of those."""
    passed = 0
    for top in a:
        x = np.arange(max(0, top - 10 * 128), top + 1).astype(np.uint16)
        blocks = np.zeros((-(-len(x) // 63), 64), np.uint16)
        blocks[:, 0] = top
        blocks[:, 1:].flat[:len(x)] = x
        codes, scale = O.act8_quantize(blocks)
        v, got = O.bf16_bits_to_f64(blocks), O.act8_values(codes, scale).astype(np.float64)
        largest = v[0, 0]
        err = np.abs(got - v) - (largest / 254 * (1 + 2.0 ** -50) + 2.0 ** -23 * np.abs(got))
        if largest >= 127 * 2.0 ** -126:
            assert np.all(err <= 0)
        else:
            assert np.all(err <= 127 * 2.0 ** -150)
            passed += bool(np.any(err > 0))
    assert (passed > 0) == (a[0] == 1)                            # the addition is needed, and for subnormal steps alone
