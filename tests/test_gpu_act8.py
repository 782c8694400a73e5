"""Activations in 8 bits through the C ABI: the codec bit for bit, the SiLU product element by
element against the fp64 oracle, and the linear's backward against fp64 and the bf16 call."""

import numpy as np
import pytest
import torch

import oracle as O
import synthetic_inputs as S
from helpers import bits_of, check_bf16_output, check_linear, half_ulp_bf16, linear_mags, to_dev_bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def _bits(a):
    return S.to_bf16_bits(a)


def _rows(t, c, seed=0):
    """Rows whose blocks differ in size by many powers of two."""
    rng = np.random.default_rng([t, c, seed])
    return _bits(rng.normal(size=(t, c)) * np.exp(2 * rng.normal(size=(t, c // 64))).repeat(64, axis=1))


def _act8(lib, bits):
    codes, scale = O.act8_quantize(bits)
    return lib.Act8(torch.from_numpy(codes).cuda(), torch.from_numpy(scale).cuda())


def _same(got, want):
    """Equal bit for bit, but for which NaN."""
    a, b = got.cpu(), torch.from_numpy(np.ascontiguousarray(want))
    if a.dtype == torch.float32:
        nan = torch.isnan(b)
        assert torch.equal(torch.isnan(a), nan)
        a, b = a.masked_fill(nan, 0).view(torch.int32), b.masked_fill(nan, 0).view(torch.int32)
    assert torch.equal(a, b)


@pytest.mark.parametrize("t,c", [(1, 64), (1, 3584), (3, 128), (40, 256), (7, 192), (513, 1088), (2, 29568), (1000, 64)])
def test_codec_equals_oracle(gpu_lib, t, c):
    lib, x = gpu_lib, _rows(t, c)
    got = lib.act8_quantize(to_dev_bf16(x))
    codes, scale = O.act8_quantize(x)
    _same(got.codes, codes)
    _same(got.scale, scale)
    back = lib.act8_dequantize(got)
    assert np.array_equal(bits_of(back), _bits(O.act8_values(codes, scale)))


def test_codec_every_bf16_value(gpu_lib):
    """Every bit pattern as its block's largest beside a half, a ramp of it, zeros and the other sign; blocks
    with infinities and NaNs; blocks of tiny and subnormal values."""
    lib = gpu_lib
    x = np.zeros((65536, 64), np.uint16)
    x[:, 0] = np.arange(65536)
    with np.errstate(all="ignore"):
        v = O.bf16_bits_to_f64(x[:, 0])
        ramp = np.where(np.isfinite(v), v, 1.0)[:, None] * np.linspace(-1, 1, 62)
    x[:, 1:63] = _bits(ramp)
    got = lib.act8_quantize(to_dev_bf16(x))
    codes, scale = O.act8_quantize(x)
    _same(got.codes, codes)
    _same(got.scale, scale)
    back = lib.act8_dequantize(got)
    want = torch.from_numpy(O.act8_values(codes, scale)).to(torch.bfloat16)
    assert torch.equal(torch.isnan(back.cpu()), torch.isnan(want))
    fine = ~torch.isnan(want)
    assert torch.equal(back.cpu()[fine], want[fine])


def test_codec_ties_go_to_even(gpu_lib):
    """A largest of 127 * 2^k makes steps of 2^k: halves of them are ties."""
    lib = gpu_lib
    x = np.zeros((2, 64))
    x[:, 0] = 127.0
    x[0, 1:] = np.arange(63) + 0.5
    x[1, 1:] = -(np.arange(63) + 0.5)
    codes = lib.act8_quantize(to_dev_bf16(_bits(x))).codes.cpu().numpy().astype(int) - 128
    want = np.rint(np.arange(63) + 0.5)
    assert np.array_equal(codes[0, 1:], want) and np.array_equal(codes[1, 1:], -want)


def _sigmoid_rel(z):
    """Relative error of the kernels' SiLU: the exponent's product (2^-24 |z|, and the constant's own
    2^-25 |z|), exp2 and the reciprocal at 2^-22 each, the sum and two products at 2^-24 each."""
    return (2 * np.abs(z) + 12) * U


def _near(got, want, bound, what):
    err = np.abs(O.bf16_bits_to_f64(bits_of(got)) - want)
    bad = ~(err <= bound + half_ulp_bf16(np.abs(want) + bound))
    assert not bad.any(), (what, int(bad.sum()), float(err[bad].max()), float(np.abs(want[bad]).max()))


def _check_silu(lib, gate, up, dm):
    """All three calls at bf16 bits gate, up, dm."""
    dg, du, dd = (to_dev_bf16(v) for v in (gate, up, dm))
    m, g8, u8 = lib.silu_mul_fwd_act8(dg, du)
    for x8, x in ((g8, gate), (u8, up)):
        codes, scale = O.act8_quantize(x)
        _same(x8.codes, codes)
        _same(x8.scale, scale)
    g, u, d = (O.bf16_bits_to_f64(v) for v in (gate, up, dm))
    tiny = 2.0 ** -125 * (1 + np.abs(g)) * (1 + np.abs(u))       # where the sigmoid passes fp32's range
    want = O.silu_mul(g, u)
    _near(m, want, _sigmoid_rel(g) * np.abs(want) + tiny, "m")
    gv, uv = (O.act8_values(*O.act8_quantize(v)).astype(np.float64) for v in (gate, up))
    again = lib.silu_mul_act8(g8, u8)
    want = O.silu_mul(gv, uv)
    e = _sigmoid_rel(gv)
    _near(again, want, e * np.abs(want) + tiny, "m again")
    dgate, dup = lib.silu_mul_bwd_act8(g8, u8, dd)
    want_g, want_u = O.silu_mul_bwd(gv, uv, d)
    tiny = tiny * (1 + np.abs(d))
    sig = 1 / (1 + np.exp(-gv))
    # s + z s (1 - s): every s off by e of itself, 1 - s by e s and an ulp, each product and sum by one more
    _near(dgate, want_g, np.abs(d * uv) * sig * (1 + 2 * np.abs(gv)) * (e + 4 * U) + tiny, "dgate")
    _near(dup, want_u, (e + 2 * U) * np.abs(want_u) + tiny, "dup")


@pytest.mark.parametrize("t,c", [(1, 64), (40, 256), (17, 704), (300, 1088), (3, 18944)])
def test_silu_product(gpu_lib, t, c):
    rng = np.random.default_rng([t, c])
    _check_silu(gpu_lib, _bits(rng.normal(size=(t, c)) * 3), _bits(rng.normal(size=(t, c))), _bits(rng.normal(size=(t, c)) * 0.1))


def test_silu_product_far_values(gpu_lib):
    """Gates from -100 to 100 (past the exponential's range), a gate of 0, large and small factors."""
    g = np.linspace(-100, 100, 128 * 64).reshape(128, 64)
    g[0, 0] = 0.0
    rng = np.random.default_rng(4)
    _check_silu(gpu_lib, _bits(g), _bits(rng.normal(size=g.shape) * np.exp(rng.normal(size=(128, 1)) * 4)),
                _bits(rng.normal(size=g.shape)))


def test_silu_non_finite_stays_in_its_block(gpu_lib):
    lib = gpu_lib
    g, u, d = (torch.randn(5, 256, device="cuda").to(torch.bfloat16) for _ in range(3))
    ref = lib.silu_mul_fwd_act8(g, u)
    ref_back = lib.silu_mul_bwd_act8(ref[1], ref[2], d)
    g[2, 70], u[4, 255] = float("nan"), float("inf")
    _, g8, u8 = lib.silu_mul_fwd_act8(g, u)
    dgate, dup = lib.silu_mul_bwd_act8(g8, u8, d)
    again = lib.silu_mul_act8(g8, u8)
    hit = torch.zeros(5, 256, dtype=torch.bool, device="cuda")
    hit[2, 64:128] = True
    hit[4, 192:] = True
    assert torch.equal(torch.isnan(again), hit) and torch.equal(torch.isnan(dgate), hit)
    assert torch.equal(dgate[~hit], ref_back[0][~hit])
    hit[4, 192:] = False                                       # dup does not read up
    assert torch.equal(torch.isnan(dup), hit) and torch.equal(dup[~hit], ref_back[1][~hit])


def test_in_place(gpu_lib):
    lib = gpu_lib
    g, u, d = (torch.randn(33, 320, device="cuda").to(torch.bfloat16) for _ in range(3))
    m, g8, u8 = lib.silu_mul_fwd_act8(g, u)
    dgate, dup = lib.silu_mul_bwd_act8(g8, u8, d)
    g2, d2 = g.clone(), d.clone()
    m2, g82, u82 = lib.silu_mul_fwd_act8(g2, u, out=g2)
    assert m2 is g2 and torch.equal(m2, m) and torch.equal(g82.codes, g8.codes) and torch.equal(u82.scale, u8.scale)
    dg2, du2 = lib.silu_mul_bwd_act8(g8, u8, d2, dgate=d2)
    assert dg2 is d2 and torch.equal(dg2, dgate) and torch.equal(du2, dup)


def _linear_inputs(t, n, k, r, seed=0):
    case = S.linear_case(t, n, k, r=r, seed=seed)
    d = {key: to_dev_bf16(case[key]) for key in ("W", "x", "dY", "A", "B")}
    return case, d


LINEARS = [(1, 16, 64, 1), (1, 128, 128, 16), (5, 3584, 512, 16), (17, 256, 704, 5), (32, 1024, 256, 64),
           (33, 128, 192, 8), (34, 16, 64, 1), (200, 48, 64, 64),
           (130, 272, 320, 16), (257, 1104, 1024, 16), (300, 256, 4160, 33), (512, 512, 18944, 16),
           (520, 128, 16512, 40), (1024, 64, 16384, 16), (1030, 1040, 16448, 64)]


def _check_adapter(dA, dB, x, u, case, r, what):
    """dA and dB element by element against fp64 on the same operands (x: what the checkpoint stands for,
    rounded to bf16): sums of exact products of bf16 values and fp32 ones held to 2^-24, so at most one
    rounding of 2^-24 of the terms' magnitudes for each addition (N or T and the shares), each product
    (with s.g and s.u) and each part of an operand: 64 more."""
    dy, b, xv = (O.bf16_bits_to_f64(v) for v in (case["dY"], case["B"], x))
    t, n = dy.shape
    f, u = 32.0 / r, u.astype(np.float64)
    for got, want, mag, terms in ((dA, f * (dy @ b).T @ xv, f * (np.abs(dy) @ np.abs(b)).T @ np.abs(xv), n + t),
                                  (dB, f * dy.T @ u, f * np.abs(dy).T @ np.abs(u), t)):
        err = np.abs(got.cpu().numpy().astype(np.float64) - want)
        assert np.all(err <= (terms + 64) * U * mag), (what, float((err / mag).max() / U))


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("t,n,k,r", LINEARS)
def test_linear_element_by_element(gpu_lib, t, n, k, r, dense):
    """dX, dA and dB against fp64 on the base's and the checkpoint's values, and the same twice."""
    lib = gpu_lib
    case, d = _linear_inputs(t, n, k, r)
    x8 = _act8(lib, case["x"])
    u = torch.randn(t, r, device="cuda")
    if dense:
        base, call, w = (d["W"],), lib.lora_linear_bwd_bf16_act8, d["W"]
    else:
        base, call = lib.quantize(d["W"]), lib.lora_linear_bwd_act8
        w = lib.dequantize(*base)
    values = bits_of(lib.act8_dequantize(x8))
    dx, dA, dB = call(*base, x8, u, d["dY"], d["A"], d["B"], 32.0)
    dy, wv, a, b = (O.bf16_bits_to_f64(v) for v in (case["dY"], bits_of(w), case["A"], case["B"]))
    f = 32.0 / r
    # N additions of dY W or dY B and r of g A; the helper has the slack of s.g in two bf16 parts
    check_bf16_output(bits_of(dx), dy @ wv + f * (dy @ b) @ a, "dx",
                      mag=np.abs(dy) @ np.abs(wv) + f * (np.abs(dy) @ np.abs(b)) @ np.abs(a), terms=n + r)
    _check_adapter(dA, dB, values, u.cpu().numpy(), case, r, "with dx")
    again = call(*base, x8, u, d["dY"], d["A"], d["B"], 32.0)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dA, dB)))
    none, dA, dB = call(*base, x8, u, d["dY"], d["A"], d["B"], 32.0, need_dx=False)
    assert none is None
    _check_adapter(dA, dB, values, u.cpu().numpy(), case, r, "without dx")


@pytest.mark.parametrize("t,n,k,r", [(1, 128, 128, 16), (20, 256, 704, 5), (130, 272, 320, 16), (600, 256, 1088, 16)])
def test_linear_against_oracle(gpu_lib, t, n, k, r):
    lib = gpu_lib
    case, d = _linear_inputs(t, n, k, r, seed=3)
    codes, absmax = lib.quantize(d["W"])
    x8 = lib.act8_quantize(d["x"])
    x = _bits(O.act8_values(*O.act8_quantize(case["x"])))
    w = O.dequantize(*O.quantize(O.bf16_bits_to_f64(case["W"]).astype(np.float32)))
    _, u = O.lora_linear_fwd(x, w, case["A"], case["B"], 32.0)
    dx, dA, dB = lib.lora_linear_bwd_act8(codes, absmax, x8, torch.from_numpy(u.astype(np.float32)).cuda(), d["dY"], d["A"],
                                          d["B"], 32.0)
    refs = dict(zip(("dx", "dA", "dB"), O.lora_linear_bwd(x, w, case["A"], case["B"], 32.0, case["dY"])))
    mags = linear_mags(x, w, case["A"], case["B"], 32.0, case["dY"])
    check_linear({"dx": bits_of(dx), "dA": dA.cpu().numpy(), "dB": dB.cpu().numpy()}, refs, mags, t, n, k, r, "act8")


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("t,n,k", [(3, 64, 192), (33, 128, 320), (140, 1040, 1088), (300, 128, 4160), (1100, 64, 16448)])
def test_linear_writes_nothing_else(gpu_lib, t, n, k, dense):
    """What lies before and behind dX, dA, dB and the workspace stays."""
    lib = gpu_lib
    _, d = _linear_inputs(t, n, k, 16)
    base = (d["W"],) if dense else lib.quantize(d["W"])
    call, ws = ((lib.lora_linear_bwd_bf16_act8, lib.bwd_bf16_act8_workspace_bytes) if dense
                else (lib.lora_linear_bwd_act8, lib.bwd_act8_workspace_bytes))
    u = torch.randn(t, 16, device="cuda")
    x8 = lib.act8_quantize(d["x"])
    want = call(*base, x8, u, d["dY"], d["A"], d["B"], 32.0)
    outs, views = [], []
    for shape, dtype in (((t, k), torch.bfloat16), ((16, k), torch.float32), ((n, 16), torch.float32),
                         ((ws(t, n, k, 16),), torch.uint8)):
        size, pad = int(np.prod(shape)), 1 << 18
        buf = torch.full((size + 2 * pad,), 7, dtype=dtype, device="cuda")
        outs.append((buf, pad, size))
        views.append(buf[pad:pad + size].view(shape))
    call(*base, x8, u, d["dY"], d["A"], d["B"], 32.0, dx=views[0], dA=views[1], dB=views[2], ws=views[3])
    assert all(torch.equal(a, b) for a, b in zip(views, want))
    for buf, pad, size in outs:
        assert torch.all(buf[:pad] == 7) and torch.all(buf[pad + size:] == 7)


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("t", [3, 40, 300])
def test_linear_without_adapter(gpu_lib, t, dense):
    lib = gpu_lib
    case, d = _linear_inputs(t, 256, 128, 16)
    base = (d["W"],) if dense else lib.quantize(d["W"])
    call = lib.lora_linear_bwd_bf16_act8 if dense else lib.lora_linear_bwd_act8
    dx, dA, dB = call(*base, None, None, d["dY"], None, None, 32.0)
    w, dy = O.bf16_bits_to_f64(bits_of(d["W"] if dense else lib.dequantize(*base))), O.bf16_bits_to_f64(case["dY"])
    assert dA is None and dB is None
    check_bf16_output(bits_of(dx), dy @ w, "dx", mag=np.abs(dy) @ np.abs(w), terms=256)


@pytest.mark.parametrize("dense", [False, True])
def test_linear_no_tokens(gpu_lib, dense):
    lib = gpu_lib
    _, d = _linear_inputs(2, 64, 128, 16)
    base = (d["W"],) if dense else lib.quantize(d["W"])
    call = lib.lora_linear_bwd_bf16_act8 if dense else lib.lora_linear_bwd_act8
    dA, dB = torch.full((16, 128), 7.0, device="cuda"), torch.full((64, 16), 7.0, device="cuda")
    dx, dA, dB = call(*base, lib.act8_quantize(d["x"][:0]), torch.zeros(0, 16, device="cuda"), d["dY"][:0], d["A"], d["B"], 32.0,
                      dA=dA, dB=dB)
    assert dx.shape == (0, 128) and not torch.any(dA) and not torch.any(dB)


@pytest.mark.parametrize("t", [3, 40, 300])
def test_checkpoints_at_their_least_alignment(gpu_lib, t):
    """Codes at 16 bytes past 32, scales at 4 bytes past 8: every call that reads or writes them."""
    lib, n, k = gpu_lib, 128, 320

    def off():
        codes = torch.empty(t * k + 16, dtype=torch.uint8, device="cuda")[16:].view(t, k)
        return lib.Act8(codes, torch.empty(t * (k // 64) + 1, device="cuda")[1:].view(t, k // 64))

    _, d = _linear_inputs(t, n, k, 16)
    x, base, u = d["x"], lib.quantize(d["W"]), torch.randn(t, 16, device="cuda")
    x8, y8 = lib.act8_quantize(x), lib.act8_quantize(x, out=off())
    up = torch.randn(t, k, device="cuda").to(torch.bfloat16)
    m = lib.silu_mul_fwd_act8(x, up, gate8=off(), up8=off())
    want = lib.silu_mul_fwd_act8(x, up)
    r, s = lib.residual_norm_fwd(x, up, n8=off()), lib.residual_norm_fwd(x, up, checkpoint=True)
    pairs = list(zip((*y8, lib.act8_dequantize(y8), m[0], *m[1], *m[2], r.n, *r.n8),
                     (*x8, lib.act8_dequantize(x8), want[0], *want[1], *want[2], s.n, *s.n8)))
    pairs += zip((lib.silu_mul_act8(*m[1:]), *lib.silu_mul_bwd_act8(*m[1:], x)),
                 (lib.silu_mul_act8(*want[1:]), *lib.silu_mul_bwd_act8(*want[1:], x)))
    pairs.append((lib.residual_norm_bwd(up, r.rstd, n8=r.n8).dh, lib.residual_norm_bwd(up, s.rstd, n8=s.n8).dh))
    for call, b in ((lib.lora_linear_bwd_act8, base), (lib.lora_linear_bwd_bf16_act8, (d["W"],))):
        args = (u, d["dY"], d["A"], d["B"], 32.0)
        pairs += zip(call(*b, y8, *args), call(*b, x8, *args))
    assert all(torch.equal(p, q) for p, q in pairs)


@pytest.mark.parametrize("dense,n", [(False, 32768), (True, 16368)])
def test_linear_largest_base(gpu_lib, dense, n):
    """The most weights that the call takes: dX's first and last columns, and dA's."""
    lib, t, k = gpu_lib, 40, 65536
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    dy, x = (torch.randn(t, c, generator=g, device="cuda").to(torch.bfloat16) for c in (n, k))
    A, B = (torch.randn(*c, generator=g, device="cuda").to(torch.bfloat16) for c in ((16, k), (n, 16)))
    u, x8 = torch.randn(t, 16, generator=g, device="cuda"), lib.act8_quantize(x)
    if dense:
        base = (torch.randn(n, k, generator=g, device="cuda", dtype=torch.bfloat16),)
        call = lib.lora_linear_bwd_bf16_act8
    else:
        base = (torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8),
                torch.rand(n, k // 64, generator=g, device="cuda"))
        call = lib.lora_linear_bwd_act8
    dx, dA, dB = call(*base, x8, u, dy, A, B, 32.0)
    values = lib.act8_dequantize(x8)
    d64, b64 = dy.double().cpu().numpy(), B.double().cpu().numpy()
    for at in (0, k - 64):
        w = base[0][:, at:at + 64] if dense else lib.dequantize(base[0][:, at // 2:at // 2 + 32].contiguous(),
                                                                 base[1][:, at // 64:at // 64 + 1].contiguous())
        wv, a = w.double().cpu().numpy(), A[:, at:at + 64].double().cpu().numpy()
        check_bf16_output(bits_of(dx[:, at:at + 64].contiguous()), d64 @ wv + 2 * (d64 @ b64) @ a, "dx",
                          mag=np.abs(d64) @ np.abs(wv) + 2 * (np.abs(d64) @ np.abs(b64)) @ np.abs(a), terms=n + 16)
        xv = values[:, at:at + 64].double().cpu().numpy()
        mag = 2 * (np.abs(d64) @ np.abs(b64)).T @ np.abs(xv)
        err = np.abs(dA[:, at:at + 64].double().cpu().numpy() - 2 * (d64 @ b64).T @ xv)
        assert np.all(err <= (n + t + 64) * U * mag)


def test_linear_non_finite_block_reaches_its_columns(gpu_lib):
    lib = gpu_lib
    for t in (7, 200):
        case, d = _linear_inputs(t, 128, 256, 16)
        codes, absmax = lib.quantize(d["W"])
        x = d["x"].clone()
        x[t // 2, 130] = float("inf")
        u = torch.randn(t, 16, device="cuda")
        dx, dA, dB = lib.lora_linear_bwd_act8(codes, absmax, lib.act8_quantize(x), u, d["dY"], d["A"], d["B"], 32.0)
        ref = lib.lora_linear_bwd_act8(codes, absmax, lib.act8_quantize(d["x"]), u, d["dY"], d["A"], d["B"], 32.0)
        nan = torch.isnan(dA)
        assert torch.all(nan[:, 128:192]) and not torch.any(nan[:, :128]) and not torch.any(nan[:, 192:])
        assert torch.equal(dx, ref[0]) and torch.equal(dB, ref[2])


def test_rows_past_32_bits(gpu_lib):
    """A matrix of 2^32 + 2^16 elements: the last rows equal a call on them alone."""
    lib, c = gpu_lib, 1 << 16
    t = (1 << 16) + 1
    x = torch.zeros(t, c, dtype=torch.bfloat16, device="cuda")
    x[-3:] = torch.randn(3, c, device="cuda").to(torch.bfloat16)
    x8 = lib.act8_quantize(x)
    want = lib.act8_quantize(x[-3:].clone())
    assert torch.equal(x8.codes[-3:], want.codes) and torch.equal(x8.scale[-3:], want.scale)
    back = lib.act8_dequantize(x8, out=x)
    assert torch.equal(back[-3:], lib.act8_dequantize(want))
    del x, back
    dm = torch.zeros(t, c, dtype=torch.bfloat16, device="cuda")
    dm[-3:] = 1.0
    dgate, dup = lib.silu_mul_bwd_act8(x8, x8, dm, dgate=dm)
    ref = lib.silu_mul_bwd_act8(want, want, torch.ones(3, c, dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(dgate[-3:], ref[0]) and torch.equal(dup[-3:], ref[1])


def test_no_rows(gpu_lib):
    lib = gpu_lib
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    x8 = lib.act8_quantize(x)
    assert x8.codes.shape == (0, 128) and x8.scale.shape == (0, 2)
    m, g8, u8 = lib.silu_mul_fwd_act8(x, x)
    assert m.shape == lib.act8_dequantize(x8).shape == lib.silu_mul_act8(g8, u8).shape == (0, 128)
    assert [v.shape for v in lib.silu_mul_bwd_act8(g8, u8, x)] == [(0, 128)] * 2


def test_refusals(gpu_lib):
    lib = gpu_lib
    x = torch.randn(8, 128, device="cuda").to(torch.bfloat16)
    x8 = lib.act8_quantize(x)
    with pytest.raises(ValueError, match="contiguous"):
        lib.act8_quantize(x[:, :64])
    with pytest.raises(ValueError, match="contiguous"):
        lib.act8_dequantize(lib.Act8(x8.codes[:, :64], x8.scale[:, :1].contiguous()))
    with pytest.raises(TypeError, match="bfloat16"):
        lib.act8_quantize(x.float())
    with pytest.raises(lib.Nf4Error, match="multiple of 64"):
        lib.act8_quantize(torch.zeros(4, 100, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(lib.Nf4Error, match="aligned"):
        lib.act8_quantize(torch.zeros(8 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 64))
    with pytest.raises(ValueError, match="shape"):
        lib.act8_dequantize(lib.Act8(x8.codes, x8.scale[:4]))
    with pytest.raises(ValueError, match="shape"):
        lib.silu_mul_act8(x8, lib.act8_quantize(x[:4]))
    with pytest.raises(lib.Nf4Error, match="overlaps"):
        lib.silu_mul_fwd_act8(x, x, gate8=x8, up8=x8)
    with pytest.raises(TypeError, match="Act8"):
        lib.lora_linear_bwd_act8(*lib.quantize(x), x, None, x[:, :8].contiguous(), x[:1], x[:, :1], 1.0)


def _step(lib, s):
    m, g8, u8 = lib.silu_mul_fwd_act8(s["g"], s["u"], out=s["m"], gate8=s["g8"], up8=s["u8"])
    lib.silu_mul_act8(g8, u8, out=s["m2"])
    lib.silu_mul_bwd_act8(g8, u8, s["dm"], dgate=s["dg"], dup=s["du"])
    lib.act8_quantize(s["m2"], out=s["m8"])
    lib.lora_linear_bwd_act8(s["codes"], s["absmax"], s["m8"], s["lu"], s["dy"], s["A"], s["B"], 32.0, dx=s["dx"], dA=s["dA"],
                             dB=s["dB"], ws=s["ws"])


def _step_state(lib, t, c, n, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    s = {"g": normal(t, c), "u": normal(t, c), "dm": normal(t, c), "dy": normal(t, n), "A": normal(16, c), "B": normal(n, 16)}
    s.update({key: torch.empty(t, c, dtype=torch.bfloat16, device="cuda") for key in ("m", "m2", "dg", "du", "dx")})
    s.update({key: lib.act8_empty(t, c) for key in ("g8", "u8", "m8")})
    s["codes"], s["absmax"] = lib.quantize(normal(n, c))
    s["lu"] = torch.randn(t, 16, generator=g, device="cuda")
    s["dA"], s["dB"] = torch.empty(16, c, device="cuda"), torch.empty(n, 16, device="cuda")
    s["ws"] = lib.workspace(lib.bwd_act8_workspace_bytes(t, n, c, 16))
    return s


OUTS = ("m", "m2", "dg", "du", "dx", "dA", "dB")


@pytest.mark.parametrize("t", [3, 150, 700])
def test_graph_replays_equal_eager(gpu_lib, t):
    """Two graphs captured over buffers of their own, replayed in turn with eager work between."""
    lib = gpu_lib
    states = [_step_state(lib, t, 320, 256, seed) for seed in (1, 2)]
    refs, graphs = [], []
    for s in states:
        _step(lib, s)
        torch.cuda.synchronize()
        refs.append({key: s[key].clone() for key in OUTS})
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _step(lib, s)
        graphs.append(graph)
    for _ in range(3):
        for s in states:
            for key in OUTS:
                s[key].fill_(7.0)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for s, ref in zip(states, refs):
            for key in OUTS:
                assert torch.equal(s[key], ref[key]), key


def test_other_stream(gpu_lib):
    """On a stream given by argument: ordered with that stream's work, allocating that stream's memory."""
    lib = gpu_lib
    x = torch.randn(2000, 1024, device="cuda").to(torch.bfloat16)
    want = lib.act8_dequantize(lib.act8_quantize(x))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        y = x.clone()
    got = lib.act8_dequantize(lib.act8_quantize(y, stream=side), stream=side)
    side.synchronize()
    assert torch.equal(got, want)


def test_calls_that_no_cache_holds(gpu_lib):
    """Codec and SiLU product of more than 256 MB, whose inputs are loaded past the caches: every row's results are those of a
    call on some of the rows."""
    lib, t, c = gpu_lib, 12900, 7040
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    gate, up, dm = (torch.randn(t, c, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3))
    m, g8, u8 = lib.silu_mul_fwd_act8(gate, up)
    again, back = lib.silu_mul_act8(g8, u8), lib.silu_mul_bwd_act8(g8, u8, dm)
    values = lib.act8_dequantize(u8, out=torch.empty_like(up))
    for at in range(0, t, 600):
        def part(x):
            return x[at:at + 600].contiguous()

        n, p8, q8 = lib.silu_mul_fwd_act8(part(gate), part(up))
        pairs = [(n, m), *zip(p8, g8), *zip(q8, u8), (lib.silu_mul_act8(p8, q8), again), (lib.act8_dequantize(q8), values)]
        pairs += zip(lib.silu_mul_bwd_act8(p8, q8, part(dm)), back)
        assert all(torch.equal(x, y[at:at + 600]) for x, y in pairs), at
