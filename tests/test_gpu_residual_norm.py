"""The residual add fused with the norms around a block, through the C ABI against the fp64 oracle,
element by element, and its gradients against the oracle's, which differences pin."""

import numpy as np
import pytest
import torch

import oracle as O
import synthetic_inputs as S
from helpers import bits_of, half_ulp_bf16, to_dev_bf16

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
# fp32 roundings on the way to a result, as units of 2^-24 of the sum of the magnitudes it is formed
# from. A row's mean: at most 32 additions in a thread, 6 between lanes, 15 between waves, and a
# product and two roundings of its terms: 56. An inverse root of it: half that, two roundings and the
# mean's product: 32. A forward result: such a root and at most 8 products and sums: 48. A gradient:
# three sums of dn, a mean and two roots with their products: 160. All doubled.
FWD, BWD = 96 * U, 320 * U


def _bits(a):
    return S.to_bf16_bits(a)


def _case(t, c, post, gate, gain, offset=0.0, dns=1, seed=0):
    rng = np.random.default_rng([t, c, post, len(gate), gain, dns, seed])
    channels = np.exp(0.7 * rng.normal(size=c))
    p = {"h": _bits(rng.normal(size=(t, c)) * channels), "o": _bits(1.5 * rng.normal(size=(t, c)))}
    p["post_gain"] = _bits(rng.normal(size=c) + 1 - offset) if post else None
    p["gate"] = {"none": None, "channel": _bits(rng.normal(size=c)), "token": _bits(rng.normal(size=(t, c)))}[gate]
    p["gain"] = _bits(rng.normal(size=c) + 1 - offset) if gain else None
    p["dn"] = [_bits(rng.normal(size=(t, c))) for _ in range(dns)]
    p["dres"] = _bits(rng.normal(size=(t, c)))
    return p


def _dev(v):
    return None if v is None else to_dev_bf16(v)


def _abs(v):
    return None if v is None else np.abs(O.bf16_bits_to_f64(v) if v.dtype == np.uint16 else v)


def _near(got, want, bound, what):
    f32 = got.dtype == torch.float32
    v = got.cpu().numpy().astype(np.float64) if f32 else O.bf16_bits_to_f64(bits_of(got))
    reach = np.abs(want) + bound
    err, room = np.abs(v - want), bound + (U * reach if f32 else half_ulp_bf16(reach))
    bad = ~(err <= room)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.size} off; worst {float((err - room).max()):.3e} over the bound"


def _check_fwd(lib, p, post, scale, offset, eps=1e-6, block=True, dev=None, **kw):
    d = {n: _dev(p[n]) for n in ("h", "o", "post_gain", "gate", "gain")} if dev is None else dev
    r = lib.residual_norm_fwd(d["h"], d["o"] if block else None, post_norm=post, post_gain=d["post_gain"],
                              gate=d["gate"] if block else None, scale=scale, gain=d["gain"], gain_offset=offset, eps=eps, **kw)
    torch.cuda.synchronize()
    args = dict(post_norm=post, post_gain=p["post_gain"], gate=p["gate"] if block else None, scale=scale, gain=p["gain"],
                offset=offset, eps=eps)
    want = O.residual_norm_fwd(p["h"], p["o"] if block else None, **args)
    h = O.bf16_bits_to_f64(p["h"])
    v = want["s"] - h                                          # what the block adds
    ds = FWD * np.abs(v) + U * (np.abs(h) + np.abs(v))
    if block:
        _near(r.h, want["s"], ds, "h")
    else:
        assert r.h is d["h"]
    # the root's error, and what the stream's own errors move it by
    rel = FWD + np.linalg.norm(ds, axis=1) / np.maximum(np.linalg.norm(want["s"], axis=1), 1e-300)
    _near(r.rstd, want["rstd"], rel * want["rstd"], "rstd")
    if post:
        _near(r.rstd_o, want["rstd_o"], FWD * want["rstd_o"], "rstd_o")
    f = np.abs(1.0 if p["gain"] is None else O.bf16_bits_to_f64(p["gain"]) + offset)
    _near(r.n, want["n"], rel[:, None] * np.abs(want["n"]) + ds * want["rstd"][:, None] * f, "n")
    return r


def _check_bwd(lib, p, post, scale, offset, block=True, act8=False, dev=None, dres=True, **kw):
    t, c = p["h"].shape
    h = O.bf16_bits_to_f64(p["h"])
    rstd = (1 / np.sqrt(np.mean(h * h, axis=1) + 1e-6)).astype(np.float32)
    o = O.bf16_bits_to_f64(p["o"])
    rstd_o = (1 / np.sqrt(np.mean(o * o, axis=1) + 1e-6)).astype(np.float32) if post else None
    if act8:
        codes, step = O.act8_quantize(_bits(h * rstd[:, None].astype(np.float64)))
        b = O.act8_values(codes, step).astype(np.float64)
        stream = {"n8": lib.Act8(torch.from_numpy(codes).cuda(), torch.from_numpy(step).cuda())}
    else:
        b = h * rstd[:, None].astype(np.float64)
        stream = {"h": _dev(p["h"]) if dev is None else dev["h"]}
    d = {n: _dev(p[n]) for n in ("o", "post_gain", "gate", "gain", "dres")} if dev is None else dev
    dn = [_dev(x) for x in p["dn"]] if dev is None else dev["dn"]
    r = lib.residual_norm_bwd(dn if len(dn) > 1 else dn[0], torch.from_numpy(rstd).cuda(), **stream,
                              dres=d["dres"] if dres else None, o=d["o"] if block else None, post_norm=post,
                              rstd_o=None if rstd_o is None else torch.from_numpy(rstd_o).cuda(), post_gain=d["post_gain"],
                              gate=d["gate"] if block else None, scale=scale, gain=d["gain"], gain_offset=offset, **kw)
    torch.cuda.synchronize()
    gate = p["gate"] if block else None
    want = O.residual_norm_bwd(p["dn"], rstd, b, p["dres"] if dres else None, p["o"] if block else None, post, rstd_o,
                               p["post_gain"], gate, scale, p["gain"], offset)
    # the same sums over magnitudes
    f = np.abs(1.0 if p["gain"] is None else O.bf16_bits_to_f64(p["gain"]) + offset)
    g, rs = sum(_abs(x) for x in p["dn"]), rstd[:, None].astype(np.float64)
    ds = rs * (g * f + np.abs(b) * np.mean(g * f * np.abs(b), axis=1, keepdims=True)) + (_abs(p["dres"]) if dres else 0)
    _near(r.dh, want["dh"], BWD * ds, "dh")
    down = BWD + (t + 4) * U                                     # sums over rows
    if p["gain"] is not None and kw.get("param_grads", True):
        _near(r.dgain, want["dgain"], down * np.sum(g * np.abs(b), axis=0), "dgain")
    else:
        assert r.dgain is None
    if not block:
        assert r.do is None and r.dgate is None and r.dpost_gain is None
        return r
    dv, u = abs(scale) * ds, np.abs(o) * (rstd_o[:, None].astype(np.float64) if post else 1.0)
    pf = np.abs(1.0 if p["post_gain"] is None else O.bf16_bits_to_f64(p["post_gain"]) + offset)
    x = dv * u * pf
    if gate is None or not kw.get("param_grads", True):
        assert r.dgate is None
    elif gate.ndim == 1:
        _near(r.dgate, want["dgate"].sum(0), down * x.sum(0), "dgate")
    else:
        _near(r.dgate, want["dgate"], BWD * x, "dgate")
    if gate is not None:
        dv = dv * _abs(gate)
    if p["post_gain"] is not None and kw.get("param_grads", True):
        _near(r.dpost_gain, want["dpost_gain"], down * np.sum(dv * u, axis=0), "dpost_gain")
    else:
        assert r.dpost_gain is None
    if post:
        dv = rstd_o[:, None] * (dv * pf + u * np.mean(dv * pf * u, axis=1, keepdims=True))
    _near(r.do, want["do"], BWD * dv, "do")
    return r


WIDTHS = [1, 2, 7, 8, 63, 64, 65, 511, 512, 520, 1001, 2048, 2056, 3583, 3584, 4097, 8191, 8192, 8200, 16383, 16384]
FORMS = [(False, "none", False, 0.0), (True, "none", True, 1.0), (True, "channel", True, 0.0), (False, "token", True, 1.0),
         (True, "token", False, 0.0), (False, "channel", False, 0.0)]


@pytest.mark.parametrize("c", WIDTHS)
def test_forward_widths(gpu_lib, c):
    for i, (post, gate, gain, offset) in enumerate(FORMS):
        t = (1, 5, 3)[i % 3]
        _check_fwd(gpu_lib, _case(t, c, post, gate, gain, offset), post, (1.0, 0.3)[i % 2], offset)
    _check_fwd(gpu_lib, _case(6, c, False, "none", True, 0.0), False, 1.0, 0.0, block=False)


@pytest.mark.parametrize("c", WIDTHS)
def test_backward_widths(gpu_lib, c):
    for i, (post, gate, gain, offset) in enumerate(FORMS):
        t = (1, 5, 3)[i % 3]
        p = _case(t, c, post, gate, gain, offset, dns=1 + i % 3)
        _check_bwd(gpu_lib, p, post, (1.0, 0.3)[i % 2], offset, dres=i != 1)
        _check_bwd(gpu_lib, p, post, 0.5, offset, param_grads=False)
    for gain in (False, True):
        _check_bwd(gpu_lib, _case(6, c, False, "none", gain, 0.0, dns=3), False, 1.0, 0.0, block=False)


@pytest.mark.parametrize("t,c", [(2, 256), (257, 384), (700, 264), (513, 3584), (1100, 1000), (300, 8192)])
def test_many_rows(gpu_lib, t, c):
    """More rows than workgroups that sum over them; ragged counts."""
    for post, gate, gain, offset in ((True, "channel", True, 1.0), (False, "token", True, 0.0), (False, "none", False, 0.0)):
        p = _case(t, c, post, gate, gain, offset, dns=2)
        _check_fwd(gpu_lib, p, post, 0.5, offset)
        _check_bwd(gpu_lib, p, post, 0.5, offset)


@pytest.mark.parametrize("t,c", [(1, 64), (3, 128), (40, 576), (9, 2048), (70, 3584), (5, 8192), (3, 16384)])
def test_checkpoint_of_the_normalised_stream(gpu_lib, t, c):
    """The forward's checkpoint is act8_quantize's of its n, bit for bit; the backward reads it."""
    lib = gpu_lib
    for block, gain in ((True, False), (False, False), (True, True)):
        p = _case(t, c, False, "none", gain)
        r = _check_fwd(lib, p, False, 0.7, 0.0, block=block, checkpoint=True)
        want = lib.act8_quantize(r.n)
        assert torch.equal(r.n8.codes, want.codes) and torch.equal(r.n8.scale, want.scale)
    for dns in (1, 2, 3):
        _check_bwd(lib, _case(t, c, False, "none", False, dns=dns), False, 1.0, 0.0, block=dns != 2, act8=True)
    _check_bwd(lib, _case(t, c, True, "channel", False), True, 0.5, 0.0, act8=True)


@pytest.mark.parametrize("c", [64, 1000, 4096])
def test_tensors_off_16_byte_alignment(gpu_lib, c):
    lib, t = gpu_lib, 7
    p = _case(t, c, True, "token", True, dns=2)

    def shifted(v):
        flat = torch.empty(v.size + 1, dtype=torch.bfloat16, device="cuda")
        flat[1:] = _dev(v).flatten()
        return flat[1:].view(v.shape)

    dev = {n: shifted(p[n]) for n in ("h", "o", "post_gain", "gate", "gain", "dres")}
    dev["dn"] = [shifted(x) for x in p["dn"]]
    a = _check_fwd(lib, p, True, 0.5, 0.0, dev=dev)
    b = _check_fwd(lib, p, True, 0.5, 0.0)
    assert torch.equal(a.h, b.h) and torch.equal(a.n, b.n) and torch.equal(a.rstd, b.rstd)
    a, b = _check_bwd(lib, p, True, 0.5, 0.0, dev=dev), _check_bwd(lib, p, True, 0.5, 0.0)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_plain_residual_equals_add_and_norm(gpu_lib):
    """Without post norm, gate and scale h_out is the add's bits, and the norm alone has unit gain's."""
    lib = gpu_lib
    h, o = (torch.randn(33, 896, device="cuda").to(torch.bfloat16) for _ in range(2))
    r = lib.residual_norm_fwd(h, o)
    assert torch.equal(r.h, lib.add_bf16(h, o)) and r.n8 is None and r.rstd_o is None
    n, rstd = lib.rmsnorm_fwd(h)
    alone = lib.residual_norm_fwd(h)
    assert alone.h is h and torch.allclose(alone.rstd, rstd, rtol=1e-6)
    # equal but where a last-bit difference of rstd moves a rounding: a step at most
    assert torch.all((alone.n.float() - n.float()).abs() <= 2.0 ** -7 * n.float().abs())
    dn, dres = (torch.randn(33, 896, device="cuda").to(torch.bfloat16) for _ in range(2))
    g = lib.residual_norm_bwd(dn, r.rstd, h=r.h, dres=dres, o=o)
    assert torch.equal(g.dh, g.do)


def test_in_place(gpu_lib):
    lib = gpu_lib
    p = _case(50, 1032, True, "token", True, dns=2)
    d = {n: _dev(p[n]) for n in ("h", "o", "post_gain", "gate", "gain", "dres")}
    kw = dict(post_norm=True, post_gain=d["post_gain"], gate=d["gate"], scale=0.5, gain=d["gain"])
    r = lib.residual_norm_fwd(d["h"], d["o"], **kw)
    h, o = d["h"].clone(), d["o"].clone()
    q = lib.residual_norm_fwd(h, o, h_out=h, n=o, **kw)
    assert q.h is h and torch.equal(h, r.h) and torch.equal(o, r.n) and torch.equal(q.rstd, r.rstd)
    dn = [_dev(x) for x in p["dn"]]
    back = dict(kw, h=r.h, rstd=r.rstd, rstd_o=r.rstd_o)
    g = lib.residual_norm_bwd(dn, dres=d["dres"], o=d["o"], **back)
    dres, o = d["dres"].clone(), d["o"].clone()
    k = lib.residual_norm_bwd(dn, dres=dres, o=o, dh=dres, do=o, **back)
    assert k.dh is dres and k.do is o and all(torch.equal(x, y) for x, y in zip(k, g))
    k = lib.residual_norm_bwd(dn, dres=d["dres"], o=d["o"], dh=dn[0], do=dn[1], **back)
    assert torch.equal(k.dh, g.dh) and torch.equal(k.do, g.do)


@pytest.mark.parametrize("c", [5, 100, 333, 1001, 4099, 8191])
def test_in_place_odd_widths(gpu_lib, c):
    """Rows whose last octet is not whole, several a workgroup, results over their inputs."""
    lib, t = gpu_lib, 3000
    h, o, d, e = (torch.randn(t, c, device="cuda").to(torch.bfloat16) for _ in range(4))
    gate = torch.randn(t, c, device="cuda").to(torch.bfloat16)
    want = lib.residual_norm_fwd(h, o, post_norm=True, gate=gate)
    h2, o2 = h.clone(), o.clone()
    got = lib.residual_norm_fwd(h2, o2, post_norm=True, gate=gate, h_out=h2, n=o2)
    assert all(torch.equal(getattr(got, n), getattr(want, n)) for n in ("h", "n", "rstd", "rstd_o"))
    args = dict(h=want.h, dres=e, post_norm=True, rstd_o=want.rstd_o, gate=gate)
    ref = lib.residual_norm_bwd(d, want.rstd, o=o, **args)
    d2, o2 = d.clone(), o.clone()
    g = lib.residual_norm_bwd(d2, want.rstd, o=o2, dh=d2, do=o2, **args)
    assert torch.equal(g.dh, ref.dh) and torch.equal(g.do, ref.do) and torch.equal(g.dgate, ref.dgate)


def test_non_finite_rows_stay_alone(gpu_lib):
    lib = gpu_lib
    p = _case(9, 192, True, "token", False)
    d = {n: _dev(p[n]) for n in ("h", "o", "post_gain", "gate", "dres")}
    kw = dict(post_norm=True, post_gain=d["post_gain"], gate=d["gate"])
    ref = lib.residual_norm_fwd(d["h"], d["o"], checkpoint=True, **kw)
    h = d["h"].clone()
    h[3, 100], h[8, 0] = float("inf"), float("nan")
    got = lib.residual_norm_fwd(h, d["o"], checkpoint=True, **kw)
    ok = torch.ones(9, dtype=torch.bool, device="cuda")
    ok[3] = ok[8] = False
    assert torch.equal(got.n[ok], ref.n[ok]) and torch.equal(got.n8.codes[ok], ref.n8.codes[ok])
    assert torch.isnan(got.n[8]).all() and torch.isnan(got.n[3, 100]) and torch.isnan(got.n8.scale[8]).all()
    dn = _dev(p["dn"][0])
    a = lib.residual_norm_bwd(dn, ref.rstd, n8=ref.n8, dres=d["dres"], o=d["o"], rstd_o=ref.rstd_o, **kw)
    dn[3, 5] = float("nan")
    b = lib.residual_norm_bwd(dn, ref.rstd, n8=ref.n8, dres=d["dres"], o=d["o"], rstd_o=ref.rstd_o, **kw)
    ok[8] = True
    assert torch.equal(a.dh[ok], b.dh[ok]) and torch.equal(a.do[ok], b.do[ok]) and torch.isnan(b.dh[3]).all()


def test_zero_rows_and_large_values(gpu_lib):
    """A row of zeros gives zeros (eps keeps the root finite); values whose squares pass fp32's range give
    an infinite mean, a root of zero and zeros."""
    lib = gpu_lib
    h = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    h[1] = 1e25
    h[2] = 1e-30
    r = lib.residual_norm_fwd(h, checkpoint=True)
    assert torch.all(r.n[:2] == 0) and r.rstd[1] == 0 and torch.all(r.n8.codes[:2] == 128)
    assert r.rstd[0].item() == pytest.approx(1e3, rel=1e-6) and torch.allclose(r.n[2].float(), torch.tensor(1e-27, device="cuda"), rtol=0.01)


def test_no_rows(gpu_lib):
    lib = gpu_lib
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    v = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    r = lib.residual_norm_fwd(x, x, post_norm=True, post_gain=v, gate=v, gain=v)
    assert r.n.shape == (0, 128) and r.rstd.shape == (0,)
    g = lib.residual_norm_bwd([x, x], r.rstd, h=x, o=x, post_norm=True, rstd_o=r.rstd_o, post_gain=v, gate=v, gain=v)
    for s in (g.dgain, g.dpost_gain, g.dgate):
        assert s.shape == (128,) and torch.all(s == 0)


@pytest.mark.parametrize("block", [False, True])
def test_more_rows_than_workgroups(gpu_lib, block):
    """A row a workgroup, and past 2^21 of them: each takes several, in registers of their own."""
    lib, t, c = gpu_lib, (1 << 21) + 77, 520
    h = torch.randn(1, c, device="cuda").to(torch.bfloat16).repeat(t, 1)
    h[-80:] = torch.randn(80, c, device="cuda").to(torch.bfloat16)
    o = h if block else None
    r = lib.residual_norm_fwd(h, o, scale=0.5)
    for rows in (slice(0, 64), slice(-80, None)):
        want = lib.residual_norm_fwd(h[rows].contiguous(), h[rows].contiguous() if block else None, scale=0.5)
        assert torch.equal(r.n[rows], want.n) and torch.equal(r.rstd[rows], want.rstd) and torch.equal(r.h[rows], want.h)
    assert torch.equal(r.n[:-80].amax(0), r.n[0]) and torch.equal(r.n[:-80].amin(0), r.n[0])
    g = lib.residual_norm_bwd(r.n, r.rstd, h=r.h)
    for rows in (slice(0, 64), slice(-80, None)):
        want = lib.residual_norm_bwd(r.n[rows].contiguous(), r.rstd[rows].contiguous(), h=r.h[rows].contiguous())
        assert torch.equal(g.dh[rows], want.dh)
    assert torch.equal(g.dh[:-80].amax(0), g.dh[0]) and torch.equal(g.dh[:-80].amin(0), g.dh[0])


@pytest.mark.parametrize("t,c", [(5, 64), (130, 576), (40, 4096), (3, 12288)])
def test_checkpoint_beside_tensors_off_alignment(gpu_lib, t, c):
    """bf16 tensors at 2 bytes past 16, the checkpoint aligned: the same results."""
    lib = gpu_lib

    def off(x):
        return torch.cat([torch.zeros(1, dtype=x.dtype, device="cuda"), x.flatten()])[1:].view(x.shape)

    h, o, d = (torch.randn(t, c, device="cuda").to(torch.bfloat16) for _ in range(3))
    want = lib.residual_norm_fwd(h, o, post_norm=True, checkpoint=True)
    got = lib.residual_norm_fwd(off(h), off(o), post_norm=True, checkpoint=True, n=off(torch.empty_like(h)))
    for a, b in zip((got.h, got.n, *got.n8, got.rstd, got.rstd_o), (want.h, want.n, *want.n8, want.rstd, want.rstd_o)):
        assert torch.equal(a, b)
    want = lib.residual_norm_bwd(d, want.rstd, n8=want.n8, dres=h, o=o, post_norm=True, rstd_o=want.rstd_o)
    got = lib.residual_norm_bwd(off(d), got.rstd, n8=got.n8, dres=off(h), o=off(o), post_norm=True, rstd_o=got.rstd_o)
    assert torch.equal(got.dh, want.dh) and torch.equal(got.do, want.do)


def test_rows_past_32_bits(gpu_lib):
    """270000 rows of 16384 (over 8 GiB): the last rows equal a call on them alone."""
    lib, t, c, n = gpu_lib, 270000, 16384, 5
    h = torch.zeros(t, c, dtype=torch.bfloat16, device="cuda")
    h[-n:] = torch.randn(n, c, device="cuda").to(torch.bfloat16)
    tail = h[-n:].clone()
    want = lib.residual_norm_fwd(tail, checkpoint=True)
    r = lib.residual_norm_fwd(h, checkpoint=True)
    assert torch.equal(r.n[-n:], want.n) and torch.equal(r.n8.codes[-n:], want.n8.codes)
    assert torch.equal(r.n8.scale[-n:], want.n8.scale) and torch.equal(r.rstd[-n:], want.rstd)
    g = lib.residual_norm_bwd(h, r.rstd, n8=r.n8, dh=r.n)
    assert torch.equal(g.dh[-n:], lib.residual_norm_bwd(tail, want.rstd, n8=want.n8).dh)
    gain = torch.ones(c, dtype=torch.bfloat16, device="cuda")
    g = lib.residual_norm_bwd(h, r.rstd, h=h, gain=gain, dh=r.n)
    k = lib.residual_norm_bwd(tail, want.rstd, h=tail, gain=gain)
    assert torch.equal(g.dh[-n:], k.dh) and torch.allclose(g.dgain, k.dgain, rtol=1e-5)


def test_repeats_and_graph_replays(gpu_lib):
    """Calls repeat bit for bit; two captured graphs with workspaces of their own, replayed in turn."""
    lib = gpu_lib
    t, c = 700, 1032
    cases = []
    for seed in (1, 2):
        p = _case(t, c, True, "channel", True, dns=3, seed=seed)
        d = {n: _dev(p[n]) for n in ("h", "o", "post_gain", "gate", "gain", "dres")}
        d["dn"] = [_dev(x) for x in p["dn"]]
        d["ws"] = lib.workspace(lib.residual_norm_bwd_workspace_bytes(t, c))
        cases.append(d)

    def step(d):
        kw = dict(post_norm=True, post_gain=d["post_gain"], gate=d["gate"], scale=0.5, gain=d["gain"])
        r = lib.residual_norm_fwd(d["h"], d["o"], **kw)
        g = lib.residual_norm_bwd(d["dn"], r.rstd, h=r.h, dres=d["dres"], o=d["o"], rstd_o=r.rstd_o, ws=d["ws"], **kw)
        return [x for x in (*r, *g) if x is not None]

    refs = [[x.clone() for x in step(d)] for d in cases]
    assert all(torch.equal(a, b) for a, b in zip(step(cases[0]), refs[0]))
    graphs, outs = [], []
    for d in cases:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(step(d))
        graphs.append(graph)
    for _ in range(3):
        for x in (*outs[0], *outs[1]):
            x.fill_(3.0)
        step(cases[1])                                            # eager work between the replays
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for out, ref in zip(outs, refs):
            assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_other_stream(gpu_lib):
    lib = gpu_lib
    h, o = (torch.randn(900, 2048, device="cuda").to(torch.bfloat16) for _ in range(2))
    gain = torch.randn(2048, device="cuda").to(torch.bfloat16)
    want = lib.residual_norm_fwd(h, o, gain=gain)
    ref = lib.residual_norm_bwd(h, want.rstd, h=want.h, gain=gain)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = lib.residual_norm_fwd(h, o, gain=gain, stream=side)
    back = lib.residual_norm_bwd(h, got.rstd, h=got.h, gain=gain, stream=side)
    side.synchronize()
    assert torch.equal(got.n, want.n) and torch.equal(back.dh, ref.dh) and torch.equal(back.dgain, ref.dgain)


def test_refusals(gpu_lib):
    lib = gpu_lib
    with pytest.raises(TypeError, match="gate"):
        lib.residual_norm_fwd(torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"),
                              torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda"), gate=0.5)
    h = torch.randn(8, 128, device="cuda").to(torch.bfloat16)
    v = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    rstd = torch.ones(8, device="cuda")
    for kw, match in (({"post_norm": True}, "block's output"), ({"gate": v}, "block's output"), ({"h_out": h}, "block's output"),
                      ({"post_gain": v}, "post_norm"), ({"gain": h}, "shape"), ({"gain": v[:64]}, "shape"),
                      ({"o": h[:4]}, "shape"), ({"o": h, "gate": h[:1]}, "shape"), ({"o": h.t().contiguous().t()}, "contiguous")):
        with pytest.raises(ValueError, match=match):
            lib.residual_norm_fwd(h, **kw)
    with pytest.raises(TypeError, match="bfloat16"):
        lib.residual_norm_fwd(h, gain=v.float())
    with pytest.raises(lib.Nf4Error, match="16384"):
        lib.residual_norm_fwd(torch.zeros(1, 16392, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(lib.Nf4Error, match="multiple of 64"):
        x = torch.zeros(2, 100, dtype=torch.bfloat16, device="cuda")
        lib.residual_norm_fwd(x, n8=lib.Act8(torch.empty(2, 100, dtype=torch.uint8, device="cuda"), torch.empty(2, 1, device="cuda")))
    with pytest.raises(lib.Nf4Error, match="overlaps"):
        lib.residual_norm_fwd(h, h.clone(), h_out=h, n=h)
    n8 = lib.act8_quantize(h)
    for kw, match in (({}, "h or as n8"), ({"h": h, "n8": n8}, "h or as n8"), ({"n8": n8, "gain": v}, "without a gain"),
                      ({"h": h, "gate": v}, "block's output"), ({"h": h, "do": h}, "block's output"),
                      ({"h": h, "post_norm": True}, "block's output"), ({"h": h, "dgain": rstd}, "not asked for"),
                      ({"h": h, "o": h, "dgate": h}, "not asked for")):
        with pytest.raises(ValueError, match=match):
            lib.residual_norm_bwd(h, rstd, **kw)
    with pytest.raises(ValueError, match="one to three"):
        lib.residual_norm_bwd([h] * 4, rstd, h=h)
    with pytest.raises(TypeError, match="rstd_o"):
        lib.residual_norm_bwd(h, rstd, h=h, o=h, post_norm=True)


@pytest.mark.parametrize("t,c", [(300, 8200), (520, 12288), (300, 16383), (400, 7001), (700, 1001), (1100, 333)])
def test_many_rows_of_wide_and_odd_widths(gpu_lib, t, c):
    """Several rows a workgroup where the sums over them lie in LDS and the gains are read again for each row (above 8192),
    and where rows are ragged: the next row's loads under way, gains kept packed."""
    for post, gate, gain, offset in ((True, "token", True, 1.0), (True, "channel", True, 0.0), (False, "token", True, 0.0),
                                     (False, "channel", False, 0.0)):
        p = _case(t, c, post, gate, gain, offset, dns=3)
        _check_fwd(gpu_lib, p, post, 0.5, offset)
        _check_bwd(gpu_lib, p, post, 0.5, offset)
        _check_bwd(gpu_lib, p, post, 0.5, offset, param_grads=False, dres=False)
    _check_bwd(gpu_lib, _case(t, c, False, "none", True, 1.0, dns=3), False, 1.0, 1.0, block=False)


@pytest.mark.parametrize("trained", [True, False])
@pytest.mark.parametrize("t,c", [(5300, 5120), (6600, 5119), (2700, 10240)])
def test_calls_that_no_cache_holds(gpu_lib, t, c, trained):
    """Forward and backward of more than 256 MB, whose inputs are loaded past the caches: every row's results are those
    of a call on some of the rows."""
    lib = gpu_lib
    g = torch.Generator(device="cuda")
    g.manual_seed(c)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    h, o, gate, dres = (normal(t, c) for _ in range(4))
    dn = [normal(t, c) for _ in range(3)]
    params = dict(post_norm=True, post_gain=normal(c), gain=normal(c), gain_offset=1.0, scale=0.5)
    fwd = lib.residual_norm_fwd(h, o, gate=gate, checkpoint=c % 64 == 0, **params)
    back = lib.residual_norm_bwd(dn, fwd.rstd, h=fwd.h, dres=dres, o=o, rstd_o=fwd.rstd_o, gate=gate, param_grads=trained, **params)
    sums = torch.zeros(2, c, dtype=torch.float64, device="cuda")
    for at in range(0, t, 500):
        def part(x):
            return x[at:at + 500].contiguous()

        f = lib.residual_norm_fwd(part(h), part(o), gate=part(gate), checkpoint=c % 64 == 0, **params)
        pairs = [(f.h, fwd.h), (f.n, fwd.n), (f.rstd, fwd.rstd), (f.rstd_o, fwd.rstd_o)]
        pairs += list(zip(f.n8 or (), fwd.n8 or ()))
        b = lib.residual_norm_bwd([part(d) for d in dn], f.rstd, h=f.h, dres=part(dres), o=part(o), rstd_o=f.rstd_o,
                                  gate=part(gate), param_grads=trained, **params)
        pairs += [(b.dh, back.dh), (b.do, back.do)] + ([(b.dgate, back.dgate)] if trained else [])
        assert all(torch.equal(x, y[at:at + 500]) for x, y in pairs), at
        if trained:
            sums += torch.stack([b.dgain, b.dpost_gain]).double()
    if trained:
        # both sides sum the same rounded products, with at most t additions in fp32 on either
        u = o.double() * fwd.rstd_o.double()[:, None]
        mag = [(sum(d.double().abs() for d in dn) * fwd.h.double().abs() * fwd.rstd.double()[:, None]).sum(0)]
        w = sum(d.double() for d in dn) * (params["gain"].double() + 1)
        b = fwd.h.double() * fwd.rstd.double()[:, None]
        ds = dres.double() + fwd.rstd.double()[:, None] * (w - b * (w * b).mean(1, keepdim=True))
        mag.append((0.5 * ds.abs() * gate.double().abs() * u.abs()).sum(0) * 1.01)      # the kernel's ds is off by far less
        for got, want, m in zip((back.dgain, back.dpost_gain), sums, mag):
            assert torch.all((got.double() - want).abs() <= 2 * t * U * m)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("c", [7, 515, 1001, 1032, 4099, 8200, 12291])
def test_results_over_either_input(gpu_lib, c, post):
    """h_out over o and n over h as well as the other way round, plain adds (whose stream is stored before any sum of the
    row) too; one gradient given for all readers, and dh or do over it."""
    lib, t = gpu_lib, 700
    h, o, gate, d, e = (torch.randn(t, c, device="cuda").to(torch.bfloat16) for _ in range(5))
    kw = dict(post_norm=post, gate=gate, scale=0.5)
    want = lib.residual_norm_fwd(h, o, **kw)
    for swap in (False, True):
        h2, o2 = h.clone(), o.clone()
        got = lib.residual_norm_fwd(h2, o2, h_out=o2 if swap else h2, n=h2 if swap else o2, **kw)
        assert all(torch.equal(getattr(got, n), getattr(want, n)) for n in ("h", "n", "rstd"))
    back = dict(kw, h=want.h, rstd_o=want.rstd_o, dres=e, param_grads=False)
    ref = lib.residual_norm_bwd([d.clone(), d.clone(), d.clone()], want.rstd, o=o, **back)
    for dh, do in ((True, False), (False, True)):
        d2 = d.clone()
        g = lib.residual_norm_bwd([d2, d2, d2], want.rstd, o=o, dh=d2 if dh else None, do=d2 if do else None, **back)
        assert torch.equal(g.dh, ref.dh) and torch.equal(g.do, ref.do)
