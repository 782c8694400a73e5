"""Host-side argument checks of the 8-bit checkpoints' and the residual norms' entry points, without
a GPU: every call fails (or is a no-op) before anything reaches the device."""

import ctypes as C

import pytest
import torch

A0 = 0x1000000          # aligned addresses far apart, never dereferenced
STEP = 0x1000000


def at(i, off=0):
    return C.c_void_p(A0 + i * STEP + off)


@pytest.fixture(scope="module")
def L():
    from nf4_weight_streamed_amd import lib

    return lib


def _err(L, rc, code, needle):
    assert rc == code and needle in L.last_error(), (rc, L.last_error())


def _calls(L):
    """name -> (call(rows, cols, pointers), pointers: (kind, input?))."""
    raw = L.raw()
    return {
        "quantize": (lambda t, c, p: raw.nf4_act8_quantize(p[0], t, c, p[1], p[2], None), ["x", "C", "S"]),
        "dequantize": (lambda t, c, p: raw.nf4_act8_dequantize(p[0], p[1], t, c, p[2], None), ["c", "s", "X"]),
        "silu_fwd": (lambda t, c, p: raw.nf4_silu_mul_fwd_act8(p[0], p[1], t, c, *p[2:], None),
                     ["x", "x", "X", "C", "S", "C", "S"]),
        "silu": (lambda t, c, p: raw.nf4_silu_mul_act8(*p[:4], t, c, p[4], None), ["c", "s", "c", "s", "X"]),
        "silu_bwd": (lambda t, c, p: raw.nf4_silu_mul_bwd_act8(*p[:5], t, c, *p[5:], None),
                     ["c", "s", "c", "s", "x", "X", "X"]),
    }


@pytest.mark.parametrize("name", ["quantize", "dequantize", "silu_fwd", "silu", "silu_bwd"])
def test_elementwise_validation(L, name):
    call, kinds = _calls(L)[name]
    good = [at(i) for i in range(len(kinds))]
    for t, c in ((-1, 64), (4, 0), (4, -64), (4, 63), (4, 100), (1, 1 << 35), (1 << 30, 64), (1 << 62, 1 << 62)):
        _err(L, call(t, c, good), L.NF4_E_SHAPE, "nf4_")
    assert call(0, 64, [None] * len(kinds)) == 0
    for i, kind in enumerate(kinds):
        _err(L, call(4, 128, good[:i] + [None] + good[i + 1:]), L.NF4_E_ARG, "NULL")
        off = 2 if kind in "sS" else 8
        _err(L, call(4, 128, good[:i] + [at(i, off)] + good[i + 1:]), L.NF4_E_ARG, "aligned")
        if kind.isupper():
            for j in range(len(kinds)):
                # a little way into another argument; the whole of a bf16 input is no overlap
                if j != i:
                    _err(L, call(4, 128, good[:i] + [at(j, 16)] + good[i + 1:]), L.NF4_E_ARG, "overlaps")
                    if not (kind == "X" and kinds[j] == "x"):
                        _err(L, call(4, 128, good[:i] + [at(j)] + good[i + 1:]), L.NF4_E_ARG, "overlaps")


def test_linear_validation(L):
    raw = L.raw()

    def nf4(x=at(0), s=at(1), N=128, K=128, T=4, r=16, ws=at(5), ws_bytes=1 << 30):
        return raw.nf4_lora_linear_bwd_act8(at(8), at(9), N, K, x, s, at(2), at(3), T, at(6), at(7), r, 32.0, at(10), at(11),
                                            at(12), ws, ws_bytes, None)

    def dense(x=at(0), s=at(1), N=128, K=128, T=4, r=16, ws=at(5), ws_bytes=1 << 30):
        return raw.nf4_lora_linear_bwd_bf16_act8(at(8), N, K, x, s, at(2), at(3), T, at(6), at(7), r, 32.0, at(10), at(11),
                                                 at(12), ws, ws_bytes, None)

    for call, need in ((nf4, L.bwd_act8_workspace_bytes), (dense, L.bwd_bf16_act8_workspace_bytes)):
        _err(L, call(K=100), L.NF4_E_SHAPE, "K=100")
        _err(L, call(N=100), L.NF4_E_SHAPE, "N=100")
        _err(L, call(T=(1 << 23) + 1), L.NF4_E_SHAPE, "T")
        _err(L, call(r=65), L.NF4_E_ARG, "r=65")
        _err(L, call(x=None), L.NF4_E_ARG, "needs x")
        _err(L, call(s=None), L.NF4_E_ARG, "needs x")
        _err(L, call(x=at(0, 8)), L.NF4_E_ARG, "aligned")
        _err(L, call(s=at(1, 2)), L.NF4_E_ARG, "aligned")
        assert call(T=0, x=None) == 0
        n = need(512, 3584, 3584, 16)
        _err(L, call(N=3584, K=3584, T=512, ws_bytes=n - 1), L.NF4_E_ARG, str(n))
        _err(L, call(ws=None), L.NF4_E_ARG, "workspace")


FWD = dict(h=at(0), o=at(1), T=4, H=128, post=1, post_gain=at(2), kind=1, gate=at(3), scale=0.5, gain=at(4), offset=0.0,
           eps=1e-6, h_out=at(5), n=at(6), codes=at(7), step=at(8), rstd_o=at(9), rstd=at(10))


def _fwd(L, **kw):
    return L.raw().nf4_residual_norm_fwd(*dict(FWD, **kw).values(), None)


def test_residual_norm_forward_validation(L):
    for kw in ({"T": -1}, {"T": (1 << 23) + 1}, {"H": 0}, {"H": 16385}, {"H": -8}):
        _err(L, _fwd(L, **kw), L.NF4_E_SHAPE, "16384")
    _err(L, _fwd(L, H=100), L.NF4_E_SHAPE, "checkpoint")
    _err(L, _fwd(L, post=2), L.NF4_E_ARG, "post_norm")
    _err(L, _fwd(L, kind=3), L.NF4_E_ARG, "gate_kind")
    _err(L, _fwd(L, kind=0), L.NF4_E_ARG, "gate")
    _err(L, _fwd(L, gate=None), L.NF4_E_ARG, "gate")
    _err(L, _fwd(L, post=0), L.NF4_E_ARG, "post_gain")
    for bad in (float("inf"), float("nan")):
        _err(L, _fwd(L, scale=bad), L.NF4_E_ARG, "scale")
        _err(L, _fwd(L, offset=bad), L.NF4_E_ARG, "gain_offset")
        _err(L, _fwd(L, eps=bad), L.NF4_E_ARG, "eps")
    _err(L, _fwd(L, eps=-1e-9), L.NF4_E_ARG, "eps")
    _err(L, _fwd(L, o=None), L.NF4_E_ARG, "block's output")
    _err(L, _fwd(L, o=None, post=0, post_gain=None, kind=0, gate=None), L.NF4_E_ARG, "h_out")
    _err(L, _fwd(L, codes=None), L.NF4_E_ARG, "go together")
    _err(L, _fwd(L, step=None), L.NF4_E_ARG, "go together")
    for name in ("h", "h_out", "n", "rstd_o", "rstd"):
        _err(L, _fwd(L, **{name: None}), L.NF4_E_ARG, "non-NULL")
    for i, name in enumerate(("h", "o", "post_gain", "gate", "gain", "h_out", "n")):
        _err(L, _fwd(L, **{name: at(20 + i, 1)}), L.NF4_E_ARG, "aligned")
    _err(L, _fwd(L, codes=at(7, 8)), L.NF4_E_ARG, "n_codes")
    _err(L, _fwd(L, rstd=at(10, 2)), L.NF4_E_ARG, "rstd")
    for name in ("h_out", "n", "codes", "step", "rstd_o", "rstd"):
        for j in range(11):
            if FWD[name].value != A0 + j * STEP:
                p = at(j, 2 if name in ("h_out", "n") else 0)
                if (name, j) not in (("h_out", 0), ("h_out", 1), ("n", 0), ("n", 1)):
                    _err(L, _fwd(L, **{name: p}), L.NF4_E_ARG, "overlaps")
    _err(L, _fwd(L, h_out=at(0, 2)), L.NF4_E_ARG, "overlaps")
    _err(L, _fwd(L, n=at(0), h_out=at(0)), L.NF4_E_ARG, "overlaps")
    assert _fwd(L, T=0, h=None, n=None) == 0


BWD = dict(dn=None, n_dn=2, dres=at(2), h=at(3), codes=None, step=None, rstd=at(6), o=at(7), rstd_o=at(8), T=4, H=128, post=1,
           post_gain=at(9), kind=1, gate=at(10), scale=0.5, gain=at(11), offset=1.0, dh=at(12), do=at(13), dgate=at(14),
           dpost_gain=at(15), dgain=at(16), ws=at(17), ws_bytes=1 << 23)


def _bwd(L, dns=None, **kw):
    a = dict(BWD, **kw)
    dns = [at(0), at(1), at(20)] if dns is None else dns
    a["dn"] = (C.c_void_p * len(dns))(*[d.value if d else None for d in dns])
    return L.raw().nf4_residual_norm_bwd(*a.values(), None)


def test_residual_norm_backward_validation(L):
    for kw in ({"T": -1}, {"T": (1 << 23) + 1}, {"H": 0}, {"H": 16385}):
        _err(L, _bwd(L, **kw), L.NF4_E_SHAPE, "16384")
    for n in (0, 4, -1):
        _err(L, _bwd(L, n_dn=n), L.NF4_E_ARG, "dn")
    _err(L, _bwd(L, post=2), L.NF4_E_ARG, "post_norm")
    _err(L, _bwd(L, kind=-1), L.NF4_E_ARG, "gate_kind")
    _err(L, _bwd(L, gate=None), L.NF4_E_ARG, "gate")
    _err(L, _bwd(L, kind=0, gate=None), L.NF4_E_ARG, "dgate")
    _err(L, _bwd(L, post=0), L.NF4_E_ARG, "post_gain")
    _err(L, _bwd(L, post_gain=None), L.NF4_E_ARG, "dpost_gain")
    _err(L, _bwd(L, gain=None), L.NF4_E_ARG, "dgain")
    _err(L, _bwd(L, scale=float("nan")), L.NF4_E_ARG, "scale")
    _err(L, _bwd(L, h=None), L.NF4_E_ARG, "exactly one")
    _err(L, _bwd(L, codes=at(4), step=at(5)), L.NF4_E_ARG, "exactly one")
    _err(L, _bwd(L, h=None, codes=at(4)), L.NF4_E_ARG, "go together")
    _err(L, _bwd(L, h=None, codes=at(4), step=at(5)), L.NF4_E_ARG, "without a gain")
    _err(L, _bwd(L, h=None, codes=at(4), step=at(5), gain=None, dgain=None, H=100), L.NF4_E_SHAPE, "checkpoint")
    _err(L, _bwd(L, dns=[at(0), None]), L.NF4_E_ARG, "dn")
    for name in ("rstd", "o", "rstd_o", "dh"):
        _err(L, _bwd(L, **{name: None}), L.NF4_E_ARG, "non-NULL")
    for i, name in enumerate(("dres", "h", "o", "post_gain", "gate", "gain", "dh", "do")):
        _err(L, _bwd(L, **{name: at(30 + i, 1)}), L.NF4_E_ARG, "aligned")
    need = L.residual_norm_bwd_workspace_bytes(4, 128)
    assert need >= 3 * 128 * 4 and need % 256 == 0
    _err(L, _bwd(L, ws_bytes=need - 1), L.NF4_E_ARG, str(need))
    _err(L, _bwd(L, ws=None), L.NF4_E_ARG, "workspace")
    _err(L, _bwd(L, ws=at(17, 16)), L.NF4_E_ARG, "256-byte")
    places = {"dres": 2, "h": 3, "rstd": 6, "o": 7, "rstd_o": 8, "post_gain": 9, "gate": 10, "gain": 11, "dh": 12, "do": 13,
              "dgate": 14, "dpost_gain": 15, "dgain": 16, "ws": 17}
    for name in ("dh", "do", "dgate", "dpost_gain", "dgain", "ws"):
        for other, j in places.items():
            if other != name and (name, other) not in (("dh", "dres"), ("do", "o")):
                _err(L, _bwd(L, **{name: at(j)}), L.NF4_E_ARG, "overlaps")
    for name in ("dh", "do"):
        _err(L, _bwd(L, **{name: at(1, 16)}), L.NF4_E_ARG, "overlaps")
    _err(L, _bwd(L, do=at(2)), L.NF4_E_ARG, "overlaps")
    assert L.residual_norm_bwd_workspace_bytes(0, 128) == 0 and L.residual_norm_bwd_workspace_bytes(4, 128, False) == 0
    assert L.residual_norm_bwd_workspace_bytes(4, 0) == 0 and L.residual_norm_bwd_workspace_bytes(4, 16385) == 0


def test_binding_refusals(L):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    a = L.Act8(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(4, 2))
    with pytest.raises(ValueError, match="GPU"):
        L.act8_quantize(x)
    with pytest.raises(ValueError, match="2-D"):
        L.act8_quantize(x[0])
    with pytest.raises(TypeError, match="torch.Tensor"):
        L.act8_quantize([1.0])
    with pytest.raises(TypeError, match="Act8"):
        L.act8_dequantize(x)
    with pytest.raises(TypeError, match="Act8"):
        L.silu_mul_act8((a.codes, a.scale), a)
    with pytest.raises(ValueError, match="GPU"):
        L.silu_mul_bwd_act8(a, a, x)
    with pytest.raises(ValueError, match="GPU"):
        L.residual_norm_fwd(x)
    with pytest.raises(ValueError, match="one to three"):
        L.residual_norm_bwd([], torch.zeros(4))


@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("T", [4, 128])
def test_linear_refuses_overlaps(L, dense, T):
    """No output of the linear may share memory with an input or another output: not dx with dy either, whose rows
    other tiles still read."""
    raw, N, K, r = L.raw(), 128, 128, 16
    names = ("x", "s", "u", "dy", "A", "B", "dx", "dA", "dB", "ws", "base") + (() if dense else ("absmax",))
    good = {n: at(i) for i, n in enumerate(names)}
    call = raw.nf4_lora_linear_bwd_bf16_act8 if dense else raw.nf4_lora_linear_bwd_act8
    need = (L.bwd_bf16_act8_workspace_bytes if dense else L.bwd_act8_workspace_bytes)(T, N, K, r)

    def run(rank=r, **kw):
        p = dict(good, **kw)
        base = (p["base"],) if dense else (p["base"], p["absmax"])
        return call(*base, N, K, p["x"], p["s"], p["u"], p["dy"], T, p["A"], p["B"], rank, 32.0, p["dx"], p["dA"], p["dB"],
                    p["ws"], need, None)

    for name in ("dx", "dA", "dB", "ws"):
        for i, other in enumerate(names):
            if other != name:
                _err(L, run(**{name: at(i)}), L.NF4_E_ARG, "overlaps")
                if name != "ws":
                    _err(L, run(**{name: at(i, 16)}), L.NF4_E_ARG, "overlaps")
    # the last bytes of the one before
    _err(L, run(dx=C.c_void_p(good["dy"].value + T * N * 2 - 16)), L.NF4_E_ARG, "dx overlaps")
    _err(L, run(dx=C.c_void_p(good["dy"].value - T * K * 2 + 16)), L.NF4_E_ARG, "dx overlaps")
    # without adapters the rest takes no part
    _err(L, run(rank=0, x=None, s=None, u=None, A=None, B=None, dA=None, dB=None, dx=good["dy"]), L.NF4_E_ARG, "dx overlaps")
