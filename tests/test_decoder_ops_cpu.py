"""Host-side argument checks of the decoder operators' C ABI, without a GPU: every call
fails (or is a no-op) before anything reaches the device."""

import ctypes as C
from types import SimpleNamespace

import pytest

FAKE = C.c_void_p(0x10000)      # aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    from nf4_weight_streamed_amd import lib

    return lib


def _err(L, rc, code, needle):
    assert rc == code and needle in L.last_error(), (rc, L.last_error())


def _fwd(L, q=FAKE, T=4, hq=4, hkv=2, D=64, cu=None, n=0, causal=1, scale=0.125, o=FAKE, lse=FAKE):
    return L.raw().nf4_attn_fwd(q, FAKE, FAKE, T, hq, hkv, D, cu, n, causal, scale, o, lse, None)


def _bwd(L, q=FAKE, T=4, hq=4, hkv=2, D=64, cu=None, n=0, causal=1, scale=0.125, do=FAKE, ws=FAKE, ws_bytes=1 << 40):
    return L.raw().nf4_attn_bwd(q, FAKE, FAKE, FAKE, FAKE, do, T, hq, hkv, D, cu, n, causal, scale, FAKE, FAKE, FAKE, ws,
                                ws_bytes, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_attention_validation(L, call):
    for D in (0, 16, 48, 96, 256):
        _err(L, call(L, D=D), L.NF4_E_SHAPE, "head_dim")
    for kw in ({"T": -1}, {"T": (1 << 23) + 1}, {"hq": 5}, {"hkv": 0}, {"hq": 0}, {"hq": 2048}, {"hq": -4, "hkv": -2}):
        _err(L, call(L, **kw), L.NF4_E_SHAPE, "hkv | hq")
    for kw in ({"n": 2}, {"n": -1}, {"cu": FAKE, "n": 0}, {"cu": FAKE, "n": (1 << 20) + 1}):
        _err(L, call(L, **kw), L.NF4_E_SHAPE, "n_seqs")
    _err(L, call(L, causal=2), L.NF4_E_ARG, "causal")
    for scale in (0.0, -1.0, float("inf"), float("nan")):
        _err(L, call(L, scale=scale), L.NF4_E_ARG, "scale")
    _err(L, call(L, cu=C.c_void_p(0x10002), n=1), L.NF4_E_ARG, "cu_seqlens")
    _err(L, call(L, q=None), L.NF4_E_ARG, "NULL")
    _err(L, call(L, q=C.c_void_p(0x10008)), L.NF4_E_ARG, "aligned")
    assert call(L, T=0, q=None) == 0


def test_attention_output_and_workspace_validation(L):
    _err(L, _fwd(L, o=None), L.NF4_E_ARG, "NULL")
    _err(L, _fwd(L, lse=None), L.NF4_E_ARG, "lse")
    _err(L, _bwd(L, do=C.c_void_p(0x10002)), L.NF4_E_ARG, "aligned")
    need = L.attn_bwd_workspace_bytes(512, 28, 4, 128)
    assert need >= 512 * 28 * 4 and need % 256 == 0
    _err(L, _bwd(L, T=512, hq=28, hkv=4, D=128, ws_bytes=need - 1), L.NF4_E_ARG, str(need))
    _err(L, _bwd(L, ws=None), L.NF4_E_ARG, "workspace")
    _err(L, _bwd(L, ws=C.c_void_p(0x10010)), L.NF4_E_ARG, "256-byte")
    assert L.attn_bwd_workspace_bytes(512, 28, 4, 100) == 0 and L.attn_bwd_workspace_bytes(0, 4, 4, 64) == 0
    assert L.attn_bwd_workspace_bytes(512, 5, 2, 64) == 0


def test_attention_overlaps_are_refused(L):
    """Ranges of T=4, hq=4, hkv=2, D=64: q, o and their gradients 2048 bytes, k and v 1024, lse 64."""
    at = lambda i: C.c_void_p(0x100000 + 0x10000 * i)
    lib = L.raw()

    def fwd(o=at(3), lse=at(4), cu=at(5)):
        return lib.nf4_attn_fwd(at(0), at(1), at(2), 4, 4, 2, 64, cu, 1, 1, 0.125, o, lse, None)

    for kw in ({"o": at(0)}, {"o": at(1)}, {"o": C.c_void_p(at(2).value + 1008)}, {"lse": at(3)}, {"lse": at(0)},
               {"lse": C.c_void_p(at(5).value + 4)}):
        _err(L, fwd(**kw), L.NF4_E_ARG, "overlaps")

    def bwd(dq=at(6), dk=at(7), dv=at(8), ws=at(9)):
        return lib.nf4_attn_bwd(at(0), at(1), at(2), at(3), at(4), at(5), 4, 4, 2, 64, at(11), 1, 1, 0.125, dq, dk, dv, ws,
                                0x10000, None)

    for kw in ({"dq": at(0)}, {"dq": at(5)}, {"dk": at(8)}, {"dk": at(1)}, {"dv": at(2)}, {"dv": at(4)}, {"ws": at(6)},
               {"dk": C.c_void_p(at(6).value + 2032)}, {"ws": at(3)}, {"dv": at(11)}):
        _err(L, bwd(**kw), L.NF4_E_ARG, "overlaps")


def test_more_workgroups_than_a_grid_holds_are_refused(L):
    """2^23 rows of 1024 heads: 2^26 workgroups of 256 threads and more (tensors of terabytes)."""
    lib, T, big = L.raw(), 1 << 23, 1 << 44
    at = [C.c_void_p(big * (i + 1)) for i in range(10)]
    rc = lib.nf4_attn_fwd(at[0], at[1], at[2], T, 1024, 1024, 64, None, 0, 1, 0.125, at[3], at[4], None)
    _err(L, rc, L.NF4_E_SHAPE, "workgroups")
    rc = lib.nf4_attn_bwd(at[0], at[1], at[2], at[3], at[4], at[5], T, 1024, 1024, 64, None, 0, 1, 0.125, at[6], at[7], at[8],
                          at[9], 1 << 43, None)
    _err(L, rc, L.NF4_E_SHAPE, "workgroups")


def test_rope_overlaps_are_refused(L):
    at = lambda i: C.c_void_p(0x100000 + 0x10000 * i)
    sections = (C.c_int * 1)(32)

    def rope(q_out=at(0), k_out=at(1)):
        return L.raw().nf4_rope(at(0), at(1), 4, 4, 2, 64, at(2), at(3), sections, 1, 0, q_out, k_out, None)

    for kw in ({"q_out": at(1)}, {"q_out": C.c_void_p(at(0).value + 16)}, {"k_out": C.c_void_p(at(1).value - 16)},
               {"k_out": at(0)}, {"q_out": at(4), "k_out": at(4)}, {"q_out": at(2)}, {"k_out": at(3)}):
        _err(L, rope(**kw), L.NF4_E_ARG, "overlaps")


def _rope(L, q=FAKE, k=FAKE, T=4, hq=4, hkv=2, D=64, pos=FAKE, inv=FAKE, sections=(32,), n=None, inverse=0, out=FAKE):
    arr = None if sections is None else (C.c_int * max(1, len(sections)))(*sections)
    return L.raw().nf4_rope(q, k, T, hq, hkv, D, pos, inv, arr, len(sections or ()) if n is None else n, inverse, out,
                            out, None)


def test_rope_validation(L):
    for kw in ({"T": -1}, {"T": (1 << 23) + 1}, {"hq": -1}, {"hkv": 1025}):
        _err(L, _rope(L, **kw), L.NF4_E_SHAPE, "T")
    for D in (0, 8, 40, 272):
        _err(L, _rope(L, D=D), L.NF4_E_SHAPE, "head_dim")
    _err(L, _rope(L, sections=None, n=1), L.NF4_E_ARG, "sections")
    _err(L, _rope(L, sections=(8,) * 5), L.NF4_E_ARG, "n_axes=5")
    _err(L, _rope(L, sections=()), L.NF4_E_ARG, "n_axes=0")
    _err(L, _rope(L, sections=(33, -1)), L.NF4_E_ARG, "section 1")
    _err(L, _rope(L, sections=(16, 15)), L.NF4_E_ARG, "31 pairs")
    _err(L, _rope(L, inverse=2), L.NF4_E_ARG, "inverse")
    _err(L, _rope(L, k=None), L.NF4_E_ARG, "NULL")
    _err(L, _rope(L, out=C.c_void_p(0x10008)), L.NF4_E_ARG, "aligned")
    _err(L, _rope(L, pos=None), L.NF4_E_ARG, "pos")
    _err(L, _rope(L, inv=C.c_void_p(0x10004)), L.NF4_E_ARG, "inv_freq")
    assert _rope(L, T=0, q=None) == 0 and _rope(L, hq=0, hkv=0) == 0


def _list(L, entries, table=FAKE, table_bytes=1 << 30):
    arr = (L.GradTensor * max(1, len(entries)))(*[L.GradTensor(*e) for e in entries])
    h = C.c_void_p()
    rc = L.raw().nf4_grad_list_create(arr, len(entries), table, table_bytes, None, C.byref(h))
    return rc, h


def test_grad_list_validation(L):
    f32 = L.NF4_DTYPE_F32
    ok = (0x20000, 0x20000, 64, f32)
    for entry, code, needle in (((0x20000, 0x20000, 64, 7), L.NF4_E_ARG, "dtype"),
                                ((0x20000, 0x20000, -1, f32), L.NF4_E_SHAPE, "count"),
                                ((0x20000, 0x20000, (1 << 36) + 1, f32), L.NF4_E_SHAPE, "count"),
                                ((0, 0x20000, 64, f32), L.NF4_E_ARG, "NULL"),
                                ((0x20002, 0x20002, 64, f32), L.NF4_E_ARG, "aligned"),
                                ((0x20000, 0x20080, 64, f32), L.NF4_E_ARG, "overlaps"),
                                ((0x20010, 0x30000, 1, f32), L.NF4_E_ARG, "overlaps"),
                                ((0x30000, 0x20010, 1, f32), L.NF4_E_ARG, "overlaps"),
                                (ok, L.NF4_E_ARG, "overlaps")):
        rc, _ = _list(L, [ok, entry])
        _err(L, rc, code, needle)
    _err(L, _list(L, [ok], table=None)[0], L.NF4_E_ARG, "table")
    _err(L, _list(L, [ok], table_bytes=8)[0], L.NF4_E_ARG, "table")
    rc = L.raw().nf4_grad_list_create(None, 2, FAKE, 1 << 20, None, C.byref(C.c_void_p()))
    _err(L, rc, L.NF4_E_ARG, "tensors")
    rc = L.raw().nf4_grad_list_create(None, 0, FAKE, 1 << 20, None, None)
    _err(L, rc, L.NF4_E_ARG, "out is NULL")


def test_empty_grad_list_and_call_validation(L):
    rc, h = _list(L, [(None, None, 0, L.NF4_DTYPE_F32)])     # nothing to copy: no device needed
    assert rc == 0 and h.value
    raw, ws = L.raw(), L.raw().nf4_grad_workspace()
    for bad in (-1.0, float("inf"), float("nan")):
        _err(L, raw.nf4_grad_clip(h, bad, FAKE, FAKE, ws, None), L.NF4_E_ARG, "max_norm")
    _err(L, raw.nf4_grad_clip(None, 1.0, FAKE, FAKE, ws, None), L.NF4_E_ARG, "NULL list")
    _err(L, raw.nf4_grad_norm(h, None, FAKE, ws, None), L.NF4_E_ARG, "norm")
    _err(L, raw.nf4_grad_norm(h, FAKE, FAKE, ws - 1, None), L.NF4_E_ARG, str(ws))
    _err(L, raw.nf4_grad_norm(h, FAKE, C.c_void_p(0x10010), ws, None), L.NF4_E_ARG, "256-byte")
    assert raw.nf4_grad_list_destroy(h) == 0
    _err(L, raw.nf4_grad_list_destroy(None), L.NF4_E_ARG, "NULL list")


def test_grad_norm_within_its_workspace_is_refused(L):
    rc, h = _list(L, [(None, None, 0, L.NF4_DTYPE_F32)])
    raw, ws = L.raw(), L.raw().nf4_grad_workspace()
    for call in (raw.nf4_grad_norm, lambda h, *a: raw.nf4_grad_clip(h, 1.0, *a)):
        for at in (0, 8, ws - 4):
            _err(L, call(h, C.c_void_p(FAKE.value + at), FAKE, ws, None), L.NF4_E_ARG, "overlaps")
    assert raw.nf4_grad_list_destroy(h) == 0


def test_grad_table_over_a_tensor_is_refused(L):
    at = 0x20000
    for grad, out in ((at, at), (at + 0x8000, at), (at, at + 0x8000)):
        rc, _ = _list(L, [(grad, out, 64, L.NF4_DTYPE_F32)], table=C.c_void_p(at))
        _err(L, rc, L.NF4_E_ARG, "table overlaps")


@pytest.mark.parametrize("T,n,hq,hkv,D,fits", [
    (40, 1 << 13, 256, 256, 64, True),             # (T/64 + n) (hq + hkv) = 2^22, both kinds in one launch
    (40, 1 << 14, 256, 256, 64, False),            # 2^23 and as many threads as pass 32 bits
    (40, (1 << 14) - 32, 256, 256, 64, True),
    (1 << 14, 1 << 14, 256, 256, 64, True),        # launches of their own, 2^22 and more workgroups each
    (1 << 14, 1 << 14, 256, 256, 128, True),
    (1 << 14, 1 << 14, 512, 512, 64, False),
    (1 << 14, (1 << 14) - 192, 512, 512, 64, True),
    (1 << 23, 0, 64, 64, 128, True),
])
def test_backward_grids_are_checked_launch_by_launch(L, T, n, hq, hkv, D, fits):
    """Without a workspace: sizes whose launches fit are refused for that, others for their workgroups
    (nothing is launched either way)."""
    at = [C.c_void_p((1 << 44) * (i + 1)) for i in range(10)]
    rc = L.raw().nf4_attn_bwd(at[0], at[1], at[2], at[3], at[4], at[5], T, hq, hkv, D, at[9] if n else None, n, 1, 0.125,
                              at[6], at[7], at[8], None, 0, None)
    _err(L, rc, *((L.NF4_E_ARG, "workspace") if fits else (L.NF4_E_SHAPE, "workgroups")))


@pytest.mark.parametrize("call", [_fwd, _bwd])
def test_more_sequences_than_the_scan_serves_are_refused(L, call):
    _err(L, call(L, T=1 << 16, cu=FAKE, n=(1 << 16) + 1), L.NF4_E_SHAPE, "n_seqs <= 2^16")
    _err(L, call(L, q=None, cu=FAKE, n=1 << 16), L.NF4_E_ARG, "NULL")   # as many pass this check


@pytest.mark.parametrize("dims,tokens,lens", [
    (dict(q=96, kv=48, head_dim=48), 8, None),             # a head width without a kernel
    (dict(q=128, kv=64, head_dim=0), 8, None),
    (dict(q=100, kv=32, head_dim=32), 8, None),            # not whole heads
    (dict(q=128, kv=40, head_dim=32), 8, None),
    (dict(q=160, kv=64, head_dim=32), 8, None),            # 5 query heads over 2
    (dict(q=2048 * 32, kv=32, head_dim=32), 8, None),
    (dict(q=128, kv=32, head_dim=32), (1 << 23) + 1, None),
    (dict(q=128, kv=32, head_dim=32), 1 << 17, [2] * (1 << 16) + [0]),
])
def test_stack_refuses_sizes_that_its_attention_does(L, dims, tokens, lens):
    """Before anything is allocated or copied: the base here holds nothing but its sizes."""
    from nf4_weight_streamed_amd import stack

    base = SimpleNamespace(dims=stack.StackDims(hidden=128, inter=256, **dims))
    with pytest.raises(ValueError, match="mixing='attention' needs"):
        stack.NF4Stack(base, None, tokens, mixing="attention", seq_lens=lens)


def test_stack_refuses_sequence_lengths_that_are_not_whole(L):
    from nf4_weight_streamed_amd import stack

    base = SimpleNamespace(dims=stack.StackDims(hidden=128, q=128, kv=32, inter=256, head_dim=32))
    with pytest.raises(ValueError, match="whole"):
        stack.NF4Stack(base, None, 8, mixing="attention", seq_lens=[4.5, 3.5])
    with pytest.raises(AttributeError):                    # whole ones of any type pass: the base here has no more
        stack.NF4Stack(base, None, 8, mixing="attention", seq_lens=[4.0, 4])
    with pytest.raises(ValueError, match="add up"):
        stack.NF4Stack(base, None, 8, mixing="attention", seq_lens=iter([4, 5]))
