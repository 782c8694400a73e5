"""Rotary positions through the C ABI against the fp64 oracle, element by element."""

import numpy as np
import pytest
import torch

import oracle as O
from helpers import bits_of, half_ulp_bf16, to_dev_bf16

pytestmark = pytest.mark.gpu


def _bits(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _check(lib, t, hq, hkv, d, sections, span, inverse=False, theta=1e6, in_place=False):
    rng = np.random.default_rng([t, hq, hkv, d, len(sections)])
    q, k = (_bits(rng.normal(size=(t, h * d))) for h in (hq, hkv))
    pos = rng.integers(span[0], span[1], size=(len(sections), t), endpoint=True).astype(np.int32)
    inv = lib.rope_inv_freq(d, theta)
    dq, dk = to_dev_bf16(q), to_dev_bf16(k)
    out = {"q_out": dq, "k_out": dk} if in_place else {}
    got = lib.rope(dq, dk, d, torch.from_numpy(pos).cuda(), inv, sections, inverse, **out)
    torch.cuda.synchronize()
    for x, g in zip((q, k), got):
        want = O.rope(x, d, pos, inv.cpu().numpy(), sections, inverse)
        # |lo| + |hi| bounds both terms: a fp32 angle in (-pi, pi] is off by 2^-24 pi, its sine
        # and cosine by 2 units more, each product and the sum by one: below 8 * 2^-24 in all;
        # the fp64 angle of a position up to 2^31 by 2^31 * 2^-51
        y = np.abs(O.bf16_bits_to_f64(x)).reshape(t, -1, 2, d // 2).sum(2, keepdims=True)
        mag = np.broadcast_to(y, (t, y.shape[1], 2, d // 2)).reshape(x.shape)
        b = (8 * 2.0 ** -24 + 2.0 ** -20) * mag
        err = np.abs(O.bf16_bits_to_f64(bits_of(g)) - want)
        assert np.all(err <= b + half_ulp_bf16(np.abs(want) + b)), float((err - b).max())


@pytest.mark.parametrize("d,sections", [(128, (64,)), (128, (16, 24, 24)), (64, (32,)), (64, (1, 31)), (32, (4, 4, 4, 4)),
                                        (16, (8,)), (48, (24,)), (80, (20, 20)), (256, (128,))])
@pytest.mark.parametrize("t", [1, 2, 33, 130])
def test_axes_and_widths(gpu_lib, t, d, sections):
    for hq, hkv, inverse in ((4, 1, False), (3, 3, True)):
        _check(gpu_lib, t, hq, hkv, d, sections, (0, 300), inverse)


@pytest.mark.parametrize("span", [(0, 0), (-5, 5), (1_000_000, 1_100_000), (-(2 ** 31), 2 ** 31 - 1)])
def test_far_and_negative_positions(gpu_lib, span):
    _check(gpu_lib, 70, 28, 4, 128, (64,), span)
    _check(gpu_lib, 70, 2, 2, 64, (10, 22), span, theta=1e4)


def test_in_place_equals_out_of_place_and_inverse_returns(gpu_lib):
    lib, t, d = gpu_lib, 300, 128
    _check(lib, t, 8, 2, d, (64,), (0, 5000), in_place=True)
    x = torch.randn(t, 8 * d, device="cuda").to(torch.bfloat16)
    pos, inv = torch.arange(t, dtype=torch.int32, device="cuda"), lib.rope_inv_freq(d)
    y, none = lib.rope(x, None, d, pos, inv)      # q alone, positions without an axis dimension
    assert none is None
    z, _ = lib.rope(y, None, d, pos, inv, inverse=True)
    # two roundings of a rotated pair: 2^-8 of |lo| + |hi| each, and a rotation of the first
    pair = x.float().abs().view(t, -1, 2, d // 2).sum(2, keepdim=True)
    assert torch.all((z.float() - x.float()).abs().view(t, -1, 2, d // 2) <= 3 * 2.0 ** -8 * pair)


def test_heads_and_rows_past_32_bits(gpu_lib):
    """270000 rows of 64 heads (over 4 GiB): the last rows equal a call on them alone."""
    lib, t, n, d = gpu_lib, 270000, 65, 128
    q = torch.empty(t, 64 * d, dtype=torch.bfloat16, device="cuda")
    q[t - n:] = torch.randn(n, 64 * d, device="cuda").to(torch.bfloat16)
    pos, inv = torch.arange(t, dtype=torch.int32, device="cuda"), lib.rope_inv_freq(d)
    want, _ = lib.rope(q[t - n:].clone(), None, d, pos[t - n:].clone(), inv)
    got, _ = lib.rope(q, None, d, pos, inv, q_out=q)
    torch.cuda.synchronize()
    assert torch.equal(got[t - n:], want)


def test_graph_replays_equal_eager(gpu_lib):
    lib, d = gpu_lib, 64
    q, k = (torch.randn(77, h * d, device="cuda").to(torch.bfloat16) for h in (6, 2))
    pos, inv = torch.arange(77, dtype=torch.int32, device="cuda"), lib.rope_inv_freq(d)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    lib.rope(q, k, d, pos, inv, q_out=qo, k_out=ko)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.rope(q, k, d, pos, inv, q_out=qo, k_out=ko)
    for rep in range(3):
        pos.add_(100)
        ref = [x.clone() for x in lib.rope(q, k, d, pos, inv)]
        qo.fill_(rep)
        ko.fill_(rep)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(qo, ref[0]) and torch.equal(ko, ref[1])


def test_python_refusals(gpu_lib):
    lib, d = gpu_lib, 32
    q = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    pos, inv = torch.zeros(1, 4, dtype=torch.int32, device="cuda"), lib.rope_inv_freq(d)
    with pytest.raises(TypeError, match="int32"):
        lib.rope(q, q, d, pos.long(), inv)
    with pytest.raises(ValueError, match="pos"):
        lib.rope(q, q, d, pos, inv, sections=(8, 8))
    with pytest.raises(TypeError, match="float64"):
        lib.rope(q, q, d, pos, inv.float())
    with pytest.raises(lib.Nf4Error, match="pairs"):
        lib.rope(q, q, d, pos, inv, sections=(15,))
    with pytest.raises(ValueError, match="heads"):
        lib.rope(q, q[:, :40].contiguous(), d, pos, inv)
    assert lib.rope(q[:0], q[:0], d, pos[:, :0].contiguous(), inv)[0].shape == (0, 64)
