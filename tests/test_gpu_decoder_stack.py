"""The stack with attention mixing (rotary positions, attention, clipping together, as a
training step runs them): against the fp64 oracle, streamed and rematerialised against
resident bit for bit, and its clipping against the gradients' fp64 norm."""

import numpy as np
import pytest
import torch

import oracle as O
import synthetic_inputs as S
from helpers import bits_of, f32_of, to_dev_bf16

pytestmark = pytest.mark.gpu
PROJS = ("q", "k", "v", "o", "gate", "up", "down")


@pytest.fixture(scope="module")
def ST(gpu_lib):
    from nf4_weight_streamed_amd import stack

    return stack


def _stack(ST, n_layers, block_size, dims):
    w = {(l, p): S.weight(*dims.shapes()[p], proj=p, layer=l) for l in range(n_layers) for p in PROJS}
    lo = {}
    for l in range(n_layers):
        for p in PROJS:
            n, k = dims.shapes()[p]
            lo[(l, p)] = (S.lora_a(16, k, proj=p, layer=l), S.lora_b(n, 16, proj=p, layer=l, std=0.05))
    base = ST.HostNF4Base(dims, n_layers, block_size, lambda l, p, n, k: to_dev_bf16(w[(l, p)]))
    lora = ST.LoraParams(dims, n_layers, 16, lambda l, p, n, k: tuple(to_dev_bf16(t) for t in lo[(l, p)]))
    return w, lo, base, lora


TINY = dict(hidden=128, q=128, kv=32, inter=256, head_dim=32)


@pytest.mark.parametrize("lens", [None, [17, 0, 23, 1]])
def test_tiny_decoder_stack_matches_oracle(ST, lens):
    """Outputs within the linears' bar. Gradients pass through three bf16-stored tensors more
    a layer than the identity stack's (dq, dk, dv, each rounded, two of them again by the
    rotation) and through P and dS in bf16: at most 4 more roundings of 2^-8 / sqrt(3) rms at
    relative size one, in quadrature with the 2e-3 bar: 9.3e-3."""
    L, T, alpha = 2, 41, 32.0
    dims = ST.StackDims(**TINY)
    w, lo, base, lora = _stack(ST, L, 1, dims)
    h0, dh = S.activations(T, dims.hidden, tensor="h0"), S.activations(T, dims.hidden, tensor="dH")
    st = ST.NF4Stack(base, lora, T, alpha, mixing="attention", seq_lens=lens)
    out, dh0 = st.step(to_dev_bf16(h0), to_dev_bf16(dh))
    torch.cuda.synchronize()
    od = O.StackLayerDims(dims.hidden, dims.q, dims.kv, dims.inter, dims.head_dim)
    layers = [{p: (O.dequantize(*O.quantize(O.bf16_bits_to_f64(w[(l, p)]).astype(np.float32))), *lo[(l, p)])
               for p in PROJS} for l in range(L)]
    pos = np.concatenate([np.arange(n) for n in (lens or [T])])
    inv = 1e6 ** (-np.arange(0, dims.head_dim, 2) / dims.head_dim)
    out_ref, saved = O.decoder_forward(h0, layers, od, alpha, pos, inv, lens)
    dh0_ref, grads = O.decoder_backward(dh, layers, od, alpha, saved, pos, inv, lens)
    bar = float(np.hypot(2e-3, 4 * 2.0 ** -8 / np.sqrt(3)))
    assert O.rel_l2(O.bf16_bits_to_f64(bits_of(out)), out_ref) <= 2e-3
    assert O.rel_l2(O.bf16_bits_to_f64(bits_of(dh0)), dh0_ref) <= bar
    for l in range(L):
        for p in PROJS:
            for got, key in zip(st.grads[l][p], ("_dA", "_dB")):
                assert torch.any(got != 0), (l, p)
                assert O.rel_l2(f32_of(got), grads[l][p + key]) <= bar, (l, p, key)
    # clipping all of them together
    before = [[tuple(t.clone() for t in gl[p]) for p in PROJS] for gl in st.grads]
    norm = O.grad_clip([f32_of(t) for gl in before for pair in gl for t in pair], 1.0)[0]
    got = st.clip_grads(0.25 * norm)
    torch.cuda.synchronize()
    assert got.item() == pytest.approx(norm, rel=2e-7)
    for gl, bl in zip(st.grads, before):
        for p, pair in zip(PROJS, bl):
            for t, b in zip(gl[p], pair):
                assert torch.allclose(t, 0.25 * b, rtol=1e-6, atol=0)
    st.close()


def _run(ST, base, lora, T, **kw):
    st = ST.NF4Stack(base, lora, T, 32.0, mixing="attention", **kw)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    h0, dh = (torch.randn(T, base.dims.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    res = []
    for _ in range(2):
        out, dh0 = st.step(h0, dh)
        norm = st.clip_grads(1.0)
        res += [out.clone(), dh0.clone(), norm.clone()]
        res += [t.clone() for gl in st.grads for p in PROJS for t in gl[p]]
    torch.cuda.synchronize()
    st.close()
    return res


@pytest.mark.parametrize("block_size", [1, 2])
def test_streamed_and_remat_equal_resident(ST, block_size):
    dims = ST.StackDims(hidden=256, q=256, kv=128, inter=256, head_dim=64)
    _, _, base, lora = _stack(ST, 5, block_size, dims)
    lens = [100, 1, 49]
    ref = _run(ST, base, lora, 150, mode="resident", seq_lens=lens)
    n = len(ref) // 2
    assert all(torch.equal(a, b) for a, b in zip(ref[:n], ref[n:]))          # step 2 equals step 1
    for kw in ({}, {"remat": True}, {"prefetch": False}, {"n_slots": 3, "remat": True}):
        got = _run(ST, base, lora, 150, mode="streamed", seq_lens=lens, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), kw


def test_qwen7b_widths_finite_and_equal(ST):
    """Two 7B-wide layers at 512 tokens, one sequence: streamed equals resident."""
    dims, _ = ST.QWEN25["7b"]
    base = ST.HostNF4Base(dims, 2, 1, ST.qwen_weight_fn())
    lora = ST.LoraParams(dims, 2, 16, ST.qwen_lora_fn())
    ref = _run(ST, base, lora, 512, mode="resident")
    got = _run(ST, base, lora, 512, mode="streamed")
    assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert all(torch.isfinite(t.float()).all() for t in ref)


def test_refusals(ST):
    dims = ST.StackDims(**TINY)
    _, _, base, lora = _stack(ST, 1, 1, dims)
    with pytest.raises(ValueError, match="mixing"):
        ST.NF4Stack(base, lora, 8, mixing="linear")
    with pytest.raises(ValueError, match="seq_lens"):
        ST.NF4Stack(base, lora, 8, seq_lens=[8])
    for lens in ([4, 3], [9, -1], []):
        with pytest.raises(ValueError, match="seq_lens"):
            ST.NF4Stack(base, lora, 8, mixing="attention", seq_lens=lens)


def test_every_scratch_buffer_is_used(ST):
    """The scratch that a stack holds beside its activations is what a step writes: no buffer keeps the
    pattern it was filled with before one, but for the identity mixing's zero gradients."""
    dims = ST.StackDims(**TINY)
    _, _, base, lora = _stack(ST, 1, 1, dims)
    h0, dh = (to_dev_bf16(S.activations(8, dims.hidden, tensor=n)) for n in ("h0", "dH"))
    for mixing in ("identity", "attention"):
        st = ST.NF4Stack(base, lora, 8, 32.0, mixing=mixing)
        scratch = {n: t for n, t in st.tmp.items() if mixing == "attention" or n not in ("zq", "zkv")}
        for t in scratch.values():
            t.view(torch.int16).fill_(0x7FA5)                  # a NaN that no step computes
        st.step(h0, dh)
        torch.cuda.synchronize()
        assert [n for n, t in scratch.items() if bool((t.view(torch.int16) == 0x7FA5).any())] == []
        st.close()
