"""The stack with 8-bit checkpoints (all of its operators together, as a training step runs them):
against the fp64 oracle at the checkpoints' values, streamed and rematerialised against resident bit
for bit, and against the bf16 stack."""

import numpy as np
import pytest
import torch

import oracle as O
import synthetic_inputs as S
from helpers import bits_of, f32_of, to_dev_bf16

pytestmark = pytest.mark.gpu
PROJS = ("q", "k", "v", "o", "gate", "up", "down")
TINY = dict(hidden=128, q=128, kv=32, inter=256, head_dim=32)


@pytest.fixture(scope="module")
def ST(gpu_lib):
    from nf4_weight_streamed_amd import stack

    return stack


def _stack(ST, n_layers, block_size, dims, dense=False):
    w = {(l, p): S.weight(*dims.shapes()[p], proj=p, layer=l) for l in range(n_layers) for p in PROJS}
    lo = {}
    for l in range(n_layers):
        for p in PROJS:
            n, k = dims.shapes()[p]
            lo[(l, p)] = (S.lora_a(16, k, proj=p, layer=l), S.lora_b(n, 16, proj=p, layer=l, std=0.05))
    kind = ST.HostBF16Base if dense else ST.HostNF4Base
    base = kind(dims, n_layers, block_size, lambda l, p, n, k: to_dev_bf16(w[(l, p)]))
    lora = ST.LoraParams(dims, n_layers, 16, lambda l, p, n, k: tuple(to_dev_bf16(t) for t in lo[(l, p)]))
    return w, lo, base, lora


@pytest.mark.parametrize("t,lens", [(41, None), (41, [17, 0, 23, 1]), (150, [150])])
def test_tiny_stack_matches_oracle(ST, t, lens):
    """Outputs within the linears' bar. A gradient's distance has two parts in quadrature: that of the bf16
    stack with attention (9.3e-3: the 2e-3 bar and four more bf16 roundings), and that of checkpoints whose
    inputs differ in last bits, so that both sides' roundings to a step are as good as independent. One
    is off by step / sqrt(12) rms, a step is a / 127 and a at most 3.3 rms for 15 of 16 runs of 64 normal
    values: 0.0075 a read and side; six reads a layer (gate and up twice, hm, ha), two layers: 0.0367."""
    L, alpha = 2, 32.0
    dims = ST.StackDims(**TINY)
    w, lo, base, lora = _stack(ST, L, 1, dims)
    h0, dh = S.activations(t, dims.hidden, tensor="h0"), S.activations(t, dims.hidden, tensor="dH")
    st = ST.NF4Stack(base, lora, t, alpha, mixing="attention", seq_lens=lens, checkpoints="int8")
    out, dh0 = st.step(to_dev_bf16(h0), to_dev_bf16(dh))
    torch.cuda.synchronize()
    od = O.StackLayerDims(dims.hidden, dims.q, dims.kv, dims.inter, dims.head_dim)
    layers = [{p: (O.dequantize(*O.quantize(O.bf16_bits_to_f64(w[(l, p)]).astype(np.float32))), *lo[(l, p)])
               for p in PROJS} for l in range(L)]
    pos = np.concatenate([np.arange(n) for n in (lens or [t])])
    inv = 1e6 ** (-np.arange(0, dims.head_dim, 2) / dims.head_dim)
    out_ref, saved = O.decoder_forward(h0, layers, od, alpha, pos, inv, lens)
    dh0_ref, grads = O.decoder_backward_act8(dh, layers, od, alpha, saved, pos, inv, lens)
    bar = float(np.sqrt(2e-3 ** 2 + (4 * 2.0 ** -8) ** 2 / 3 + 2 * 12 * 0.0075 ** 2))
    assert O.rel_l2(O.bf16_bits_to_f64(bits_of(out)), out_ref) <= 2e-3
    assert O.rel_l2(O.bf16_bits_to_f64(bits_of(dh0)), dh0_ref) <= bar
    for l in range(L):
        for p in PROJS:
            for got, key in zip(st.grads[l][p], ("_dA", "_dB")):
                assert torch.any(got != 0), (l, p)
                assert O.rel_l2(f32_of(got), grads[l][p + key]) <= bar, (l, p, key)
    st.close()


def _run(ST, base, lora, T, **kw):
    st = ST.NF4Stack(base, lora, T, 32.0, checkpoints="int8", **kw)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    h0, dh = (torch.randn(T, base.dims.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    res = []
    for _ in range(2):
        out, dh0 = st.step(h0, dh)
        res += [out.clone(), dh0.clone(), st.clip_grads(1.0).clone()]
        res += [t.clone() for gl in st.grads for p in PROJS for t in gl[p]]
    torch.cuda.synchronize()
    st.close()
    return res


@pytest.mark.parametrize("block_size", [1, 2])
@pytest.mark.parametrize("dense", [False, True])
@pytest.mark.parametrize("mixing", ["identity", "attention"])
def test_streamed_and_remat_equal_resident(ST, block_size, dense, mixing):
    dims = ST.StackDims(hidden=256, q=256, kv=128, inter=320, head_dim=64)
    _, _, base, lora = _stack(ST, 5, block_size, dims, dense)
    lens = {"seq_lens": [100, 1, 49]} if mixing == "attention" else {}
    ref = _run(ST, base, lora, 150, mode="resident", mixing=mixing, **lens)
    n = len(ref) // 2
    assert all(torch.equal(a, b) for a, b in zip(ref[:n], ref[n:]))          # step 2 equals step 1
    for kw in ({}, {"remat": True}, {"prefetch": False}, {"n_slots": 3, "remat": True}):
        got = _run(ST, base, lora, 150, mode="streamed", mixing=mixing, **lens, **kw)
        assert all(torch.equal(a, b) for a, b in zip(got, ref)), kw


def test_beside_the_bf16_stack(ST):
    """Two 7B-wide layers at 512 tokens: what is held falls to 41 to 45 % (by count: ha, hm, gate, up at 1.0625
    bytes, q, k, v, a at 2 and no h, h1, m, against all of them at 2); gradients move by at most what the
    checkpoints' rounding allows: six reads a layer of 0.0075 each, two layers, doubled for widths whose
    runs of 64 are not all alike."""
    dims, _ = ST.QWEN25["7b"]
    base = ST.HostNF4Base(dims, 2, 1, ST.qwen_weight_fn())
    lora = ST.LoraParams(dims, 2, 16, ST.qwen_lora_fn())
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    h0, dh = (torch.randn(512, dims.hidden, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    grads, held = [], []
    for kind in ("bf16", "int8"):
        st = ST.NF4Stack(base, lora, 512, 32.0, mode="resident", mixing="attention", checkpoints=kind)
        _, dh0 = st.step(h0, dh)
        torch.cuda.synchronize()
        grads.append([dh0.float().clone()] + [t.clone() for gl in st.grads for p in PROJS for t in gl[p]])
        held.append(st.activation_bytes())
        st.close()
    assert 0.40 <= held[1] / held[0] <= 0.46
    for a, b in zip(*grads):
        assert float((a - b).norm() / a.norm()) <= 2 * 12 ** 0.5 * 0.0075


def test_refusals_and_scratch(ST):
    dims = ST.StackDims(**TINY)
    _, _, base, lora = _stack(ST, 1, 1, dims)
    with pytest.raises(ValueError, match="checkpoints"):
        ST.NF4Stack(base, lora, 8, checkpoints="fp8")
    h0, dh = (to_dev_bf16(S.activations(8, dims.hidden, tensor=n)) for n in ("h0", "dH"))
    for mixing in ("identity", "attention"):
        st = ST.NF4Stack(base, lora, 8, 32.0, mixing=mixing, checkpoints="int8")
        scratch = {n: t for n, t in st.tmp.items() if mixing == "attention" or n not in ("zq", "zkv")}
        for t in scratch.values():
            t.view(torch.int16).fill_(0x7FA5)                  # a NaN that no step computes
        st.step(h0, dh)
        torch.cuda.synchronize()
        assert [n for n, t in scratch.items() if bool((t.view(torch.int16) == 0x7FA5).any())] == []
        st.close()


@pytest.mark.parametrize("t,lens", [(41, None), (150, [100, 1, 49])])
def test_backward_at_the_stacks_own_checkpoints(ST, t, lens):
    """The oracle's backward from what the stack itself kept: its checkpoints' values, a, rotated q and k, v, lse and
    1 / rms. What is left to differ are the backward's roundings, as in the bf16 stack with attention (the linears' 2e-3
    bar, four more of 2^-8 / sqrt(3) rms), and one of those for dB, whose u comes from the forward's own x: 1.15e-2,
    a third of what a test has to allow where each side rounds to steps of its own."""
    L, alpha = 2, 32.0
    dims = ST.StackDims(**TINY)
    w, lo, base, lora = _stack(ST, L, 1, dims)
    h0, dh = S.activations(t, dims.hidden, tensor="h0"), S.activations(t, dims.hidden, tensor="dH")
    st = ST.NF4Stack(base, lora, t, alpha, mode="resident", mixing="attention", seq_lens=lens, checkpoints="int8")
    _, dh0 = st.step(to_dev_bf16(h0), to_dev_bf16(dh))
    torch.cuda.synchronize()
    od = O.StackLayerDims(dims.hidden, dims.q, dims.kv, dims.inter, dims.head_dim)
    layers = [{p: (O.dequantize(*O.quantize(O.bf16_bits_to_f64(w[(l, p)]).astype(np.float32))), *lo[(l, p)])
               for p in PROJS} for l in range(L)]
    pos = np.concatenate([np.arange(n) for n in (lens or [t])])
    inv = 1e6 ** (-np.arange(0, dims.head_dim, 2) / dims.head_dim)
    _, saved = O.decoder_forward(h0, layers, od, alpha, pos, inv, lens)
    kept = []
    for l in reversed(range(L)):
        A = st.acts[l]
        for name in ("ha", "hm", "gate", "up"):                     # the order in which the backward reads them
            x8 = A[name + "8"]
            kept.append(O.act8_values(x8.codes.cpu().numpy(), x8.scale.cpu().numpy()).astype(np.float64))
            # half a step, 0.0075 rms, and the forward's own bar, doubled: what it says it is
            assert O.rel_l2(kept[-1], saved[l][name]) <= 2 * (0.0075 + 2e-3), (l, name)
        for name in ("a", "q", "k", "v"):
            saved[l][name] = O.bf16_bits_to_f64(bits_of(A[name]))
        saved[l]["lse"] = f32_of(A["lse"]).astype(np.float64)
        for name, rs in (("h", "rs_h"), ("h1", "rs_h1")):            # rows of that 1 / rms: nothing else is read of them
            ms = 1 / f32_of(A[rs]).astype(np.float64) ** 2 - O.RMS_EPS
            saved[l][name] = np.sqrt(ms)[:, None] * np.ones((1, dims.hidden))
    values = iter(kept)
    dh0_ref, grads = O.decoder_backward_act8(dh, layers, od, alpha, saved, pos, inv, lens, keep=lambda x: next(values))
    assert next(values, None) is None
    bar = float(np.hypot(2e-3, 5 * 2.0 ** -8 / np.sqrt(3)))
    assert O.rel_l2(O.bf16_bits_to_f64(bits_of(dh0)), dh0_ref) <= bar
    for l in range(L):
        for p in PROJS:
            for got, key in zip(st.grads[l][p], ("_dA", "_dB")):
                assert O.rel_l2(f32_of(got), grads[l][p + key]) <= bar, (l, p, key)
    st.close()
