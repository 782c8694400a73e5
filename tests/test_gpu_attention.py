"""Attention forward and backward through the C ABI against the fp64 oracle, element by
element within the bounds that oracle.attention_bounds derives, and against central
differences of the oracle's forward; head layouts, odd and empty sequences, rows outside
the sequences, non-finite neighbours, offsets past 32 bits, streams, graphs, refusals."""

import numpy as np
import pytest
import torch

import oracle as O
from helpers import bits_of, f32_of, half_ulp_bf16, to_dev_bf16

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def stream_pair_first(gpu_lib):
    """The library's compute/copy pair, made for the life of the process, before this file
    makes streams and graphs: made later, the two may fall on one hardware queue."""
    gpu_lib.pool_streams()


def _bits(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def _case(t, hq, hkv, d, seed=0, q_std=1.5):
    rng = np.random.default_rng([t, hq, hkv, d, seed])
    return {n: _bits(rng.normal(0, q_std if n == "q" else 1.0, size=(t, h * d)))
            for n, h in (("q", hq), ("k", hkv), ("v", hkv), ("do", hq))}


def _cu(lens):
    return None if lens is None else torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32).cuda()


def _inside(got, exact, bound, what):
    # second-order products of the bound's terms stay below 1 % of it
    err, lim = np.abs(got - exact), 1.01 * bound
    assert np.all(np.isfinite(got)), what
    assert np.all(err <= lim), f"{what}: worst {np.max(err - lim):.3e} beyond, at {np.argmax(err - lim)}"


def _within(got, exact, bound, what):
    _inside(O.bf16_bits_to_f64(bits_of(got)), exact, bound + half_ulp_bf16(np.abs(exact) + 1.01 * bound), what)


def _check(lib, c, d, lens=None, causal=True, scale=None, ds_unit=2.0 ** -8, names=("dq", "dk", "dv")):
    t = c["q"].shape[0]
    hq, hkv = c["q"].shape[1] // d, c["k"].shape[1] // d
    dev = {n: to_dev_bf16(x) for n, x in c.items()}
    # rows outside the sequences keep what they held: zeros here, as in the oracle
    z = lambda h: torch.zeros(t, h * d, dtype=torch.bfloat16, device="cuda")
    o, lse = lib.attn_fwd(dev["q"], dev["k"], dev["v"], d, _cu(lens), causal, scale, o=z(hq),
                          lse=torch.zeros(hq, t, device="cuda"))
    o_ref, lse_ref = O.attention_fwd(c["q"], c["k"], c["v"], d, lens, causal, scale)
    # the backward gets the oracle's forward in the storage types
    ob, l32 = _bits(o_ref), lse_ref.astype(np.float32)
    dq, dk, dv = lib.attn_bwd(dev["q"], dev["k"], dev["v"], to_dev_bf16(ob), torch.from_numpy(l32).cuda(), dev["do"], d,
                              _cu(lens), causal, scale, dq=z(hq), dk=z(hkv), dv=z(hkv))
    torch.cuda.synchronize()
    bound = O.attention_bounds(c["q"], c["k"], c["v"], ob, l32, c["do"], d, lens, causal, scale, ds_unit)
    refs = O.attention_bwd(c["q"], c["k"], c["v"], ob, l32, c["do"], d, lens, causal, scale)
    _within(o, o_ref, bound["o"], "o")
    _inside(f32_of(lse), lse_ref, bound["lse"], "lse")
    for name, got, ref in zip(("dq", "dk", "dv"), (dq, dk, dv), refs):
        if name in names:
            _within(got, ref, bound[name], name)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("t", [1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 200, 321])
def test_lengths_and_head_widths(gpu_lib, t, d):
    for causal in (True, False):
        _check(gpu_lib, _case(t, 2, 1, d), d, causal=causal)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (7, 1), (6, 2), (5, 5), (6, 3), (8, 8), (14, 2), (16, 8), (32, 16)])
def test_head_layouts(gpu_lib, hq, hkv):
    _check(gpu_lib, _case(150, hq, hkv, 64), 64)
    _check(gpu_lib, _case(70, hq, hkv, 128), 128, causal=False)


@pytest.mark.parametrize("lens", [[1] * 70, [0, 5, 0, 0, 129, 64, 1, 0], [200, 1, 63, 65], [0, 0], [130],
                                  list(range(20)), [0] * 100 + [40] + [0] * 80 + [90]])
def test_packed_sequences(gpu_lib, lens):
    t = sum(lens)
    if t == 0:
        t = 3                                   # rows, but no sequence holds them
    for d, causal in ((64, True), (128, False), (32, True)):
        _check(gpu_lib, _case(t, 4, 2, d), d, lens, causal)


@pytest.mark.parametrize("hq,hkv,t", [(2, 2, 5), (8, 1, 300), (32, 1, 40), (64, 64, 1400)])
def test_sequences_of_one_token_pass_nothing_to_q_and_k(gpu_lib, hq, hkv, t):
    """A softmax over one key is 1 whatever its score: dq and dk are exactly zero, dv is the
    sum of do over the kv head's queries, and o is v."""
    for d, causal in ((64, True), (128, False)):
        c = {n: to_dev_bf16(x) for n, x in _case(t, hq, hkv, d).items()}
        cu = _cu([1] * t)
        o, lse = gpu_lib.attn_fwd(c["q"], c["k"], c["v"], d, cu, causal)
        dq, dk, dv = gpu_lib.attn_bwd(c["q"], c["k"], c["v"], o, lse, c["do"], d, cu, causal)
        torch.cuda.synchronize()
        assert torch.equal(o.view(t, hkv, -1, d), c["v"].view(t, hkv, 1, d).expand(-1, -1, hq // hkv, -1))
        assert not dq.any() and not dk.any()
        exact = c["do"].double().view(t, hkv, -1, d).sum(2).view(t, -1)
        # P is 2^(S - lse) with both in fp32, about 2^-18 off at |S| < 64; rounded to bf16 it is 1
        parts = c["do"].double().abs().view(t, hkv, -1, d).sum(2).view(t, -1)
        assert bool(((dv.double() - exact).abs() <= exact.abs() * 2.0 ** -8 + parts * 2.0 ** -18).all())


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("lens", [[2], [3, 0, 5], [17], [1, 1, 2], [30, 34], [64]])
def test_short_calls_round_ds_twice(gpu_lib, lens, d):
    """Up to 64 tokens dq and dk come from dS as the sum of two bf16 values, 2^-16 off."""
    for hq, hkv, causal in ((4, 2, True), (3, 3, False), (512, 64, True)):
        if hq == 512 and (d == 128 or sum(lens) > 20):
            continue
        _check(gpu_lib, _case(sum(lens), hq, hkv, d), d, lens, causal, ds_unit=2.0 ** -16, names=("dq", "dk"))


@pytest.mark.parametrize("hq,hkv", [(8, 1), (14, 2), (9, 1), (16, 1), (26, 2), (17, 1), (40, 2), (33, 11)])
def test_short_calls_of_many_heads_a_kv_head(gpu_lib, hq, hkv):
    """Blocks of queries of a kv head's heads side by side, eight at a time, or one after the other."""
    for lens, d, causal in (([64], 64, False), ([40, 0, 23], 128, True), ([33, 31], 32, True)):
        _check(gpu_lib, _case(sum(lens), hq, hkv, d), d, lens, causal, ds_unit=2.0 ** -16, names=("dq", "dk"))
        _check(gpu_lib, _case(sum(lens), hq, hkv, d), d, lens, causal)


def test_narrow_heads_round_ds_of_dq_twice(gpu_lib):
    for hq, hkv, t in ((4, 2, 300), (128, 64, 1000)):  # one launch and two
        _check(gpu_lib, _case(t, hq, hkv, 32), 32, None, False, ds_unit=2.0 ** -16, names=("dq",))


def test_longer_sequences_and_split_gradients(gpu_lib):
    """Key tiles by the dozen, and dk, dv from several shares (few kv heads) or one (many)."""
    _check(gpu_lib, _case(1100, 2, 1, 128), 128)
    _check(gpu_lib, _case(900, 4, 2, 64), 64, [500, 0, 400], causal=False)
    _check(gpu_lib, _case(650, 128, 128, 32), 32)


def test_scores_far_apart(gpu_lib):
    """Scores of hundreds, rising and falling along the keys: every rescaling of the running
    maximum and sums; the probabilities are near one-hot."""
    t, d = 300, 64
    c = _case(t, 2, 1, d, q_std=30.0)
    _check(gpu_lib, c, d)
    ramp = np.linspace(0.1, 6.0, t)[:, None]
    for r in (ramp, ramp[::-1]):
        c["k"] = _bits(np.abs(O.bf16_bits_to_f64(c["k"])) * r)
        c["q"] = _bits(np.abs(O.bf16_bits_to_f64(c["q"])) / 8)
        _check(gpu_lib, c, d)
        _check(gpu_lib, c, d, causal=False)
    _check(gpu_lib, _case(100, 2, 1, d), d, scale=1e-6)


def test_gradients_against_differences(gpu_lib):
    """<dq, x> + <dk, y> + <dv, z> equals the central difference of <do, o> along (x, y, z).
    The kernel's gradients are off by at most their bounds, summed against |x|, |y|, |z|; the
    difference's own error is of order step^2 and 2^-52/step, below 1e-6 of it."""
    t, d, lens = 90, 32, [40, 50]
    c = _case(t, 4, 2, d)
    f = {n: O.bf16_bits_to_f64(c[n]) for n in c}
    o_ref, lse_ref = O.attention_fwd(f["q"], f["k"], f["v"], d, lens)
    dev = {n: to_dev_bf16(x) for n, x in c.items()}
    o, lse = gpu_lib.attn_fwd(dev["q"], dev["k"], dev["v"], d, _cu(lens))
    grads = gpu_lib.attn_bwd(dev["q"], dev["k"], dev["v"], o, lse, dev["do"], d, _cu(lens))
    bound = O.attention_bounds(f["q"], f["k"], f["v"], o_ref, lse_ref, f["do"], d, lens)
    # o is the kernel's here: delta is off by at most |do| times o's bound, dS by P times that
    off = 1.01 * bound["o"]
    far = (np.abs(f["do"]) * (off + half_ulp_bf16(np.abs(o_ref) + off))).reshape(t, 4, d).sum(2)
    rng = np.random.default_rng(9)
    for name, g in zip("qkv", grads):
        x = rng.normal(size=f[name].shape)
        val = [float(np.sum(f["do"] * O.attention_fwd(*({**f, name: f[name] + s * x}[n] for n in "qkv"), d, lens)[0]))
               for s in (1e-5, -1e-5)]
        want = (val[0] - val[1]) / 2e-5
        got = O.bf16_bits_to_f64(bits_of(g))
        b = bound["d" + name] + half_ulp_bf16(np.abs(got))
        lim = float(np.sum(1.02 * b * np.abs(x))) + 1e-6 * abs(want) + 1e-6
        if name != "v":                          # P <= 1 sums to 1 a row, |k|, |q| <= max
            other = float(np.abs(f["k" if name == "q" else "q"]).max())
            lim += d ** -0.5 * other * float(far.sum()) * float(np.abs(x).reshape(t, -1, d).sum(2).max())
        assert abs(float(np.sum(got * x)) - want) <= lim, name


def test_outside_rows_and_neighbours(gpu_lib):
    """Rows before the first and behind the last sequence are left as they were, and NaN or
    infinities there, or in another sequence, reach nothing."""
    lib, d, t = gpu_lib, 64, 260
    c = _case(t, 4, 2, d)
    cu = torch.tensor([3, 100, 131, 240], dtype=torch.int32).cuda()
    clean = {n: to_dev_bf16(x) for n, x in c.items()}
    dirty = {n: x.clone() for n, x in clean.items()}
    for n in dirty:
        dirty[n][:3], dirty[n][240:], dirty[n][100:131] = float("nan"), float("inf"), float("nan")
    res = []
    for x in (clean, dirty):
        bufs = {n: torch.full_like(x["q" if n in ("o", "dq") else "k"], 7.0) for n in ("o", "dq", "dk", "dv")}
        lse = torch.full((4, t), 7.0, device="cuda")
        lib.attn_fwd(x["q"], x["k"], x["v"], d, cu, o=bufs["o"], lse=lse)
        lib.attn_bwd(x["q"], x["k"], x["v"], bufs["o"], lse, x["do"], d, cu, dq=bufs["dq"], dk=bufs["dk"],
                     dv=bufs["dv"])
        torch.cuda.synchronize()
        res.append({**bufs, "lse": lse.t().contiguous()})
    for n in res[0]:
        for r in res:
            assert torch.all(r[n][:3].float() == 7.0) and torch.all(r[n][240:].float() == 7.0), n
        for rows in (slice(3, 100), slice(131, 240)):
            assert torch.equal(res[0][n][rows], res[1][n][rows]), n
            assert torch.isfinite(res[0][n][rows].float()).all()


def test_bad_bounds_on_the_device_stay_inside(gpu_lib):
    """Sequence bounds outside 0..T are clamped: the rows they leave are as if given clamped."""
    lib, d, t = gpu_lib, 32, 70
    x = {n: to_dev_bf16(v) for n, v in _case(t, 2, 2, d).items()}
    out = []
    for cu in ([-50, 30, 1 << 30], [0, 30, t]):
        cu = torch.tensor(cu, dtype=torch.int32).cuda()
        o, lse = lib.attn_fwd(x["q"], x["k"], x["v"], d, cu)
        out.append((o, lse, *lib.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], d, cu)))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*out))


def test_repeated_calls_give_the_same_bits_on_any_stream(gpu_lib):
    lib, d = gpu_lib, 128
    x = {n: to_dev_bf16(v) for n, v in _case(500, 14, 2, d).items()}
    side = torch.cuda.Stream()
    res = []
    for stream in (None, None, side):
        torch.cuda.synchronize()
        o, lse = lib.attn_fwd(x["q"], x["k"], x["v"], d, stream=stream)
        ws = lib.workspace(lib.attn_bwd_workspace_bytes(500, 14, 2, d))
        ws.fill_(0xFF)                            # contents on entry are ignored
        torch.cuda.synchronize()
        g = lib.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["do"], d, ws=ws, stream=stream)
        torch.cuda.synchronize()
        res.append((o, lse, *g))
    for r in res[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, res[0]))


def test_graph_replays_equal_eager(gpu_lib):
    lib, d = gpu_lib, 64
    x = {n: to_dev_bf16(v) for n, v in _case(333, 8, 2, d).items()}
    cu = _cu([100, 0, 233])
    out = {n: torch.empty_like(x["q" if n in ("o", "dq") else "k"]) for n in ("o", "dq", "dk", "dv")}
    out["lse"] = torch.empty(8, 333, device="cuda")
    ws = lib.workspace(lib.attn_bwd_workspace_bytes(333, 8, 2, d, 3))

    def step():
        lib.attn_fwd(x["q"], x["k"], x["v"], d, cu, o=out["o"], lse=out["lse"])
        lib.attn_bwd(x["q"], x["k"], x["v"], out["o"], out["lse"], x["do"], d, cu, dq=out["dq"], dk=out["dk"],
                     dv=out["dv"], ws=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for rep in range(3):
        x["q"].mul_(0.5)                          # new inputs between the replays, eager work on them
        step()
        torch.cuda.synchronize()
        ref = {n: t.clone() for n, t in out.items()}
        for t in out.values():
            t.view(torch.uint8).fill_(0xA5 + rep)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], ref[n]) for n in out), rep


def test_offsets_past_32_bits(gpu_lib):
    """The last rows of tensors over 4 GiB (q, o, do, dq) give the bits of the same sequences
    at the front of the same tensors."""
    lib, d, hq, hkv, t, n = gpu_lib, 128, 64, 8, 270000, 300
    big = {}
    for k, v in _case(n, hq, hkv, d).items():
        v = to_dev_bf16(v)
        big[k] = torch.empty(t, v.shape[1], dtype=torch.bfloat16, device="cuda")
        big[k][:n], big[k][t - n:] = v, v
    assert big["q"].numel() * 2 > 1 << 32
    res = []
    for first in (0, t - n):
        cu = torch.tensor([first, first + n - 100, first + n], dtype=torch.int32).cuda()
        o, lse = lib.attn_fwd(big["q"], big["k"], big["v"], d, cu)
        g = lib.attn_bwd(big["q"], big["k"], big["v"], o, lse, big["do"], d, cu)
        res.append([x[first:first + n].clone() for x in (o, *g)] + [lse[:, first:first + n].clone()])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*res))
    assert all(torch.isfinite(a.float()).all() and a.any() for a in res[0])


def test_python_refusals(gpu_lib):
    lib = gpu_lib
    q = torch.zeros(8, 128, dtype=torch.bfloat16, device="cuda")
    k = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError, match="heads"):
        lib.attn_fwd(q[:, :100].contiguous(), k, k, 64)
    with pytest.raises(ValueError, match="contiguous"):
        lib.attn_fwd(torch.zeros(128, 8, dtype=torch.bfloat16, device="cuda").t(), k, k, 64)
    with pytest.raises(TypeError, match="bfloat16"):
        lib.attn_fwd(q.float(), k, k, 64)
    with pytest.raises(TypeError, match="int32"):
        lib.attn_fwd(q, k, k, 64, cu_seqlens=torch.tensor([0, 8]).cuda())
    with pytest.raises(ValueError, match="shape"):
        lib.attn_fwd(q, k, k[:4], 64)
    with pytest.raises(ValueError, match="GPU"):
        lib.attn_fwd(q, k, k, 64, cu_seqlens=torch.tensor([0, 8], dtype=torch.int32))
    with pytest.raises(lib.Nf4Error, match="head_dim"):
        lib.attn_fwd(q, q, q, 16)
    with pytest.raises(lib.Nf4Error, match="scale"):
        lib.attn_fwd(q, k, k, 64, scale=-1.0)
    with pytest.raises(lib.Nf4Error, match="workspace"):
        o, lse = lib.attn_fwd(q, k, k, 64)
        lib.attn_bwd(q, k, k, o, lse, q, 64, ws=lib.workspace(256)[:16])
    o, lse = lib.attn_fwd(q[:0], k[:0], k[:0], 64)   # no rows: a no-op
    assert o.shape == (0, 128) and lse.shape == (2, 0)
    lib.attn_bwd(q[:0], k[:0], k[:0], o, lse, o, 64)


def _away(t, hq, hkv, d, k_scores):
    """q and k whose score at key j is about k_scores[j] for every row, heads, elements and rows varying."""
    c = _case(t, hq, hkv, d)
    # E|N| = 0.8: a dot product of D magnitudes is 0.64 D, scaled 0.64 sqrt(D)
    c["q"] = _bits(np.abs(O.bf16_bits_to_f64(c["q"])) / 1.5)
    c["k"] = _bits(np.abs(O.bf16_bits_to_f64(c["k"])) * (np.asarray(k_scores) / (0.64 * d ** 0.5))[:, None])
    return c


# (query heads, kv heads) whose 130 rows take the forward's small and its full workgroups, and the
# backward's one launch and its two
FILLS = {32: (512, 256), 64: (384, 192), 128: (256, 128)}


@pytest.mark.parametrize("full", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_scores_far_below_zero(gpu_lib, d, full):
    """Rows whose first keys' scores, or all of them, lie far below zero (e^S is zero in fp32): rising
    and falling along the keys, at the first keys only, and in sequences of one token."""
    t = 130
    hq, hkv = FILLS[d] if full else (2, 1)
    ramp = np.linspace(-1000.0, -100.0, t)
    for k_scores in (ramp, ramp[::-1]):
        for causal in (True, False):
            _check(gpu_lib, _away(t, hq, hkv, d, k_scores), d, causal=causal)
    for first in (32, 64):
        _check(gpu_lib, _away(t, hq, hkv, d, np.where(np.arange(t) < first, -400.0, 2.0)), d)
    _check(gpu_lib, _away(t, hq, hkv, d, ramp), d, [1, 1, 0, 31, 1, 65, 1, 30])
    _check(gpu_lib, _away(t, hq, hkv, d, np.full(t, -250.0)), d, [1] * t)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d,hq,hkv", [(64, 256, 128), (128, 256, 64), (32, 352, 352)])
def test_calls_that_fill_the_card(gpu_lib, d, hq, hkv, causal):
    """Three row tiles of enough heads for the forward's full workgroups and the backward's dq and dk/dv in
    launches of their own, one sequence and several."""
    _check(gpu_lib, _case(260, hq, hkv, d), d, causal=causal)
    if causal:
        _check(gpu_lib, _case(260, hq, hkv, d), d, [3, 0, 130, 127])
