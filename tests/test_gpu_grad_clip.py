"""The gradients' global norm and clipping through the C ABI against fp64."""

import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def stream_pair_first(gpu_lib):
    """The library's compute/copy pair, made for the life of the process, before this file
    makes streams and graphs: made later, the two may fall on one hardware queue."""
    gpu_lib.pool_streams()


def _tensors(sizes, seed=0, std=1.0):
    """fp32 and bf16 in turn, each cut from a larger buffer at an odd element offset."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    out = []
    for i, n in enumerate(sizes):
        dtype = torch.float32 if i % 2 == 0 else torch.bfloat16
        buf = (torch.randn(n + 16, generator=g, device="cuda") * std).to(dtype)
        out.append(buf[i % 9:i % 9 + n])
    return out


def _norm64(ts):
    return math.sqrt(sum(float(t.double().square().sum()) for t in ts))


def _ulp(dtype):
    return torch.finfo(dtype).eps / 2            # half a step, relative


SIZES = [[1], [3, 5], [0, 7, 0, 4096], [16384, 32768, 16385, 32769, 16383], [100_003, 999_999, 8, 1_000_001],
         [33] * 300]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("in_place", [True, False])
def test_norm_and_scaling(gpu_lib, sizes, in_place):
    lib = gpu_lib
    grads = _tensors(sizes)
    before = [t.clone() for t in grads]
    outs = None if in_place else [torch.full_like(t, 9.0) for t in grads]
    gl = lib.GradList(grads, outs)
    want = _norm64(before)
    n = gl.norm()
    torch.cuda.synchronize()
    assert abs(n.item() - want) <= 2 * 2.0 ** -24 * want       # fp64 sums; one rounding to fp32
    assert all(torch.equal(a, b) for a, b in zip(grads, before))
    for max_norm in (2 * want + 1.0, 0.37 * want, 0.0):
        for t, b in zip(grads, before):
            t.copy_(b)
        n = gl.clip(max_norm)
        torch.cuda.synchronize()
        assert abs(n.item() - want) <= 2 * 2.0 ** -24 * want
        f = min(1.0, max_norm / (want + 1e-6))
        for b, t, o in zip(before, grads, gl.outs):
            exact = b.double() * f
            # the factor rounded to fp32, the product, and the product's rounding to the type
            lim = exact.abs() * (3 * 2.0 ** -24 + _ulp(b.dtype)) + 1e-44
            assert torch.all((o.double() - exact).abs() <= lim)
            if f == 1.0:
                assert torch.equal(o, b)
            if not in_place:
                assert torch.equal(t, b)
    gl.close()


def test_stack_sized_list_of_one_type(gpu_lib):
    """1120 aligned fp32 tensors (the adapters of 80 layers), more pieces than shares."""
    lib = gpu_lib
    flat = torch.randn(80 * 14 * 120_000, device="cuda")
    gl = lib.GradList(list(flat.split(120_000)), list(torch.empty_like(flat).split(120_000)))
    n = gl.clip(1.0)
    want = _norm64([flat])
    assert abs(n.item() - want) <= 2 * 2.0 ** -24 * want
    got = torch.cat(gl.outs)
    assert torch.all((got.double() - flat.double() / (want + 1e-6)).abs() <= 4 * 2.0 ** -24 * flat.double().abs() + 1e-44)


def test_huge_tiny_and_non_finite_values(gpu_lib):
    lib = gpu_lib
    for v in (1e30, 1e-30):                       # squares outside fp32
        t = torch.full((1000,), v, device="cuda")
        gl = lib.GradList([t])
        assert gl.norm().item() == pytest.approx(_norm64([t]), rel=1e-6)
    big = torch.full((4,), 3e38, device="cuda")   # the norm itself is past fp32
    gl = lib.GradList([big])
    assert math.isinf(gl.clip(1.0).item())
    assert big[0].item() == pytest.approx(0.5, rel=1e-6)
    for bad in (float("inf"), float("nan")):
        t = torch.ones(100, device="cuda")
        t[7] = bad
        o = torch.zeros_like(t)
        n = lib.GradList([t], [o]).clip(1.0)
        assert not math.isfinite(n.item())
        assert torch.equal(o.isnan(), t.isnan()) and torch.equal(o.nan_to_num(), t.nan_to_num())
    z = torch.zeros(100, device="cuda")
    gl = lib.GradList([z])
    assert gl.clip(1.0).item() == 0.0 and not z.any()
    assert lib.GradList([torch.empty(0, device="cuda")]).clip(1.0).item() == 0.0


def test_same_bits_again_on_another_stream_and_in_graphs(gpu_lib):
    lib = gpu_lib
    grads = _tensors([50_001, 70_000, 33, 16_384], seed=3)
    outs = [torch.empty_like(t) for t in grads]
    gl = lib.GradList(grads, outs)
    ref_n = gl.clip(1.5).clone()
    ref = [o.clone() for o in outs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    n = gl.clip(1.5, stream=side)
    side.synchronize()
    assert torch.equal(n, ref_n) and all(torch.equal(a, b) for a, b in zip(outs, ref))
    norm, ws = torch.empty(1, device="cuda"), lib.workspace(gl._ws_bytes)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gl.clip(1.5, norm=norm, ws=ws)
    for rep in range(3):
        grads[0].mul_(1.25)
        ref_n = gl.clip(1.5).clone()
        ref = [o.clone() for o in outs]
        ws.fill_(0xFF)
        for o in outs:
            o.fill_(rep)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(norm, ref_n) and all(torch.equal(a, b) for a, b in zip(outs, ref)), rep


def test_python_refusals(gpu_lib):
    lib = gpu_lib
    a, b = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
    with pytest.raises(ValueError, match="at least one"):
        lib.GradList([])
    with pytest.raises(ValueError, match="outs"):
        lib.GradList([a, b], [a])
    with pytest.raises(TypeError, match="bfloat16 or float32"):
        lib.GradList([a.half()])
    with pytest.raises(ValueError, match="contiguous"):
        lib.GradList([torch.zeros(8, 8, device="cuda").t()])
    with pytest.raises(lib.Nf4Error, match="overlaps"):
        lib.GradList([a, b, a])
    with pytest.raises(lib.Nf4Error, match="overlaps"):
        lib.GradList([a[:32]], [a[16:48]])
    with pytest.raises(lib.Nf4Error, match="overlaps"):
        lib.GradList([a, b], [b, torch.empty_like(b)])
    gl = lib.GradList([a, b])
    for bad in (-1.0, float("nan"), float("inf")):
        with pytest.raises(lib.Nf4Error, match="max_norm"):
            gl.clip(bad)
    with pytest.raises(lib.Nf4Error, match="workspace"):
        gl.clip(1.0, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    gl.close()
    with pytest.raises(lib.Nf4Error, match="closed"):
        gl.norm()


def test_a_list_is_not_made_within_a_capture(gpu_lib):
    """Making one waits for a copy: refused, and the capture around it stays whole."""
    lib = gpu_lib
    a, x = torch.full((64,), 2.0, device="cuda"), torch.zeros(1, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.add_(1)
        with pytest.raises(lib.Nf4Error, match="before a capture"):
            lib.GradList([a])
        x.add_(1)
    for n in (1, 2):
        graph.replay()
        torch.cuda.synchronize()
        assert x.item() == 2.0 * n
    assert lib.GradList([a]).norm().item() == 16.0


def test_list_freed_while_another_stream_still_reads_its_table(gpu_lib):
    """A list used on a side stream and dropped at once: its table's memory is not handed out
    again before that stream is done (the stream is held up by a bounded spin)."""
    lib = gpu_lib
    grads = [torch.ones(1000, device="cuda") for _ in range(200)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    gl = lib.GradList(grads)
    nbytes = gl._table.numel()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    at = gl._table.data_ptr()
    n = gl.clip(1.0, stream=side)
    del gl
    again = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert all(t.data_ptr() != at for t in again)   # checked before anything could be written there
    torch.cuda.synchronize()
    assert n.item() == pytest.approx(math.sqrt(200_000), rel=1e-6)


def test_outputs_of_a_side_stream_call_are_that_streams_memory(gpu_lib):
    """Results allocated for a call on a side stream are not blocks that the current stream
    has freed but still writes (behind a bounded spin)."""
    lib = gpu_lib
    g = torch.ones(5000, device="cuda")
    gl = lib.GradList([g])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    freed = torch.empty(1, device="cuda")
    torch.cuda._sleep(20_000_000)
    freed.fill_(7.0)                                # pending on the current stream
    at = freed.data_ptr()
    del freed
    n = gl.norm(stream=side)
    assert n.data_ptr() != at
    torch.cuda.synchronize()
    assert n.item() == pytest.approx(math.sqrt(5000), rel=1e-6)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size,max_norm", [(1e38, 1e-3), (3e38, 1e-5), (1e30, 1e-12), (1e-30, 1e-38)])
def test_factors_below_fp32s_normal_range(gpu_lib, dtype, size, max_norm):
    """max_norm / norm down to 10^-45, where fp32 holds a few bits or none: the scaled values are right
    to their own rounding all the same (values that would round below the normal range left out)."""
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    t = ((torch.rand(5000, generator=g, device="cuda") * 2 - 1) * size).to(dtype)
    want = _norm64([t])
    exact = t.double() * (max_norm / (want + 1e-6))
    gpu_lib.GradList([t]).clip(max_norm)
    torch.cuda.synchronize()
    normal = exact.abs() >= 2.0 ** -126
    assert normal.any() or max_norm == 1e-38
    # one rounding to the type, for bf16 behind one to fp32; the fp64 factor and product below 2^-48
    lim = exact.abs() * (_ulp(dtype) + 2.0 ** -24 + 2.0 ** -48) + torch.where(normal, 0.0, 2.0 ** -126)
    assert torch.all((t.double() - exact).abs() <= lim)


def test_unscaled_tensors_in_place_are_left_alone_beside_others(gpu_lib):
    """In a list of tensors in place and not, the former keep every bit when nothing is to be scaled: below
    the bound, and with a norm that is not finite, signalling NaN among the gradients."""
    for bad in (False, True):
        a, b = torch.randn(5000, device="cuda"), torch.randn(3001, device="cuda")
        if bad:
            a.view(torch.int32)[7] = 0x7F800001
            a.view(torch.int32)[4999] = 0x7FA00000
        bits, out = a.view(torch.int32).clone(), torch.zeros_like(b)
        n = gpu_lib.GradList([a, b], [a, out]).clip(1e6)
        torch.cuda.synchronize()
        assert math.isnan(n.item()) == bad
        assert torch.equal(a.view(torch.int32), bits) and torch.equal(out, b)


def test_norms_and_workspaces_over_the_lists_memory_are_refused(gpu_lib):
    """The tensors, wherever they lie in the order of addresses, their outputs and the table."""
    lib = gpu_lib
    flat = torch.ones(40_000, device="cuda")
    grads = [flat[4 * i:4 * i + 2] for i in range(1000)] + [flat[8000:8001], flat[20_000:30_000]]
    outs = grads[:1001] + [torch.zeros(10_000, device="cuda")]
    gl = lib.GradList(grads, outs)
    free_norm, free_ws = torch.empty(1, device="cuda"), lib.workspace(gl._ws_bytes)
    refused = [flat[0:1], flat[1:2], flat[2000:2001], flat[3997:3998], flat[8000:8001], flat[20_000:20_001],
               flat[29_999:30_000], outs[1001][:1], outs[1001][9999:], gl._table[:4].view(torch.float32),
               free_ws[:4].view(torch.float32)]
    for norm in refused:
        with pytest.raises(lib.Nf4Error, match="overlaps"):
            gl.norm(norm=norm, ws=free_ws)
        with pytest.raises(lib.Nf4Error, match="overlaps"):
            gl.clip(1.0, norm=norm, ws=free_ws)
    n = gl._ws_bytes // 4
    for first in (0, 8000 - n + 64, 19_968, 29_952):           # 256-byte aligned, over tensors before, behind or within
        with pytest.raises(lib.Nf4Error, match="overlaps"):
            gl.norm(norm=free_norm, ws=flat[first:first + n])
    want = math.sqrt(2000 + 1 + 10_000)
    for norm in (flat[2:3], flat[3998:3999], flat[8001:8002], flat[19_999:20_000], flat[30_000:30_001]):  # between them
        assert gl.norm(norm=norm, ws=flat[32_000:32_000 + n]).item() == pytest.approx(want, rel=1e-6)
    assert torch.all(flat[:2] == 1) and torch.all(flat[20_000:29_999] == 1)
