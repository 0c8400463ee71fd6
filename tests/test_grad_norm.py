"""ra_grad_norm against the 64-bit norm, over odd lists of tensors.

Tolerance: squares and their sums in fp32 along chains of at most n/32 + 64
terms per thread, CTA partials rounded once, the rest in fp64: with u = 2^-24
the sum is relatively off by at most (chain + 4) u, and the square root halves
that. Chains are bounded by the elements a thread sees: count / 256 + 64 here."""

import math

import pytest
import torch

U = 2.0 ** -24
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16


@pytest.fixture(scope="module")
def ra():
    from ring_all_reduce_02_gb300 import build, ra as binding

    build.build()
    return binding


def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def run(ra, grads, max_norm=1.0, prescale=1.0, ws=None):
    out = torch.full((2,), -1.0, device="cuda")
    if ws is None:
        ws = torch.zeros(ra.ra_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
    ra.ra_grad_norm(grads, max_norm, out, ws, prescale=prescale)
    torch.cuda.synchronize()
    return [float(v) for v in out.double().cpu()]


def check(ra, grads, max_norm=1.0, prescale=1.0, ws=None):
    norm, scale = run(ra, grads, max_norm, prescale, ws)
    want = math.sqrt(sum(float((g.double() * prescale).square().sum()) for g in grads))
    n = sum(g.numel() for g in grads)
    tol = (n / 256 + 64 + 8) * U / 2 + 2 * U
    assert abs(norm - want) <= tol * want
    # denormal squares (fp32) are only possible below 1e-19, which no case here has
    assert abs(scale - prescale * min(1.0, max_norm / (want + 1e-6))) <= (tol + 4 * U) * abs(prescale)


def tensors(counts, dtype, seed, shift=0, std=1e-2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    flat = torch.randn(sum(counts) + shift, generator=gen, device="cuda").mul_(std).to(dtype)
    out, at = [], shift
    for c in counts:
        out.append(flat[at:at + c])
        at += c
    return out


LISTS = [[1], [2], [31], [255, 1, 0, 7], [4096], [4097], [100000, 3, 50000], [1] * 40, [17] * 700, [1000003], [5, 3000001, 11],
         list(range(0, 1500, 7)), [33] * 3000]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, F16, BF16])
@pytest.mark.parametrize("k", range(len(LISTS)))
def test_norm(ra, dtype, k):
    gpu()
    for shift in (0, 1, 5):
        check(ra, tensors(LISTS[k], dtype, 10 * k + shift, shift))


@pytest.mark.gpu
def test_every_element_counts_once(ra):
    # ones: the sum of squares is the count, exact in fp32 below 2^24 whatever the order
    gpu()
    ws = torch.zeros(ra.ra_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
    for counts in ([1], [3, 5], [4095], [12345, 0, 777], [8000000], [1999, 2000] * 900, [3] * 4001):
        for dtype in (F32, BF16):
            g = [torch.ones(c, dtype=dtype, device="cuda") for c in counts]
            assert run(ra, g, ws=ws)[0] == float(torch.tensor(float(sum(counts))).sqrt())


@pytest.mark.gpu
def test_more_than_32_bits_of_elements(ra):
    # 2^32 + 5 ones and a 300: every thread's and CTA's sums stay below 2^24, so that they are exact
    gpu()
    n = (1 << 32) + 6
    g = torch.ones(n, dtype=BF16, device="cuda")
    g[-1] = 300.0
    want = float(torch.tensor(n - 1 + 90000.0, dtype=torch.float64).sqrt())
    assert abs(run(ra, [g])[0] - want) <= 2 * U * want


@pytest.mark.gpu
def test_clip_scale_and_prescale(ra):
    gpu()
    g = tensors([5000, 123], F32, 3, std=1.0)
    for max_norm, prescale in ((1.0, 1.0), (1e9, 1.0), (math.inf, 1.0), (0.0, 1.0), (3.0, 1.0 / 1024), (0.01, 1.0 / 1024), (2.0, -1.0)):
        check(ra, g, max_norm, prescale)
    assert run(ra, [], 1.0) == [0.0, 1.0]
    assert run(ra, [torch.zeros(100, device="cuda")], 1.0, prescale=0.5) == [0.0, 0.5]


@pytest.mark.gpu
def test_not_finite(ra):
    gpu()
    ws = torch.zeros(ra.ra_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
    for dtype in (F32, F16, BF16):
        for bad in (math.inf, -math.inf, math.nan):
            g = tensors([1000, 70001], dtype, 4)
            g[1][70000] = bad
            norm, scale = run(ra, g, ws=ws)
            assert not math.isfinite(norm) and math.isnan(scale)
            check(ra, tensors([1000, 70001], dtype, 4), ws=ws)  # the workspace is as good as new
    assert run(ra, [torch.full((4,), 1e20, device="cuda")])[0] == math.inf  # the squares pass fp32


@pytest.mark.gpu
def test_same_bits_every_time(ra):
    gpu()
    g = tensors([3000001, 12345, 7], BF16, 8)
    ws = torch.zeros(ra.ra_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
    assert len({tuple(run(ra, g, ws=ws)) for _ in range(10)}) == 1


@pytest.mark.gpu
def test_another_stream_and_a_graph(ra):
    gpu()
    g = ra.grad_tensors(tensors([300001, 12345, 7], F32, 8))
    ws = torch.zeros(ra.ra_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
    want = run(ra, g, ws=ws)
    out = torch.zeros(2, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    ra.ra_grad_norm(g, 1.0, out, ws, stream=side)
    torch.cuda.synchronize()
    assert out.tolist() == [pytest.approx(v, rel=0, abs=0) for v in want]
    out.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        ra.ra_grad_norm(g, 1.0, out, ws)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert out.tolist() == want


def test_refusals(ra):
    import ctypes

    base, mb = 0x7F0000000000, 1 << 20

    def call(grads=(base, base + mb), counts=(1000, 1000), dt=0, prescale=1.0, max_norm=1.0, out=base + 4 * mb,
             ws=base + 5 * mb, nws=None, n=None):
        nws = ra.ra_grad_norm_workspace() if nws is None else nws
        c = (ctypes.c_size_t * len(counts))(*counts)
        return ra.lib().ra_grad_norm(ra.ptr_array(grads), c, len(counts) if n is None else n, dt, prescale, max_norm, out, ws,
                                     nws, None)

    bad, alias = ra.RA_ERR_INVALID_ARG, ra.RA_ERR_ALIAS
    assert call(dt=3) == ra.RA_ERR_UNSUPPORTED and call(dt=9) == bad
    assert call(n=-1) == call(grads=(base, 0)) == call(grads=(base, base + 2)) == call(counts=(1 << 58, 1)) == bad
    assert call(max_norm=-1.0) == call(max_norm=math.nan) == call(prescale=math.inf) == call(prescale=math.nan) == bad
    assert call(out=0) == call(out=base + 1) == call(ws=0) == call(ws=base + 5 * mb + 8) == call(nws=16) == bad
    assert call(out=base + 4) == call(ws=base + mb) == call(out=base + 5 * mb) == alias
    with pytest.raises(ValueError, match="CUDA"):
        ra.grad_tensors([torch.zeros(3)])
