"""Calls from several host threads at once, each on its own stream and buffers: a kernel's limit of dynamic shared
memory belongs to the process, so a call that set it to its own need could have another call's launch refused. No call
may fail, and every result has to be the one it has alone."""

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from ring_all_reduce_02_gb300 import build, ra as binding

    build.build()
    return binding


def together(calls, repeats):
    """Every call repeated in a thread of its own; the statuses that were not success."""
    bad, start = [], threading.Barrier(len(calls))

    def work(call):
        start.wait()
        bad.extend(st for st in (call() for _ in range(repeats)) if st)

    threads = [threading.Thread(target=work, args=(c,)) for c in calls]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return bad


def layernorm_calls(ra, widths, rows, dtype):
    """One backward and one forward call for each width, of the C entry points, with their outputs."""
    calls, outputs, keep = [], [], []
    code = 0 if dtype == torch.float32 else 2
    for cols in widths:
        gen = torch.Generator(device="cuda").manual_seed(cols)
        x, dy = (torch.randn(rows, cols, generator=gen, device="cuda").to(dtype) for _ in range(2))
        y, dx = torch.empty_like(x), torch.empty_like(x)
        mean, rstd, dw, db = (torch.zeros(n, device="cuda") for n in (rows, rows, cols, cols))
        ws = torch.empty(ra.ra_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
        streams = [torch.cuda.Stream() for _ in range(2)]
        one, half = torch.ones(rows, device="cuda"), torch.full((rows,), 0.5, device="cuda")
        p = {k: v.data_ptr() for k, v in dict(x=x, dy=dy, y=y, dx=dx, mean=mean, rstd=rstd, dw=dw, db=db, ws=ws, one=one, half=half).items()}
        fwd = (p["x"], cols, None, None, p["y"], cols, p["mean"], p["rstd"], rows, cols, 1e-5, code, 0, streams[0].cuda_stream)
        bwd = (p["dy"], cols, p["x"], cols, None, p["half"], p["one"], p["dx"], cols, p["dw"], p["db"], 0, rows, cols, code, 0,
               p["ws"], ws.numel(), streams[1].cuda_stream)
        calls += [lambda a=fwd: ra.lib().ra_layernorm_forward(*a), lambda a=bwd: ra.lib().ra_layernorm_backward(*a)]
        outputs += [y, mean, rstd, dx, dw, db]
        keep += [x, dy, ws, one, half, streams]
    return calls, outputs, keep


# widths that share a kernel and differ in the shared memory that it takes: on the 16-byte grid, off it, and rows
# shared by several CTAs
@pytest.mark.parametrize("widths", [(1024, 2048, 4096, 6144), (6201, 7001, 7601, 8101), (17000, 18000, 19000, 20000)])
def test_layer_norm(ra, widths):
    calls, outputs, keep = layernorm_calls(ra, widths, 3, torch.bfloat16)
    torch.cuda.synchronize()
    assert not [st for st in (c() for c in calls) if st]
    torch.cuda.synchronize()
    want = [o.clone() for o in outputs]
    for o in outputs:
        o.zero_()
    torch.cuda.synchronize()
    assert not together(calls, 10000)
    assert all(torch.equal(a, b) for a, b in zip(outputs, want))


# rank counts that share a kernel and differ in the shared memory that it takes
@pytest.mark.parametrize("ranks,how", [((32, 27, 48, 40), dict(order="tree")), ((32, 64), dict(order="rabenseifner")),
                                       ((8, 11, 13, 16), dict(engine="bulk"))], ids=str)
def test_all_reduce(ra, ranks, how):
    calls, outputs, keep = [], [], []
    for n in ranks:
        count = n * 1024 + 3
        gen = torch.Generator(device="cuda").manual_seed(n)
        sends = [torch.randint(-5, 6, (count,), generator=gen, device="cuda").float() for _ in range(n)]
        recvs = [torch.zeros(count, device="cuda") for _ in range(n)]
        status, stream = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
        args = ([t.data_ptr() for t in sends], [t.data_ptr() for t in recvs], count, 0, 0, n,
                ra.ORDER_CODES[how.get("order", "ring")], 0, stream.cuda_stream, 0, ra.ENGINE_CODES[how.get("engine", "registers")],
                status.data_ptr())
        calls.append(lambda a=args: ra.call_ex("ra_allreduce_ex", *a))
        outputs.append((recvs, sum(sends)))
        keep += [sends, status, stream]
    torch.cuda.synchronize()
    assert not [st for st in (c() for c in calls) if st]
    assert not together(calls, 5000)
    for recvs, want in outputs:  # whole numbers: exact in any order
        assert all(torch.equal(t, want) for t in recvs)
