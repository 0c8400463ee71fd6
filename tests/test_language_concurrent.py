"""The embedding and the cross entropy from several host threads at once, each with its own stream and buffers, and
captured into a graph that is replayed on other tokens: the bits are those that a call alone has."""

import threading

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def ra():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from ring_all_reduce_02_gb300 import build, ra as binding

    build.build()
    return binding


class Step:
    """Both ends of a tied model without what lies between: lookup, loss, gradients, the lookup's gradient on top."""

    def __init__(self, ra, rows, cols, vocab, dtype, seed):
        self.ra, self.gen, self.vocab = ra, torch.Generator(device="cuda").manual_seed(seed), vocab
        self.table = (torch.randn(vocab, cols, generator=self.gen, device="cuda") * 0.1).to(dtype)
        self.tokens, self.targets = (torch.zeros(rows, dtype=torch.int64, device="cuda") for _ in range(2))
        self.hidden, self.dhidden = (torch.zeros(rows, cols, dtype=dtype, device="cuda") for _ in range(2))
        self.loss, self.lse = (torch.zeros(rows, device="cuda") for _ in range(2))
        self.dtable = torch.zeros(vocab, cols, dtype=dtype, device="cuda")
        sizes = (ra.ra_cross_entropy_workspace(self.hidden, self.table), ra.ra_cross_entropy_workspace(self.hidden, self.table, backward=True),
                 ra.ra_embedding_workspace(rows, cols, vocab))
        self.scratch = [torch.zeros(n, dtype=torch.uint8, device="cuda") for n in sizes]
        self.outputs = [self.hidden, self.loss, self.lse, self.dhidden, self.dtable]
        self.draw()

    def draw(self):
        rows = self.tokens.numel()
        self.tokens.copy_(torch.randint(0, self.vocab, (rows,), generator=self.gen, device="cuda") ** 2 // self.vocab)
        self.targets.copy_(torch.randint(0, self.vocab, (rows,), generator=self.gen, device="cuda"))
        self.targets[torch.rand(rows, generator=self.gen, device="cuda") < 0.3] = -100

    def run(self, stream=None):
        ra, s = self.ra, dict(stream=stream)
        ra.ra_embedding_forward(self.table, self.tokens, self.hidden, scale=2.0, **s)
        ra.ra_cross_entropy_forward(self.hidden, self.table, self.targets, self.loss, self.lse, workspace=self.scratch[0], **s)
        ra.ra_cross_entropy_backward(self.hidden, self.table, self.targets, self.lse, None, self.dhidden, self.dtable, workspace=self.scratch[1], **s)
        ra.ra_embedding_backward(self.dhidden, self.tokens, self.dtable, scale=2.0, accumulate=True, workspace=self.scratch[2], **s)

    def alone(self):
        self.run()
        torch.cuda.synchronize()
        return [t.clone() for t in self.outputs]

    def holds(self, want):
        return all(torch.equal(a, b) for a, b in zip(self.outputs, want))


# few rows and many, the weight in place and packed, a sort by one cluster and one of several passes
SIZES = [(7, 256, 9000, BF16), (600, 136, 20011, F16), (1500, 515, 3001, BF16), (300, 512, 140_000, F16)]


def test_from_several_threads(ra):
    steps = [Step(ra, *size, seed=i) for i, size in enumerate(SIZES)]
    want = [s.alone() for s in steps]
    streams = [torch.cuda.Stream() for _ in steps]
    for s in steps:
        for t in s.outputs:
            t.zero_()
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(steps))

    def work(step, stream):
        try:
            start.wait()
            for _ in range(20):
                step.run(stream)
        except Exception as e:  # a thread's exception would be lost
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(steps, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed
    assert all(s.holds(w) for s, w in zip(steps, want))


@pytest.mark.parametrize("size", SIZES, ids=lambda s: f"{s[0]}x{s[1]}x{s[2]}")
def test_replayed_on_other_tokens(ra, size):
    step = Step(ra, *size, seed=9)
    first = step.alone()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step.run()
    graph.replay()
    torch.cuda.synchronize()
    assert step.holds(first)
    step.draw()
    want = step.alone()
    assert not all(torch.equal(a, b) for a, b in zip(first, want))
    for t in step.outputs:
        t.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert step.holds(want)


def test_two_graphs_share_a_workspace(ra):
    # replayed one after the other on one stream
    a, b = (Step(ra, 200, 256, 5000, BF16, seed=i) for i in (1, 2))
    b.scratch = a.scratch
    want = [a.alone(), b.alone()]
    graphs, side = [], torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for step in (a, b):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.stream(side), torch.cuda.graph(graphs[-1], stream=side):
            step.run()
    for t in a.outputs + b.outputs:
        t.zero_()
    torch.cuda.synchronize()
    for graph in (*graphs, graphs[1], graphs[0]):
        graph.replay()
    torch.cuda.synchronize()
    assert a.holds(want[0]) and b.holds(want[1])
