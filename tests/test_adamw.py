"""ra_adamw against the formula in 64 bits.

Tolerances, with u = 2^-24 and before any run: each moment is two rounded
products and a rounded sum (with the rounded coefficients and the scaled
gradient at most 4 u of its terms' magnitudes); the denominator is relatively
off by half of v's error and at most 8 u for its own operations, the quotient
by 4 u more, which leaves room for square roots and quotients of a few ulp.
8-bit moments are checked against the rounding rule itself: rounding is
monotone, so the stored value must lie between the ones that the exact value
times 1 -+ 2^-19 rounds to with the same random bits."""

import math

import numpy as np
import pytest
import torch

U = 2.0 ** -24
ROUND = {torch.float32: U, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
F32, F16, BF16 = torch.float32, torch.float16, torch.bfloat16
F8 = torch.float8_e4m3fn
MASK = 0xFFFFFFFF
BLOCK = 256
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8)


@pytest.fixture(scope="module")
def ra():
    from ring_all_reduce_02_gb300 import build, ra as binding

    build.build()
    return binding


def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


# ---- the definition, in 64 bits --------------------------------------------------


def mix(x):
    x = np.asarray(x, dtype=np.uint64) & MASK
    x = x ^ (x >> 16)
    x = (x * 0xB7E15163) & MASK
    x = x ^ (x >> 15)
    x = (x * 0x9E3779B9) & MASK
    return x ^ (x >> 16)


def random_bits(seed, step, ordinal, n):
    key = int(mix((seed & MASK) + int(mix((seed >> 32) + step * 0x9E3779B9))))
    key = int(mix(key + ordinal * 0xB7E15163))
    i = np.arange(n, dtype=np.uint64)
    return mix((i * 0x9E3779B9 + key) & MASK)


def round_e4m3(t, bits):
    """|t| <= 448 to e4m3: up or down by 16 random bits in the normal range, to nearest even below it."""
    t = np.minimum(np.abs(t), 448.0)
    mant, expo = np.frexp(t)
    q = np.ldexp(np.floor(mant * 16 + bits / 65536.0), expo - 4)
    return np.rint(np.minimum(q, 448.0) * 512) / 512


def step64(p, g, m, v, wd, scale, step, lr, beta1, beta2, eps, underflow=False):
    g = g * scale
    m, v = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    if underflow:  # the operations are fp32: squares of values below 1e-19 leave its normal range (from v = 0)
        g32 = g.astype(np.float32)
        v = (np.float32(1 - beta2) * g32 * g32).astype(np.float64)
    d = np.sqrt(v) / math.sqrt(1 - beta2 ** step) + eps
    return p * (1 - lr * wd) - lr / (1 - beta1 ** step) * m / d, m, v


class Case:
    """Tensors of a step, cut from flat buffers at `shift`ed offsets, or allocated one by one."""

    def __init__(self, counts, pdt, gdt, eight, copy=None, seed=0, shift=0, flat=True, zeros=False):
        gen = torch.Generator().manual_seed(seed)
        self.counts, self.eight = counts, eight

        def cut(dtype, std, square=False):
            if flat:
                base = torch.zeros(sum(counts) + shift + 1, dtype=F32)
                at = np.cumsum([shift] + counts[:-1])
            else:
                base, at = None, None
            out = []
            values = [torch.zeros(c) if zeros and dtype != gdt else torch.randn(c, generator=gen) * std for c in counts]
            values = [x.square() if square else x for x in values]
            if flat:
                for a, c, x in zip(at, counts, values):
                    base[a:a + c] = x
                base = base.to(dtype).cuda()
                return [base[a:a + c] for a, c in zip(at, counts)]
            return [x.to(dtype).cuda() for x in values]

        self.p, self.g = cut(pdt, 0.5), cut(gdt, 0.1)
        self.copies = cut(copy, 1.0) if copy else None
        if not eight:
            self.m, self.v = cut(F32, 0.05), cut(F32, 0.1, square=True)
            self.ms = self.vs = None
        else:
            self.m, self.v = cut(F8, 60.0), [x.float().abs().to(F8) for x in cut(F8, 60.0)]
            self.ms = [torch.rand(-(-c // BLOCK), generator=gen).mul(1e-3).cuda() for c in counts]
            self.vs = [torch.rand(-(-c // BLOCK), generator=gen).mul(1e-3).cuda() for c in counts]
        self.wd = [0.1 if i % 2 else 0.0 for i in range(len(counts))]

    def table(self, ra):
        scales = (self.ms, self.vs) if self.eight else ()
        return ra.adamw_tensors(self.p, self.g, self.m, self.v, *scales, weight_decay=self.wd, copies=self.copies)

    def host(self):
        out = []
        for i, n in enumerate(self.counts):
            p, g = (t[i].double().cpu().numpy() for t in (self.p, self.g))
            m, v = (t[i].float().cpu().double().numpy() for t in (self.m, self.v))
            if self.eight:
                m = m * np.repeat(self.ms[i].cpu().double().numpy(), BLOCK)[:n]
                v = (v * np.repeat(self.vs[i].cpu().double().numpy(), BLOCK)[:n]) ** 2
            out.append((p, g, m, v))
        return out

    def check(self, ra, step=3, seed=12345678901234, scale=0.75, underflow=False, **hyper):
        hyper = {**HYPER, **hyper}
        before = self.host()
        s = torch.tensor([scale], device="cuda") if scale is not None else None
        ra.ra_adamw(self.table(ra), step=step, grad_scale=s, seed=seed, **hyper)
        torch.cuda.synchronize()
        for i, (p0, g, m0, v0) in enumerate(before):
            n = self.counts[i]
            if n == 0:
                continue
            k = 1.0 if scale is None else scale
            p, m, v = step64(p0, g, m0, v0, self.wd[i], k, step, underflow=underflow, **hyper)
            sg = np.abs(g * k)
            tm = 4 * U * (hyper["beta1"] * np.abs(m0) + (1 - hyper["beta1"]) * sg)
            tv = 8 * U * v
            d = np.sqrt(v) / math.sqrt(1 - hyper["beta2"] ** step) + hyper["eps"]
            lr1 = hyper["lr"] / (1 - hyper["beta1"] ** step)
            tp = 1.01 * (4 * U * (np.abs(p0) + np.abs(p)) + lr1 * (tm + 20 * U * np.abs(m)) / d)
            for got, name in ((self.p[i], "p"), (self.copies[i] if self.copies else None, "copy")):
                if got is None:
                    continue
                tol = tp + ROUND[got.dtype] * np.abs(p) * 1.01 + 2.0 ** -25 * (got.dtype == F16)
                off = np.abs(got.double().cpu().numpy() - p)
                assert (off <= tol).all(), f"{name}[{i}]: {(off / tol).max()} of the bound"
            if not self.eight:
                for got, want, tol, name in ((self.m[i], m, tm, "m"), (self.v[i], v, tv, "v")):
                    off = np.abs(got.double().cpu().numpy() - want)
                    assert (off <= 1.01 * tol + 2.0 ** -149).all(), f"{name}[{i}]: off by {off.max()}"
                continue
            rand = random_bits(seed, step, i, n)
            for got, scales, want, tol, bits, name in ((self.m[i], self.ms[i], m, tm, rand & 0xFFFF, "m"),
                                                       (self.v[i], self.vs[i], np.sqrt(v), 8 * U * np.sqrt(v), rand >> 16, "r")):
                got, scales = got.float().cpu().double().numpy(), scales.cpu().double().numpy()
                pad = np.zeros(len(scales) * BLOCK)
                pad[:n] = np.abs(want)
                amax = pad.reshape(-1, BLOCK).max(1)
                some = amax > 2.0 ** -100
                # amax's own error is its element's, relative to what cancels in m
                pad_tol = np.zeros(len(scales) * BLOCK)
                pad_tol[:n] = tol
                rel = pad_tol.reshape(-1, BLOCK).max(1) / np.where(some, amax, 1.0) + 4 * U
                assert (np.abs(scales - np.where(some, amax / 448, 0.0)) <= rel * amax / 448 * 1.01).all(), f"{name}[{i}] scales"
                inv = np.repeat(np.where(some, 448 / np.where(some, amax, 1.0), 0.0), BLOCK)[:n]
                slack = np.repeat(rel, BLOCK)[:n] + 2.0 ** -19
                lo = round_e4m3(np.maximum(np.abs(want) - tol, 0) * inv * (1 - slack), bits)
                hi = round_e4m3((np.abs(want) + tol) * inv * (1 + slack), bits)
                if name == "r":
                    floor = np.where((want > 0) & (inv > 0), 2.0 ** -9, 0.0)
                    lo, hi = np.maximum(lo, floor), np.maximum(hi, floor)
                assert ((lo <= np.abs(got)) & (np.abs(got) <= hi)).all(), f"{name}[{i}] values"
                clear = np.abs(want) > tol
                assert (np.sign(got)[clear & (got != 0)] == np.sign(want)[clear & (got != 0)]).all(), f"{name}[{i}] signs"
                exact = lo == hi
                assert exact.mean() > 0.9 or n < 100


LISTS = [[1], [7], [256], [257], [2048, 1, 0, 300], [5000], [255, 3, 511, 1025, 77777], [64] * 20, [3] * 450 + [2500] * 2, [100003]]


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("pdt,gdt,copy", [(F32, F32, None), (F32, BF16, BF16), (F32, F16, F16), (BF16, BF16, None),
                                          (BF16, F32, None), (F16, F16, None), (F16, BF16, F32), (BF16, F16, F16),
                                          (F16, F32, BF16)])
@pytest.mark.parametrize("k", range(len(LISTS)))
def test_step(ra, eight, pdt, gdt, copy, k):
    gpu()
    Case(LISTS[k], pdt, gdt, eight, copy, seed=k).check(ra)


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("shift", [0, 1, 2, 4, 7, 8, 16])
def test_alignment(ra, eight, shift):
    gpu()
    for counts in ([10000], [1024, 4096, 999, 5000], [8] * 30 + [3001]):
        Case(counts, F32, BF16, eight, BF16, seed=shift, shift=shift).check(ra)
    Case([1000, 3000, 17], BF16, F32, eight, seed=shift, flat=False).check(ra)


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_buffers_of_different_phases(ra, eight):
    # the parameters' alignment is not the gradients', nor the moments'
    gpu()
    n = 3001
    for kp, kg, km in ((0, 1, 0), (1, 0, 0), (0, 0, 1), (3, 2, 5), (8, 4, 2)):
        c = Case([n], F32, F16, eight, seed=kp + kg)

        def moved(t, k):
            base = torch.zeros(n + 16, dtype=F32).to(t.dtype).cuda()
            base[k:k + n] = t
            return base[k:k + n]

        c.p, c.g, c.m = [moved(c.p[0], kp)], [moved(c.g[0], kg)], [moved(c.m[0], km)]
        c.check(ra)


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_hyperparameters(ra, eight):
    gpu()
    for hyper in (dict(step=1), dict(step=100000), dict(beta1=0.0), dict(beta2=0.0), dict(lr=0.0), dict(eps=1e-3), dict(scale=None),
                  dict(scale=0.0), dict(seed=0), dict(seed=(1 << 64) - 1)):
        Case([3000, 100], F32, F32, eight, seed=1).check(ra, **hyper)


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_first_step_from_zero_states_and_zero_gradients(ra, eight):
    gpu()
    c = Case([1000, 300], F32, BF16, eight, seed=2, zeros=True)
    for m in (c.ms or []) + (c.vs or []):
        m.zero_()
    c.g[1].zero_()
    c.check(ra, step=1)
    assert (c.m[1].float() == 0).all() and (c.v[1].float() == 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_scale_that_is_not_finite_skips_the_step(ra, eight, bad):
    gpu()
    c = Case([3000, 17], F32, BF16, eight, BF16, seed=3)
    lists = [t for t in (c.p, c.m, c.v, c.ms, c.vs, c.copies) if t]
    before = [[x.clone() for x in t] for t in lists]
    ra.ra_adamw(c.table(ra), step=1, grad_scale=torch.tensor([bad], device="cuda"), **HYPER)
    torch.cuda.synchronize()
    for t, b in zip(lists, before):
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(t, b))


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_a_gradient_that_is_not_finite(ra, bad):
    gpu()
    c = Case([2000], F32, F32, False, seed=4)
    c.g[0][777] = bad
    ra.ra_adamw(c.table(ra), step=1, **HYPER)
    assert not torch.isfinite(c.p[0][777]) and int(torch.isfinite(c.p[0]).sum()) == 1999
    c = Case([2000], F32, F32, True, seed=4)
    c.g[0][777] = bad
    ra.ra_adamw(c.table(ra), step=1, **HYPER)
    torch.cuda.synchronize()
    hit = torch.zeros(2000, dtype=torch.bool, device="cuda")
    hit[768:1024] = True  # its block of the 8-bit moments
    assert torch.equal(torch.isnan(c.m[0].float()), hit) and torch.equal(torch.isnan(c.v[0].float()), hit)
    assert torch.equal(torch.isnan(c.ms[0]), torch.arange(8, device="cuda") == 3)
    assert int(torch.isfinite(c.p[0]).sum()) == 1999


@pytest.mark.gpu
def test_range_of_the_8_bit_moments(ra):
    # gradients over 40 powers of ten in one tensor: tiny blocks become zeros, nothing overflows, no moment that
    # divides is lost
    gpu()
    n = 20 * BLOCK
    g = torch.randn(n, generator=torch.Generator().manual_seed(5)) * torch.logspace(-36, 4, n)
    c = Case([n], F32, F32, True, seed=5, zeros=True)
    c.g[0].copy_(g)
    c.ms[0].zero_(), c.vs[0].zero_()
    c.check(ra, step=1, underflow=True)
    r = c.v[0].float().view(-1, BLOCK)
    live = c.vs[0] > 0
    assert live.any() and not live.all()
    g32 = g.numpy() * np.float32(0.75)
    v32 = torch.from_numpy(np.float32(0.01) * g32 * g32).cuda().view(-1, BLOCK)  # zero where the square underflows
    assert (r[live][v32[live] != 0] > 0).all()


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_more_than_32_bits_of_elements(ra, eight):
    # a tensor of 2^32 + 1007 elements: its last 2031 against the formula, the random bits of their places included
    gpu()
    n, tail = (1 << 32) + 1007, 2031
    start = n - tail  # 2^32 - 1024: on a block, and across 2^32
    gen = torch.Generator(device="cuda").manual_seed(11)
    p, g = torch.zeros(n, dtype=BF16, device="cuda"), torch.zeros(n, dtype=BF16, device="cuda")
    p[start:], g[start:] = torch.randn(tail, generator=gen, device="cuda"), torch.randn(tail, generator=gen, device="cuda")
    if eight:
        m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(F8) for _ in range(2))
        state = (m, v, *(torch.zeros(-(-n // BLOCK), device="cuda") for _ in range(2)))
    else:
        m, v = state = [torch.zeros(n, device="cuda") for _ in range(2)]
    p0, g0 = p[start:].double().cpu().numpy(), g[start:].double().cpu().numpy()
    ra.ra_adamw(ra.adamw_tensors([p], [g], *([s] for s in state)), step=1, seed=5, **HYPER)
    want, m1, v1 = step64(p0, g0, 0 * p0, 0 * p0, 0.0, 1.0, 1, **HYPER)
    off = np.abs(p[start:].double().cpu().numpy() - want)
    assert (off <= 2.0 ** -8 * np.abs(want) + 1e-5 * HYPER["lr"]).all()
    assert float(p[:start].abs().max()) == 0.0
    if not eight:
        assert np.allclose(m[start:].double().cpu().numpy(), m1, rtol=8 * U, atol=0)
        return
    i = np.arange(start, n, dtype=np.uint64)
    key = int(mix((5 & MASK) + int(mix(0 + 1 * 0x9E3779B9))))
    key = int(mix(key))
    bits = mix(((i & MASK) * 0x9E3779B9 + (i >> np.uint64(32)) * 0xB7E15163 + key) & MASK)
    for got, x, rand in ((m, m1, bits & 0xFFFF), (v, np.sqrt(v1), bits >> 16)):
        got = np.abs(got[start:].float().cpu().double().numpy())
        pad = np.zeros(-(-tail // BLOCK) * BLOCK)
        pad[:tail] = np.abs(x)
        inv = np.repeat(448 / pad.reshape(-1, BLOCK).max(1), BLOCK)[:tail]
        lo, hi = (round_e4m3(np.abs(x) * inv * (1 + e), rand) for e in (-(2.0 ** -19), 2.0 ** -19))
        assert ((lo <= got) & (got <= hi)).all() and (lo == hi).mean() > 0.9


@pytest.mark.gpu
def test_stochastic_rounding_is_unbiased(ra):
    # a second moment that shrinks by 3% (its root by 1.5%): nearest rounding would leave it where it was
    gpu()
    n, trials = 16 * BLOCK, 400
    total = torch.zeros(n, dtype=torch.float64, device="cuda")
    gen = torch.Generator().manual_seed(6)
    r0 = (torch.rand(n, generator=gen) * 300 + 100).to(F8).cuda()
    r0.view(-1, BLOCK)[:, 0] = torch.tensor(448.0).to(F8)
    g = torch.zeros(n).cuda()
    g.view(-1, BLOCK)[:, 0] = 448.0  # keeps each block's scale, so the others' shrinking falls between the values
    for k in range(trials):
        r = r0.clone()
        vs = torch.ones(n // BLOCK, device="cuda")
        t = ra.adamw_tensors([torch.zeros(n, device="cuda")], [g], [torch.zeros(n).to(F8).cuda()], [r],
                             [torch.zeros(n // BLOCK, device="cuda")], [vs])
        ra.ra_adamw(t, step=1 + k, lr=0.0, beta2=0.97, seed=99)
        total += (r.float().view(-1, BLOCK) * vs[:, None]).view(-1).double()
    want = torch.sqrt(0.97 * r0.float().double().square() + 0.03 * g.double().square())
    # a stored value's deviation is at most half of its 32-wide step; the mean's is 16 / sqrt(trials) = 0.8
    off = (total / trials - want).abs()
    assert float(off.max()) <= 6 * 16 / math.sqrt(trials)
    assert abs(float((total / trials - want).mean())) <= 6 * 16 / math.sqrt(trials * n)


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_repeats_exactly_on_any_stream_and_in_a_graph(ra, eight):
    gpu()
    hyper = dict(HYPER, step=5, seed=42)
    cases = [Case([70000, 33, 4096], F32, BF16, eight, BF16, seed=7) for _ in range(3)]
    torch.cuda.synchronize()
    ra.ra_adamw(cases[0].table(ra), **hyper)
    side = torch.cuda.Stream()
    ra.ra_adamw(cases[1].table(ra), stream=side, **hyper)
    graph = torch.cuda.CUDAGraph()
    table = cases[2].table(ra)
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        ra.ra_adamw(table, **hyper)
    graph.replay()
    torch.cuda.synchronize()
    for c in cases[1:]:
        for name in ("p", "m", "v", "ms", "vs", "copies"):
            for x, y in zip(getattr(c, name) or [], getattr(cases[0], name) or []):
                assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# ---- refusals: fake addresses that are never dereferenced ---------------------------

BASE = 0x7F0000000000
MB = 1 << 20


def refuse(ra, pdt=0, gdt=0, n=2, options=None, **fields):
    state = (options or {}).get("state", 0)
    table = (ra.AdamwTensor * 2)()
    for i, t in enumerate(table):
        at = BASE + i * 64 * MB
        t.param, t.grad, t.exp_avg, t.exp_avg_sq = at, at + 4 * MB, at + 8 * MB, at + 12 * MB
        t.exp_avg_scale, t.exp_avg_sq_scale = at + 16 * MB, at + 17 * MB
        t.count, t.weight_decay = 1000, 0.1
    for k, v in fields.items():
        setattr(table[1], k, v)
    o = ra.AdamwOptions(1e-3, 0.9, 0.999, 1e-8, 1, None, state, 0, 0)
    for k, v in (options or {}).items():
        setattr(o, k, v)
    import ctypes

    return ra.lib().ra_adamw(table, n, pdt, gdt, ctypes.byref(o), None)


def test_refusals(ra):
    bad, alias, no = ra.RA_ERR_INVALID_ARG, ra.RA_ERR_ALIAS, ra.RA_ERR_UNSUPPORTED
    assert refuse(ra, pdt=3) == refuse(ra, gdt=3) == no
    assert refuse(ra, pdt=8) == refuse(ra, gdt=-1) == refuse(ra, n=-1) == bad
    for k, v in (("lr", -1.0), ("lr", math.nan), ("beta1", 1.0), ("beta1", -0.1), ("beta2", 1.5), ("beta2", math.nan),
                 ("eps", -1e-8), ("eps", math.inf), ("step", 0), ("step", -3), ("state", 2), ("grad_scale", BASE + 2)):
        assert refuse(ra, options={k: v}) == bad, k
    for k in ("param", "grad", "exp_avg", "exp_avg_sq"):
        assert refuse(ra, **{k: None}) == refuse(ra, **{k: BASE + 40 * MB + 2}) == bad, k
    assert refuse(ra, weight_decay=-1.0) == refuse(ra, weight_decay=math.nan) == refuse(ra, count=1 << 58) == bad
    for k in ("exp_avg_scale", "exp_avg_sq_scale"):
        assert refuse(ra, options={"state": 1}, **{k: None}) == bad
        assert refuse(ra, options={"state": 1}, **{k: BASE + 40 * MB + 2}) == bad
    assert refuse(ra, copy=BASE + 40 * MB, options={"copy_dtype": 3}) == no
    assert refuse(ra, copy=BASE + 40 * MB, options={"copy_dtype": 5}) == bad
    # written buffers overlap nothing: inside a tensor, between tensors, or the scale
    assert refuse(ra, param=BASE + 64 * MB + 4 * MB) == refuse(ra, param=BASE + 400) == refuse(ra, exp_avg=BASE + 64 * MB) == alias
    assert refuse(ra, copy=BASE + 8 * MB) == refuse(ra, options={"grad_scale": BASE + 64}) == alias
    assert refuse(ra, options={"state": 1}, exp_avg_scale=BASE + 17 * MB) == alias
    assert refuse(ra, exp_avg=BASE + 12 * MB + 3999) == bad and refuse(ra, exp_avg=BASE + 12 * MB + 3996) == alias
    # gradients may overlap each other: the call then only fails where there is no GPU
    assert refuse(ra, n=0) == ra.RA_SUCCESS
    # empty tensors need no memory
    assert refuse(ra, n=0, count=0, param=None) == ra.RA_SUCCESS


def test_binding_refusals(ra):
    z = [torch.zeros(3)]
    with pytest.raises(ValueError, match="CUDA"):
        ra.adamw_tensors(z, z, z, z)
    with pytest.raises(ValueError, match="entry"):
        ra.adamw_tensors(z, z + z, z, z)
    with pytest.raises(ValueError, match="scales"):
        ra.adamw_tensors(z, z, z, z, z)


def test_random_bits_are_even(ra):
    # the hash on the host: both halves uniform, and neighbours, tensors and steps unrelated
    a = random_bits(1, 1, 0, 1 << 18)
    others = [np.roll(a, 1), random_bits(1, 1, 1, 1 << 18), random_bits(1, 2, 0, 1 << 18), random_bits(2, 1, 0, 1 << 18)]
    for half in (a & 0xFFFF, a >> 16):
        counts = np.bincount((half >> 8).astype(int), minlength=256)
        # 1024 expected in each of 256 cells, deviation 32: chi-square 255 +- 23
        chi = float(((counts - 1024.0) ** 2 / 1024.0).sum())
        assert abs(chi - 255) < 6 * 23
    for b in others:
        for x, y in ((a & 0xFFFF, b & 0xFFFF), (a >> 16, b >> 16), (a & 0xFFFF, b >> 16)):
            r = np.corrcoef(x.astype(float), y.astype(float))[0, 1]
            assert abs(r) < 6 / 512  # 1 / sqrt(2^18) a deviation
