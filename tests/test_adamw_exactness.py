"""What ra_adamw stores, bit for bit: the moments are the fp32 formula written out, every product and sum rounded on
its own, and the 8-bit values what include/ra.h makes of them. The reference below is numpy's fp32, whose operations
round once each."""

import numpy as np
import pytest
import torch

from test_adamw import BF16, BLOCK, F8, F16, F32, HYPER, Case, gpu, random_bits, refuse

f32 = np.float32


@pytest.fixture(scope="module")
def ra():
    from ring_all_reduce_02_gb300 import build, ra as binding

    build.build()
    return binding


def moments(g, m, v, scale, beta1, beta2):
    g = g * f32(scale)
    m = m * f32(beta1) + g * f32(1 - beta1)
    v = v * f32(beta2) + (g * f32(1 - beta2)) * g
    return m, v


def stored(x, bits, root):
    """[blocks, 256] fp32 -> the e4m3 values and the scales that stand for them."""
    amax = np.abs(x).max(1)
    some = amax > f32(2.0 ** -100)
    inv = np.where(some, f32(448) * (f32(1) / np.where(some, amax, f32(1))), f32(0))
    t = x * inv[:, None]
    t = ((t.view(np.uint32) + (bits.astype(np.uint32) << 4)) & np.uint32(0xFFF00000)).view(f32)
    if root:
        t = np.where((x > 0) & some[:, None], np.maximum(t, f32(2.0 ** -9)), t)
    t = torch.from_numpy(np.clip(t, f32(-448), f32(448))).to(F8).float().numpy()
    return t, np.where(some, amax * (f32(1) / f32(448)), f32(0))


def blocks_of(x):
    out = np.zeros((-(-len(x) // BLOCK), BLOCK), dtype=x.dtype)
    out.reshape(-1)[:len(x)] = x
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("pdt,gdt", [(F32, BF16), (BF16, F32), (F16, F16)])
@pytest.mark.parametrize("counts,shift", [([100003], 0), ([4096, 512, 65536], 0), ([5000, 255, 1, 7777], 3), ([512] * 60, 8)])
def test_moments_bit_for_bit(ra, eight, pdt, gdt, counts, shift):
    gpu()
    c = Case(counts, pdt, gdt, eight, seed=shift + len(counts), shift=shift)
    for g, v in zip(c.g, c.v):  # zero gradients and zero second moments, alone and together
        g[::7] = 0
        v.view(torch.uint8 if eight else F32)[::5] = 0
    if eight:
        for scales in c.vs:
            scales[::3] = 0
    seed, step, scale = 987654321012345, 11, 0.7
    before = []
    for i in range(len(counts)):
        g, m, v = (t[i].float().cpu().numpy() for t in (c.g, c.m, c.v))
        if eight:
            spread = [np.repeat(s[i].cpu().numpy(), BLOCK)[:counts[i]] for s in (c.ms, c.vs)]
            m, v = m * spread[0], v * spread[1]
            v = v * v
        before.append((g, m, v))
    ra.ra_adamw(c.table(ra), step=step, grad_scale=torch.tensor([scale], device="cuda"), seed=seed, **HYPER)
    torch.cuda.synchronize()
    for i, (g, m, v) in enumerate(before):
        m, v = moments(g, m, v, scale, HYPER["beta1"], HYPER["beta2"])
        if not eight:
            assert np.array_equal(c.m[i].cpu().numpy(), m) and np.array_equal(c.v[i].cpu().numpy(), v)
            continue
        bits = random_bits(seed, step, i, counts[i])
        for got, scales, x, b, root in ((c.m[i], c.ms[i], m, bits & 0xFFFF, False), (c.v[i], c.vs[i], np.sqrt(v), bits >> 16, True)):
            want, want_scales = stored(blocks_of(x), blocks_of(b), root)
            assert np.array_equal(scales.cpu().numpy(), want_scales)
            assert np.array_equal(got.float().cpu().numpy(), want.reshape(-1)[:counts[i]])


@pytest.mark.gpu
def test_square_root_of_every_significand(ra):
    # v = fl(fl(s^2)/2 + fl(g/2 g)) with s and g chosen so that v is the wanted one; a block's scale is then
    # fl(sqrt(v) / 448), which tells neighbouring roots apart where their significand is below 1.75 (and half of
    # the others)
    gpu()
    per = 1 << 20  # significands at a time, a block of equal elements for each
    seen = 0
    for octave in (1.0, 2.0):
        for first in range(0, 1 << 23, per):
            v = ((torch.arange(first, first + per, device="cuda", dtype=torch.float64) / (1 << 23) + 1.0) * octave).float()
            ulp = 2.0 ** -23 * octave
            s = (2.0 * (v.double() - 4 * ulp)).sqrt().float()
            rest = v.double() - (s * s * 0.5).double()
            g = (2.0 * rest.clamp(min=0)).sqrt().float()
            made = s * s * 0.5 + (g * 0.5) * g
            ok = made == v
            assert float(ok.float().mean()) > 0.99
            seen += int(ok.sum())
            count = per * BLOCK
            m, r = (torch.full((count,), k, dtype=torch.uint8, device="cuda").view(F8) for k in (0, 0x38))  # 0 and 1
            ms, rs = torch.zeros(per, device="cuda"), s.clone()
            table = ra.adamw_tensors([torch.zeros(count, dtype=BF16, device="cuda")], [g.repeat_interleave(BLOCK)], [m], [r], [ms], [rs])
            ra.ra_adamw(table, lr=0.0, step=1, beta1=0.5, beta2=0.5, seed=1)
            want = made.double().sqrt().float() * torch.tensor(1.0 / 448, dtype=F32, device="cuda")
            assert torch.equal(rs, want)
    assert seen > 0.99 * (1 << 24)


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
def test_gradients_may_overlap_each_other(ra, eight):
    gpu()
    counts = [3000, 3000, 2000]
    shared, apart = (Case(counts, F32, BF16, eight, seed=3) for _ in range(2))
    flat = torch.randn(4000, generator=torch.Generator().manual_seed(1)).to(BF16).cuda()
    shared.g = [flat[:3000], flat[1000:], flat[1000:3000]]
    apart.g = [g.clone() for g in shared.g]
    for c in (shared, apart):
        ra.ra_adamw(c.table(ra), step=2, seed=5, **HYPER)
    torch.cuda.synchronize()
    for name in ("p", "m", "v", "ms", "vs"):
        for x, y in zip(getattr(shared, name) or [], getattr(apart, name) or []):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("eps", [2.0 ** -126, 1e-30])
def test_the_smallest_eps_leaves_elements_without_a_gradient(ra, eight, eps):
    gpu()
    c = Case([3000, 100], F32, F32, eight, seed=1, zeros=True)
    for t in c.g + c.m + c.v + (c.ms or []) + (c.vs or []):
        t.view(torch.uint8).zero_()
    c.p[0].fill_(3.0), c.p[1].fill_(-2.0)
    c.wd = [0.0, 0.0]
    ra.ra_adamw(c.table(ra), step=1, **{**HYPER, "eps": eps})
    assert (c.p[0] == 3.0).all() and (c.p[1] == -2.0).all()


def test_an_eps_whose_reciprocal_is_infinite_is_refused(ra):
    for eps in (2.0 ** -127, 1e-40, 1e-60, 5e-324):
        assert refuse(ra, options={"eps": eps}) == ra.RA_ERR_INVALID_ARG
