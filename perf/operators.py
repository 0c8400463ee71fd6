"""The operators on either side of a data-parallel gradient all-reduce, as workloads.

Layer norm (forward, and backward with the reduction of the weight's and bias's
gradients), the global gradient norm with its clip factor, and the AdamW step
over many tensors at once with its two moments in 32 bits or in 8.

``run`` computes an operator in its plain form (elementary torch operations in
fp32, rounded once at the end), or, with ``own`` set, by the library's entry
points. ``exact`` computes it in 64 bits.

Many-tensor cases keep their tensors as consecutive slices of flat buffers, as
gradient buckets do; the 8-bit moments are blocked by 256 elements from each
tensor's start, so there every slice starts on a multiple of 256 (the gaps are
zero and stay zero).
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
BLOCK = 256  # elements per scale of an 8-bit moment
E4M3_MAX = 448.0
MIN_AMAX = 2.0 ** -100  # blocks below this are stored as zeros
LR, BETA1, BETA2, ADAM_EPS = 1e-3, 0.9, 0.999, 1e-8
STEP, SEED = 7, 20240229
LN_EPS = 1e-5
MAX_NORM = 1.0


def listed():
    # The many-tensor lists are the parameter list of the repository's GPT-2-medium-like gradient workload
    # (24 layers, d = 1024, vocab 50257, 1024 positions: 292 tensors, 354,823,168 elements), one layer of it,
    # and odd-sized lists.
    model = {"layers": 24, "width": 1024, "vocab": 50257, "positions": 1024}
    layer = {"layers": 1, "width": 1024, "vocab": 0, "positions": 0}
    return [
        # one new token of the model: nothing but latency
        {"name": "ln_fwd_token", "op": "ln_fwd", "rows": 1, "cols": 1024, "dtype": "bf16", "wdtype": "bf16"},
        # 8 sequences of 1024 positions through one of the model's norms
        {"name": "ln_fwd_batch", "op": "ln_fwd", "rows": 8192, "cols": 1024, "dtype": "bf16", "wdtype": "bf16"},
        # an odd row length: no row but the first starts on a 4-byte boundary
        {"name": "ln_fwd_odd", "op": "ln_fwd", "rows": 6001, "cols": 4095, "dtype": "f16", "wdtype": "f32"},
        # the backward pass of ln_fwd_batch
        {"name": "ln_bwd_batch", "op": "ln_bwd", "rows": 8192, "cols": 1024, "dtype": "bf16", "wdtype": "bf16"},
        # a wide model's norm over 32 sequences of 1024 positions
        {"name": "ln_bwd_wide", "op": "ln_bwd", "rows": 32768, "cols": 8192, "dtype": "bf16", "wdtype": "f32"},
        # full precision, odd sizes
        {"name": "ln_bwd_odd", "op": "ln_bwd", "rows": 2047, "cols": 1537, "dtype": "f32", "wdtype": "f32"},
        # one layer's gradients, just reduced
        {"name": "norm_layer", "op": "norm", "gdtype": "bf16", **layer},
        # the whole model's gradients in full precision
        {"name": "norm_model", "op": "norm", "gdtype": "f32", **model},
        # a few odd-sized tensors: latency
        {"name": "adamw_small", "op": "adamw", "pdtype": "f32", "gdtype": "f32", "copy": "", "tensors": 14,
         "elements": 40001, "split": 3},
        # mixed precision: fp32 master weights, bf16 gradients, the bf16 weights written along
        {"name": "adamw_model", "op": "adamw", "pdtype": "f32", "gdtype": "bf16", "copy": "bf16", **model},
        # 8-bit moments, odd-sized tensors, fp16 gradients onto fp32 weights
        {"name": "adamw8_odd", "op": "adamw8", "pdtype": "f32", "gdtype": "f16", "copy": "", "tensors": 37,
         "elements": 9000011, "split": 5},
        # 8-bit moments, pure bf16 training of the whole model
        {"name": "adamw8_model", "op": "adamw8", "pdtype": "bf16", "gdtype": "bf16", "copy": "", **model},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["ln_fwd", "ln_bwd", "norm", "adamw", "adamw8"])
    if op in ("ln_fwd", "ln_bwd"):
        cols = log(33, 20000)
        if rng.random() < 0.6:  # most models' widths are round, some are not
            cols = max(64, cols // 64 * 64)
        rows = log(1, min(40000, 100_000_000 // cols))
        dtype = rng.choice(["bf16", "f16", "f32"])
        return {"op": op, "rows": rows, "cols": cols, "dtype": dtype, "wdtype": rng.choice([dtype, "f32"])}
    tensors = log(1, 400)
    case = {"op": op, "gdtype": rng.choice(["bf16", "f16", "f32"]), "tensors": tensors,
            "elements": log(max(1000, 4 * tensors), 150_000_000), "split": rng.randrange(1 << 30)}
    if op != "norm":
        case["pdtype"] = rng.choice(["f32", "bf16"])
        case["copy"] = rng.choice(["", "bf16", "f16"]) if case["pdtype"] == "f32" else ""
    return case


def _counts(case):
    """The element counts of a many-tensor case."""
    if "layers" in case:
        d = case["width"]
        one = [d, d, d * 3 * d, 3 * d, d * d, d, d, d, d * 4 * d, 4 * d, 4 * d * d, d]
        head = [case["vocab"] * d, case["positions"] * d] if case["vocab"] else []
        return head + one * case["layers"] + ([d, d] if case["vocab"] else [])
    r = np.random.RandomState(case["split"])
    share = np.exp(1.5 * r.standard_normal(case["tensors"]))
    n = np.maximum(1, (share / share.sum() * case["elements"]).astype(np.int64))
    return [int(v) for v in n]


def _starts(case, counts):
    """Where each tensor starts in the flat buffers, and their length."""
    step = BLOCK if case["op"] == "adamw8" else 1
    padded = -(-np.array(counts, dtype=np.int64) // step) * step
    ends = np.cumsum(padded)
    return [int(v) for v in ends - padded], int(ends[-1])


def work(case):
    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        n, e, w = case["rows"] * case["cols"], BYTES[case["dtype"]], BYTES[case["wdtype"]] * case["cols"]
        if op == "ln_fwd":
            return {"bytes": 2 * n * e + 8 * case["rows"] + 2 * w, "flops": 8 * n}
        return {"bytes": 3 * n * e + 8 * case["rows"] + 3 * w, "flops": 16 * n}
    n = sum(_counts(case))
    if op == "norm":
        return {"bytes": n * BYTES[case["gdtype"]], "flops": 2 * n}
    per = 2 * BYTES[case["pdtype"]] + BYTES[case["gdtype"]] + (BYTES[case["copy"]] if case["copy"] else 0)
    if op == "adamw":
        return {"bytes": n * (per + 16), "flops": 14 * n}
    blocks = sum(-(-c // BLOCK) for c in _counts(case))
    return {"bytes": n * (per + 4) + 16 * blocks, "flops": 24 * n}


# ---- inputs ------------------------------------------------------------------


def _quantise_nearest(x):
    """[blocks, 256] fp32 -> (e4m3 values, fp32 scales): the 8-bit moments a program starts from."""
    amax = x.abs().amax(dim=1, keepdim=True)
    inv = torch.where(amax > MIN_AMAX, E4M3_MAX / amax, torch.zeros_like(amax))
    q = (x * inv).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q, torch.where(amax > MIN_AMAX, amax * (1.0 / E4M3_MAX), torch.zeros_like(amax)).reshape(-1)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    op = case["op"]
    if op in ("ln_fwd", "ln_bwd"):
        rows, cols, dt, wdt = case["rows"], case["cols"], DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        # a residual stream: rows of different magnitude, a common offset per row
        x = normal(rows, cols)
        x = x.mul_(normal(rows, 1).abs_().add_(0.5)).add_(normal(rows, 1, std=0.5)).to(dt)
        s = {"op": op, "x": x, "w": normal(cols, std=0.2).add_(1.0).to(wdt), "b": normal(cols, std=0.1).to(wdt)}
        s["mean"] = torch.empty(rows, device="cuda")
        s["rstd"] = torch.empty(rows, device="cuda")
        if op == "ln_fwd":
            s["y"] = torch.empty_like(x)
            return s
        s["dy"] = normal(rows, cols, std=0.02).to(dt)
        xf = x.float()
        s["mean"] = xf.mean(dim=1)
        s["rstd"] = (xf - s["mean"][:, None]).square().mean(dim=1).add(LN_EPS).rsqrt()
        s["dx"], s["dw"], s["db"] = torch.empty_like(x), torch.empty_like(s["w"]), torch.empty_like(s["w"])
        if own:  # scratch that a training program keeps
            from ring_all_reduce_02_gb300 import ra

            s["workspace"] = torch.empty(ra.ra_layernorm_workspace(rows, cols), dtype=torch.uint8, device="cuda")
        return s

    counts = _counts(case)
    starts, total = _starts(case, counts)

    def cut(flat):
        return [flat[a:a + n] for a, n in zip(starts, counts)]

    gdt = DTYPES[case["gdtype"]]
    g = normal(total, std=1e-3).to(gdt)
    if op == "norm":
        s = {"op": op, "g": g, "out": torch.empty(2, device="cuda")}
        if own:
            from ring_all_reduce_02_gb300 import ra

            s["workspace"] = torch.zeros(ra.ra_grad_norm_workspace(), dtype=torch.uint8, device="cuda")
            s["grads"] = ra.grad_tensors(cut(g))
        return s

    # matrices decay, the vectors (norms and biases: the short tensors) do not
    decay = [0.1 if n > 65536 else 0.0 for n in counts]
    s = {"op": op, "g": g, "p": normal(total, std=0.02).to(DTYPES[case["pdtype"]]), "scale": normal(1).abs_().add_(0.5)}
    s["copy"] = torch.empty(total, dtype=DTYPES[case["copy"]], device="cuda") if case["copy"] else None
    m = normal(total, std=3e-4)
    v = normal(total, std=1e-3).square_()
    s["keep"] = torch.tensor([1.0 - LR * d for d in decay], dtype=torch.float32, device="cuda")
    s["ordinal"] = torch.arange(len(counts), device="cuda")
    s["lengths"] = torch.tensor(np.diff(starts + [total]), device="cuda")
    s["starts"] = torch.tensor(starts, device="cuda")
    s["total"] = total
    if op == "adamw":
        s["m"], s["v"] = m, v
        state = (cut(m), cut(v))
    else:
        gap = torch.ones(total, dtype=torch.bool, device="cuda")
        inside = [gap[a:a + n].fill_(False) for a, n in zip(starts, counts)]
        del inside
        for t in (s["g"], s["p"], m, v):
            t.masked_fill_(gap, 0)
        if s["copy"] is not None:
            s["copy"].zero_()
        s["m8"], s["m_scale"] = _quantise_nearest(m.view(-1, BLOCK))
        s["r8"], s["r_scale"] = _quantise_nearest(v.sqrt_().view(-1, BLOCK))
        del m, v

        def blocks(scale):
            return [scale[a // BLOCK:a // BLOCK + -(-n // BLOCK)] for a, n in zip(starts, counts)]

        state = (cut(s["m8"].view(-1)), cut(s["r8"].view(-1)), blocks(s["m_scale"]), blocks(s["r_scale"]))
    if own:  # the list of tensors that an optimiser keeps
        from ring_all_reduce_02_gb300 import ra

        s["tensors"] = ra.adamw_tensors(cut(s["p"]), cut(g), *state, weight_decay=decay,
                                        copies=cut(s["copy"]) if s["copy"] is not None else None)
    return s


# ---- the library's calls -------------------------------------------------------


def _run_own(s):
    from ring_all_reduce_02_gb300 import ra

    op = s["op"]
    if op == "ln_fwd":
        ra.ra_layernorm_forward(s["x"], s["w"], s["b"], s["y"], s["mean"], s["rstd"], eps=LN_EPS)
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "ln_bwd":
        ra.ra_layernorm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["dx"], s["dw"], s["db"],
                                 workspace=s["workspace"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    if op == "norm":
        ra.ra_grad_norm(s["grads"], MAX_NORM, s["out"], workspace=s["workspace"])
        return s["out"]
    ra.ra_adamw(s["tensors"], lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS, step=STEP, grad_scale=s["scale"], seed=SEED)
    return _adamw_outputs(s)


def _adamw_outputs(s):
    keys = ("p", "copy", "m", "v") if s["op"] == "adamw" else ("p", "copy", "m8", "m_scale", "r8", "r_scale")
    return {k: s[k] for k in keys if s[k] is not None}


# ---- the plain forms -------------------------------------------------------------


def _ln_fwd(s):
    x = s["x"].float()
    mean = x.mean(dim=1, keepdim=True)
    xc = x - mean
    rstd = 1.0 / torch.sqrt((xc * xc).mean(dim=1, keepdim=True) + LN_EPS)
    y = xc * rstd * s["w"].float() + s["b"].float()
    return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _ln_bwd(s):
    dy, xhat = s["dy"].float(), (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    a = dy * s["w"].float()
    dx = s["rstd"][:, None] * (a - a.mean(dim=1, keepdim=True) - xhat * (a * xhat).mean(dim=1, keepdim=True))
    wdt = s["w"].dtype
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * xhat).sum(dim=0).to(wdt), "db": dy.sum(dim=0).to(wdt)}


def _norm(s):
    g = s["g"].float()
    norm = torch.sqrt((g * g).sum())
    scale = torch.clamp(MAX_NORM / (norm + 1e-6), max=1.0)
    return torch.stack([norm, torch.where(torch.isfinite(norm), scale, torch.full_like(scale, math.nan))])


MASK = 0xFFFFFFFF


def _mix(x):
    """A 32-bit mix of integers (held in int64 tensors, or Python integers)."""
    x = x ^ (x >> 16)
    x = (x * 0xB7E15163) & MASK
    x = x ^ (x >> 15)
    x = (x * 0x9E3779B9) & MASK
    return x ^ (x >> 16)


def _random_bits(s):
    """32 bits for every element, from the seed, the step, the tensor's place in the list and the element's in it."""
    key = _mix((SEED + _mix((SEED >> 32) + STEP * 0x9E3779B9 & MASK)) & MASK)
    keys = _mix((key + s["ordinal"] * 0xB7E15163) & MASK)
    of = torch.repeat_interleave(s["ordinal"], s["lengths"], output_size=s["total"])
    i = torch.arange(s["total"], device=of.device) - s["starts"][of]
    return _mix(((i & MASK) * 0x9E3779B9 + (i >> 32) * 0xB7E15163 + keys[of]) & MASK)


def _quantise(x, rand16):
    """Blocks of fp32 -> (e4m3 values, fp32 scales), rounded up or down by 16 random bits a value."""
    amax = x.abs().amax(dim=1, keepdim=True)
    some = amax > MIN_AMAX
    inv = torch.where(some, E4M3_MAX / amax, torch.zeros_like(amax))
    t = (x * inv).clamp(-E4M3_MAX, E4M3_MAX)
    t = ((t.view(torch.int32) + (rand16 << 4).to(torch.int32)) & -0x100000).view(torch.float32)
    return t, torch.where(some, amax * (1.0 / E4M3_MAX), torch.zeros_like(amax)), some


def _adamw(s):
    eight = s["op"] == "adamw8"
    if eight:
        m_old = (s["m8"].float() * s["m_scale"][:, None]).view(-1)
        r_old = (s["r8"].float() * s["r_scale"][:, None]).view(-1)
        v_old = r_old * r_old
    else:
        m_old, v_old = s["m"], s["v"]
    g = s["g"].float() * s["scale"]
    m = m_old * BETA1 + g * (1.0 - BETA1)
    v = v_old * BETA2 + (g * (1.0 - BETA2)) * g
    r = torch.sqrt(v)
    u = m / (r * (1.0 / math.sqrt(1.0 - BETA2 ** STEP)) + ADAM_EPS)
    keep = torch.repeat_interleave(s["keep"], s["lengths"], output_size=s["total"])
    p = s["p"].float() * keep - u * (LR / (1.0 - BETA1 ** STEP))
    s["p"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    if not eight:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return _adamw_outputs(s)
    rand = _random_bits(s).view(-1, BLOCK)
    t, scale, some = _quantise(m.view(-1, BLOCK), rand & 0xFFFF)
    s["m8"].copy_(t.to(torch.float8_e4m3fn))
    s["m_scale"].copy_(scale[:, 0])
    r = r.view(-1, BLOCK)
    t, scale, some = _quantise(r, rand >> 16)
    # a second moment that is not zero is not stored as zero: it divides the next step
    t = torch.where(some & (r > 0), t.clamp(min=2.0 ** -9), t)
    s["r8"].copy_(t.to(torch.float8_e4m3fn))
    s["r_scale"].copy_(scale[:, 0])
    return _adamw_outputs(s)


def run(state):
    if own:
        return _run_own(state)
    return {"ln_fwd": _ln_fwd, "ln_bwd": _ln_bwd, "norm": _norm, "adamw": _adamw, "adamw8": _adamw}[state["op"]](state)


# ---- 64 bits -------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "ln_fwd":
        x, w, b = s["x"].double(), s["w"].double(), s["b"].double()
        var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
        return {"y": torch.addcmul(b, (x - mean) / (var + LN_EPS).sqrt(), w), "mean": mean.squeeze(1),
                "rstd": (var + LN_EPS).pow(-0.5).squeeze(1)}
    if op == "ln_bwd":
        # by the definition: the gradient of sum(dy * y) with y linear in the row's projection off (1, xhat)
        n = s["x"].shape[1]
        dw, db = torch.zeros(n, dtype=torch.float64, device="cuda"), torch.zeros(n, dtype=torch.float64, device="cuda")
        dx = torch.empty(s["x"].shape, dtype=torch.float64, device="cuda")
        for a in range(0, s["x"].shape[0], 4096):
            at = slice(a, a + 4096)
            dy, rstd = s["dy"][at].double(), s["rstd"][at, None].double()
            h = (s["x"][at].double() - s["mean"][at, None].double()) * rstd
            dw += torch.einsum("rc,rc->c", dy, h)
            db += dy.sum(0)
            dh = dy * s["w"].double()
            dx[at] = (dh - (dh.sum(1, keepdim=True) + h * torch.einsum("rc,rc->r", dh, h)[:, None]) / n) * rstd
        return {"dx": dx, "dw": dw, "db": db}
    if op == "norm":
        norm = torch.linalg.vector_norm(s["g"].double())
        return torch.stack([norm, torch.minimum(MAX_NORM / (norm + 1e-6), torch.ones_like(norm))])
    eight = op == "adamw8"
    g = s["g"].double() * s["scale"].double()
    if eight:
        m = torch.lerp((s["m8"].double() * s["m_scale"].double()[:, None]).view(-1), g, 1 - BETA1)
        v = torch.lerp((s["r8"].double() * s["r_scale"].double()[:, None]).view(-1).square(), g.square(), 1 - BETA2)
    else:
        m, v = torch.lerp(s["m"].double(), g, 1 - BETA1), torch.lerp(s["v"].double(), g.square(), 1 - BETA2)
    del g
    mhat, vhat = m / (1 - BETA1 ** STEP), v / (1 - BETA2 ** STEP)
    shrink = torch.repeat_interleave(s["keep"].double(), s["lengths"], output_size=s["total"])
    p = s["p"].double() * shrink - LR * mhat / (vhat.sqrt() + ADAM_EPS)
    out = {"p": p}
    if s["copy"] is not None:
        out["copy"] = p
    if not eight:
        return {**out, "m": m, "v": v}
    # the 8-bit values: the neighbour below in e4m3's normal range, or the one above when the random bits say so
    rand = _random_bits(s).view(-1, BLOCK)
    for name, x, bits in (("m", m, rand & 0xFFFF), ("r", v.sqrt(), rand >> 16)):
        x = x.view(-1, BLOCK)
        scale = x.abs().amax(1, keepdim=True) / E4M3_MAX
        scale = torch.where(scale > MIN_AMAX / E4M3_MAX, scale, torch.zeros_like(scale))
        t = torch.where(scale > 0, x / scale, torch.zeros_like(x))
        mant, expo = torch.frexp(t.abs())
        t = t.sign() * torch.ldexp(torch.floor(mant * 16 + bits.double() / 65536), expo - 4)
        t = (t * 512).round() / 512  # below the normal range, the nearest of the even steps of 2^-9
        if name == "r":
            t = torch.where((x > 0) & (scale > 0), t.clamp(min=2.0 ** -9), t)
        out[name + "8"], out[name + "_scale"] = t, scale.squeeze(1)
    return out
