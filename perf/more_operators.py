"""The two ends of a language model's training step, as workloads.

The embedding lookup with scaling and its gradient (the sum of dy over the
places of each token), and softmax cross entropy over the vocabulary straight
from the hidden states and the head's weight, with its gradients, without
keeping the logits.

``run`` computes an operator in its plain form (elementary torch operations in
fp32, rounded once at the end), or, with ``own`` set, by the library's entry
points. ``exact`` computes it in 64 bits.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}
INDEX = {"i32": torch.int32, "i64": torch.int64}
IGNORE = -100  # the target of a position that has no loss


def listed():
    # Width, vocabulary and batch of the repository's GPT-2-medium-like workload (d = 1024, vocab 50257, 8 sequences of
    # 1024 positions), its wide norm's batch (32 sequences, d = 8192), and odd sizes.
    return [
        # one new token of each of 8 sequences: nothing but latency
        {"name": "embed_fwd_tokens", "op": "embed_fwd", "rows": 8, "cols": 1024, "vocab": 50257, "dtype": "bf16",
         "index": "i64", "text": True, "accumulate": False},
        # the model's batch
        {"name": "embed_fwd_batch", "op": "embed_fwd", "rows": 8192, "cols": 1024, "vocab": 50257, "dtype": "bf16",
         "index": "i64", "text": True, "accumulate": False},
        # odd rows in full precision, added to what the positions gave
        {"name": "embed_fwd_odd", "op": "embed_fwd", "rows": 30011, "cols": 771, "vocab": 10007, "dtype": "f32",
         "index": "i32", "text": False, "accumulate": True},
        # a short sequence's gradient, added to a tied head's
        {"name": "embed_bwd_short", "op": "embed_bwd", "rows": 61, "cols": 1024, "vocab": 50257, "dtype": "bf16",
         "index": "i64", "text": True, "accumulate": True, "padded": 0.0},
        # the model's batch, added to a tied head's gradient
        {"name": "embed_bwd_batch", "op": "embed_bwd", "rows": 8192, "cols": 1024, "vocab": 50257, "dtype": "bf16",
         "index": "i64", "text": True, "accumulate": True, "padded": 0.0},
        # a wide model's batch: a table's whole gradient
        {"name": "embed_bwd_wide", "op": "embed_bwd", "rows": 32768, "cols": 8192, "vocab": 50257, "dtype": "bf16",
         "index": "i64", "text": True, "accumulate": False, "padded": 0.0},
        # odd rows, padded sequences
        {"name": "embed_bwd_odd", "op": "embed_bwd", "rows": 20011, "cols": 515, "vocab": 10007, "dtype": "f16",
         "index": "i32", "text": True, "accumulate": False, "padded": 0.2},
        # the loss of one token: the head's weight streams past
        {"name": "ce_fwd_token", "op": "ce_fwd", "rows": 1, "cols": 1024, "vocab": 50257, "dtype": "bf16",
         "index": "i64", "ignored": 0.0},
        # the model's batch, as evaluation has it
        {"name": "ce_fwd_batch", "op": "ce_fwd", "rows": 8192, "cols": 1024, "vocab": 50257, "dtype": "bf16",
         "index": "i64", "ignored": 0.0},
        # a short sequence's gradients
        {"name": "ce_bwd_short", "op": "ce_bwd", "rows": 61, "cols": 1024, "vocab": 50257, "dtype": "bf16",
         "index": "i64", "ignored": 0.0, "accumulate": False},
        # the model's batch
        {"name": "ce_bwd_batch", "op": "ce_bwd", "rows": 8192, "cols": 1024, "vocab": 50257, "dtype": "bf16",
         "index": "i64", "ignored": 0.0, "accumulate": False},
        # odd sizes, a quarter of the positions without a loss
        {"name": "ce_bwd_odd", "op": "ce_bwd", "rows": 1537, "cols": 771, "vocab": 10007, "dtype": "f16",
         "index": "i32", "ignored": 0.25, "accumulate": True},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["embed_fwd", "embed_bwd", "ce_fwd", "ce_bwd"])
    case = {"op": op, "index": rng.choice(["i32", "i64"])}
    odd = rng.random() < 0.4  # most models' widths are round, some are not
    if op in ("embed_fwd", "embed_bwd"):
        cols = log(33, 8192)
        cols = cols if odd else max(64, cols // 64 * 64)
        vocab = log(100, min(150_000, 400_000_000 // cols))
        case.update(rows=log(1, min(200_000, 260_000_000 // cols)), cols=cols, vocab=vocab,
                    dtype=rng.choice(["bf16", "f16", "f32"]), text=rng.random() < 0.7, accumulate=rng.random() < 0.5)
        if op == "embed_bwd":
            case["padded"] = rng.choice([0.0, 0.3])
        return case
    cols = log(64, 4096)
    cols = cols if odd else max(64, cols // 64 * 64)
    vocab = log(100, min(130_000, 200_000_000 // cols))
    case.update(rows=log(1, min(16384, 400_000_000_000 // (cols * vocab))), cols=cols, vocab=vocab,
                dtype=rng.choice(["bf16", "f16"]), ignored=rng.choice([0.0, 0.1, 0.5]))
    if op == "ce_bwd":
        case["accumulate"] = rng.random() < 0.3
    return case


def _left(case, share):
    """The rows of a case that are not padded or ignored."""
    return case["rows"] - int(case["rows"] * share)


def _distinct(case, rows):
    """The distinct tokens that `rows` draws are expected to hold."""
    v = case["vocab"]
    p = np.log1p(1.0 / np.arange(1, v + 1)) / math.log(v + 1) if case["text"] else np.full(v, 1.0 / v)
    return float(-np.expm1(rows * np.log1p(-p.clip(max=1 - 1e-12))).sum())


def work(case):
    rows, cols, vocab, e = case["rows"], case["cols"], case["vocab"], BYTES[case["dtype"]]
    index = 4 if case["index"] == "i32" else 8
    if case["op"] == "embed_fwd":
        per = 2 if case["accumulate"] else 1
        return {"bytes": (_distinct(case, rows) + per * rows) * cols * e + rows * index, "flops": per * rows * cols}
    if case["op"] == "embed_bwd":
        left = _left(case, case["padded"])
        table = 2 * _distinct(case, left) if case["accumulate"] else vocab
        return {"bytes": (left + table) * cols * e + rows * index, "flops": left * cols}
    left = _left(case, case["ignored"])
    if case["op"] == "ce_fwd":
        return {"bytes": (left + vocab) * cols * e + rows * (index + 8), "flops": 2 * left * cols * vocab}
    table = 3 if case["accumulate"] else 2
    return {"bytes": (left + rows + table * vocab) * cols * e + rows * (index + 8), "flops": 6 * left * cols * vocab}


# ---- inputs ------------------------------------------------------------------


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).mul_(std).to(dtype)

    def some(share):
        """That share of the rows, at random places."""
        return torch.randperm(rows, generator=gen, device="cuda")[:int(rows * share)]

    op, rows, cols, vocab = case["op"], case["rows"], case["cols"], case["vocab"]
    dt = DTYPES[case["dtype"]]
    s = {"op": op}
    if op in ("embed_fwd", "embed_bwd"):
        u = torch.rand(rows, generator=gen, device="cuda", dtype=torch.float64)
        # text: the k-th most frequent token comes up about 1/k as often as the first, and has a low number
        place = torch.expm1(u * math.log(vocab + 1)) if case["text"] else u * vocab
        tokens = place.long().clamp_(0, vocab - 1)
        s["scale"], s["accumulate"] = math.sqrt(cols), case["accumulate"]
        if op == "embed_fwd":
            s["table"] = normal(vocab, cols, std=0.02, dtype=dt)
            s["out"] = normal(rows, cols, std=0.02, dtype=dt)
        else:
            s["padding"] = 0 if case["padded"] else None
            tokens[some(case["padded"])] = 0
            s["dy"] = normal(rows, cols, std=0.02, dtype=dt)
            s["dtable"] = normal(vocab, cols, std=0.02, dtype=dt)
            if own:  # scratch that a training program keeps
                from ring_all_reduce_02_gb300 import ra

                s["workspace"] = torch.empty(ra.ra_embedding_workspace(rows, cols, vocab), dtype=torch.uint8, device="cuda")
        s["tokens"] = tokens.to(INDEX[case["index"]])
        return s

    # hidden states behind a norm, a head of the usual initial deviation
    s["hidden"] = normal(rows, cols, dtype=dt)
    s["weight"] = normal(vocab, cols, std=0.02, dtype=dt)
    targets = torch.randint(0, vocab, (rows,), generator=gen, device="cuda")
    targets[some(case["ignored"])] = IGNORE
    s["targets"] = targets.to(INDEX[case["index"]])
    s["loss"], s["lse"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    if op == "ce_bwd":
        s["loss"], s["lse"] = _loss(s)
        # the gradient of a mean over the positions that have a loss, under a loss scale
        s["dloss"] = normal(1).abs_().add_(0.5).expand(rows).contiguous().mul_(256.0 / _left(case, case["ignored"]))
        s["dhidden"] = torch.empty_like(s["hidden"])
        s["accumulate"] = case["accumulate"]
        s["dweight"] = normal(vocab, cols, std=0.02, dtype=dt)
    if own:
        from ring_all_reduce_02_gb300 import ra

        bytes_ = ra.ra_cross_entropy_workspace(s["hidden"], s["weight"], backward=op == "ce_bwd")
        s["workspace"] = torch.empty(bytes_, dtype=torch.uint8, device="cuda")
    return s


# ---- the library's calls -------------------------------------------------------


def _run_own(s):
    from ring_all_reduce_02_gb300 import ra

    op = s["op"]
    if op == "embed_fwd":
        ra.ra_embedding_forward(s["table"], s["tokens"], s["out"], scale=s["scale"], accumulate=s["accumulate"])
        return s["out"]
    if op == "embed_bwd":
        ra.ra_embedding_backward(s["dy"], s["tokens"], s["dtable"], scale=s["scale"], accumulate=s["accumulate"],
                                 padding=s["padding"], workspace=s["workspace"])
        return s["dtable"]
    if op == "ce_fwd":
        ra.ra_cross_entropy_forward(s["hidden"], s["weight"], s["targets"], s["loss"], s["lse"], ignore=IGNORE,
                                    workspace=s["workspace"])
        return {"loss": s["loss"], "lse": s["lse"]}
    ra.ra_cross_entropy_backward(s["hidden"], s["weight"], s["targets"], s["lse"], s["dloss"], s["dhidden"], s["dweight"],
                                 ignore=IGNORE, accumulate=s["accumulate"], workspace=s["workspace"])
    return {"dhidden": s["dhidden"], "dweight": s["dweight"]}


# ---- the plain forms -------------------------------------------------------------


def _embed_fwd(s):
    x = s["table"][s["tokens"].long()].float() * s["scale"]
    if s["accumulate"]:
        x = x + s["out"].float()
    return s["out"].copy_(x)


def _embed_bwd(s):
    dy = s["dy"].float()
    if s["padding"] is not None:
        dy = dy * (s["tokens"] != s["padding"])[:, None]
    total = torch.zeros(s["dtable"].shape, device="cuda").index_add_(0, s["tokens"].long(), dy) * s["scale"]
    if s["accumulate"]:
        total = total + s["dtable"].float()
    return s["dtable"].copy_(total)


def _loss(s):
    logits = s["hidden"].float() @ s["weight"].float().t()
    top = logits.amax(dim=1, keepdim=True)
    lse = top[:, 0] + torch.log(torch.exp(logits - top).sum(dim=1))
    counts = s["targets"] != IGNORE
    at = torch.where(counts, s["targets"], torch.zeros_like(s["targets"])).long()
    loss = lse - logits.gather(1, at[:, None])[:, 0]
    zero = torch.zeros_like(loss)
    return torch.where(counts, loss, zero), torch.where(counts, lse, zero)


def _ce_fwd(s):
    loss, lse = _loss(s)
    return {"loss": loss, "lse": lse}


def _ce_bwd(s):
    h, w = s["hidden"].float(), s["weight"].float()
    counts = s["targets"] != IGNORE
    d = torch.exp(h @ w.t() - s["lse"][:, None])
    at = torch.where(counts, s["targets"], torch.zeros_like(s["targets"])).long()
    d[torch.arange(h.shape[0], device="cuda"), at] -= 1.0
    d = d * torch.where(counts, s["dloss"], torch.zeros_like(s["dloss"]))[:, None]
    dw = d.t() @ h
    if s["accumulate"]:
        dw = dw + s["dweight"].float()
    s["dhidden"].copy_(d @ w)
    s["dweight"].copy_(dw)
    return {"dhidden": s["dhidden"], "dweight": s["dweight"]}


def run(state):
    if own:
        return _run_own(state)
    return {"embed_fwd": _embed_fwd, "embed_bwd": _embed_bwd, "ce_fwd": _ce_fwd, "ce_bwd": _ce_bwd}[state["op"]](state)


# ---- 64 bits -------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "embed_fwd":
        x = torch.nn.functional.embedding(s["tokens"].long(), s["table"].double())
        return torch.add(s["out"].double() if s["accumulate"] else torch.zeros_like(x), x, alpha=s["scale"])
    if op == "embed_bwd":
        # by sorted tokens: a token's sum is the difference of two running sums
        keep = torch.ones_like(s["tokens"], dtype=torch.bool) if s["padding"] is None else s["tokens"] != s["padding"]
        tokens, order = torch.sort(s["tokens"].long()[keep])
        want = s["dtable"].double() if s["accumulate"] else torch.zeros(s["dtable"].shape, dtype=torch.float64, device="cuda")
        which, ends = torch.unique_consecutive(tokens, return_counts=True)
        ends = ends.cumsum(0)
        for a in range(0, want.shape[1], 256):
            running = s["dy"][keep][:, a:a + 256].double()[order].cumsum(0)[ends - 1]
            want[which, a:a + 256] += s["scale"] * torch.diff(running, dim=0, prepend=torch.zeros_like(running[:1]))
        return want
    h, w, targets = s["hidden"].double(), s["weight"].double(), s["targets"].long()
    if op == "ce_fwd":
        out = {"loss": torch.zeros(len(targets), dtype=torch.float64, device="cuda"), "lse": torch.zeros(len(targets), dtype=torch.float64, device="cuda")}
        for a in range(0, len(targets), 1024):
            at = slice(a, a + 1024)
            logits = h[at] @ w.t()
            out["lse"][at] = torch.logsumexp(logits, 1) * (targets[at] != IGNORE)
            out["loss"][at] = torch.nn.functional.cross_entropy(logits, targets[at], ignore_index=IGNORE, reduction="none")
        return out
    dh, dw = torch.zeros_like(h), s["dweight"].double() if s["accumulate"] else torch.zeros_like(w)
    for a in range(0, len(targets), 1024):
        at = slice(a, a + 1024)
        # the stored lse is an input: the gradient is that of dloss (exp(logit - lse) - [target])
        d = torch.exp(h[at] @ w.t() - s["lse"][at, None].double())
        there = targets[at] != IGNORE
        d[there] -= torch.nn.functional.one_hot(targets[at][there], len(w)).double()
        d *= (s["dloss"][at].double() * there)[:, None]
        dh[at] = d @ w
        dw += d.t() @ h[at]
    return {"dhidden": dh, "dweight": dw}
