"""Measured cases of the vocabulary-sized operators at the two ends of a language model:

* ``ce_train``  softmax cross entropy of hidden states against a head matrix, with the gradients of both
  (targets below zero are not counted, each token may carry a weight, the mean is over the counted weights);
* ``ce_score``  the same loss and the log of the softmax's sum for each token, without gradients;
* ``embed``     embedding lookup with a scale (ids below zero are padding and give zero rows);
* ``embed_grad``  the gradient of that lookup as a whole table, written or added to what the table's gradient holds.

``own`` false computes them from elementary torch operations in 32 bits, ``own`` true through the package.
"""

import math

import torch

own = False

_handle = None


def _ops():
    """The one handle that a user's program keeps for all of its calls."""
    global _handle
    if _handle is None:
        import matrix_optimizer_step_gb300 as mos

        _handle = mos.VocabOps(0)
    return _handle


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    return [
        # One training sequence of 8192 tokens against the Llama-3-8B head (128256 x 4096): the head's share of a step.
        {"name": "ce_train_8192x128256x4096", "op": "ce_train", "tokens": 8192, "vocab": 128256, "dim": 4096,
         "ignored": 0.0, "weighted": False},
        # A micro-batch of four 1024-token sequences with the GPT-2-small width and a vocabulary of odd size.
        {"name": "ce_train_4096x50257x768", "op": "ce_train", "tokens": 4096, "vocab": 50257, "dim": 768,
         "ignored": 0.0, "weighted": False},
        # Supervised fine-tuning with prompts masked out and a weight per token, every size ragged.
        {"name": "ce_train_1023x32003x1000", "op": "ce_train", "tokens": 1023, "vocab": 32003, "dim": 1000,
         "ignored": 0.4, "weighted": True},
        # A few answer tokens only: the head's gradient is one long write.
        {"name": "ce_train_24x128256x4096", "op": "ce_train", "tokens": 24, "vocab": 128256, "dim": 4096,
         "ignored": 0.0, "weighted": False},
        # Scoring a document of about a thousand tokens (evaluation, ranking of answers).
        {"name": "ce_score_1000x128256x4096", "op": "ce_score", "tokens": 1000, "vocab": 128256, "dim": 4096,
         "ignored": 0.1, "weighted": False},
        # Scoring one token, as while generating.
        {"name": "ce_score_1x128256x4096", "op": "ce_score", "tokens": 1, "vocab": 128256, "dim": 4096,
         "ignored": 0.0, "weighted": False},
        # Lookup of four 8192-token sequences in the Llama-3-8B table.
        {"name": "embed_32768x128256x4096", "op": "embed", "tokens": 32768, "vocab": 128256, "dim": 4096,
         "table": "bf16", "out": "bf16", "scale": 1.0, "padded": 0.0},
        # One token of a small model with a scaled embedding and an fp32 table: launch latency.
        {"name": "embed_1x50257x768", "op": "embed", "tokens": 1, "vocab": 50257, "dim": 768,
         "table": "f32", "out": "bf16", "scale": math.sqrt(768.0), "padded": 0.0},
        # The whole bf16 gradient of the Llama-3-8B table, as the AdamW route takes it.
        {"name": "embed_grad_32768x128256x4096", "op": "embed_grad", "tokens": 32768, "vocab": 128256, "dim": 4096,
         "out": "bf16", "grad": "bf16", "scale": 1.0, "padded": 0.0, "add": False, "spread": "zipf"},
        # A further micro-batch added to an fp32 gradient (gradient accumulation): only the looked-up rows move.
        {"name": "embed_grad_add_4096x50257x768", "op": "embed_grad", "tokens": 4096, "vocab": 50257, "dim": 768,
         "out": "bf16", "grad": "f32", "scale": math.sqrt(768.0), "padded": 0.1, "add": True, "spread": "zipf"},
        # Ragged sizes and a batch in which a handful of ids carries every token (byte-like data, special tokens).
        {"name": "embed_grad_5001x1031x1000", "op": "embed_grad", "tokens": 5001, "vocab": 1031, "dim": 1000,
         "out": "f32", "grad": "f32", "scale": 1.0, "padded": 0.0, "add": False, "spread": "few"},
        # A few tokens added to the gradient of a large table: latency.
        {"name": "embed_grad_add_17x128256x4096", "op": "embed_grad", "tokens": 17, "vocab": 128256, "dim": 4096,
         "out": "bf16", "grad": "bf16", "scale": 1.0, "padded": 0.0, "add": True, "spread": "zipf"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["ce_train", "ce_train", "ce_score", "embed", "embed_grad"])
    vocab = _log_int(rng, 1000, 128256)
    # Widths are multiples of 8 in nearly every model; one in eight here is not.
    dim = _log_int(rng, 256, 4096)
    if rng.random() < 0.875:
        dim = max(256, dim // 8 * 8)
    if op.startswith("ce"):
        return {"op": op, "tokens": _log_int(rng, 1, 8192), "vocab": vocab, "dim": dim,
                "ignored": rng.choice([0.0, 0.0, 0.3]), "weighted": op == "ce_train" and rng.random() < 0.3}
    case = {"op": op, "tokens": _log_int(rng, 1, 32768), "vocab": vocab, "dim": dim,
            "out": rng.choice(["bf16", "bf16", "f32"]), "scale": rng.choice([1.0, math.sqrt(dim)]),
            "padded": rng.choice([0.0, 0.2])}
    if op == "embed":
        return {**case, "table": rng.choice(["bf16", "f32"])}
    return {**case, "grad": rng.choice(["bf16", "f32"]), "add": rng.random() < 0.4, "spread": rng.choice(["zipf", "zipf", "few"])}


def _tokens(n, vocab, spread, g):
    """Ids as text has them: the share of id k falls as 1 / (k + 1); or all tokens on eight ids."""
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    if spread == "few":
        few = torch.randint(0, vocab, (8,), generator=g, device="cuda")
        return few[(u * 8).long().clamp_(max=7)]
    return ((vocab + 1.0) ** u - 1.0).long().clamp_(0, vocab - 1)


def _masked(ids, share, g):
    if share > 0.0:
        ids[torch.rand(ids.numel(), generator=g, device="cuda") < share] = -100
    return ids


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    dev = torch.device("cuda")
    s = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    if case["op"].startswith("ce"):
        # Logits of unit-like spread; the target's is raised by 0 to 12, so that tokens run from unforeseen to certain.
        w = (normal(v, d) * (1.3 / math.sqrt(d))).to(torch.bfloat16)
        t = _tokens(n, v, "zipf", g)
        x = normal(n, d) + (torch.rand(n, 1, generator=g, device=dev) * (12.0 / 1.69)) * w[t].float()
        s.update(x=x.to(torch.bfloat16), w=w, targets=_masked(t, case["ignored"], g), weights=None)
        if case["weighted"]:
            s["weights"] = torch.rand(n, generator=g, device=dev) + 0.5
        s.update(loss=torch.empty(n, device=dev), lse=torch.empty(n, device=dev), total=torch.empty(1, device=dev))
        if case["op"] == "ce_train":
            s.update(dx=torch.empty_like(s["x"]), dw=torch.empty_like(w))
        return s
    s["ids"] = _masked(_tokens(n, v, case.get("spread", "zipf"), g), case["padded"], g)
    out = _TYPES[case["out"]]
    if case["op"] == "embed":
        s.update(table=(normal(v, d) * 0.02).to(_TYPES[case["table"]]), out=torch.empty(n, d, device=dev, dtype=out))
        return s
    s["dout"] = (normal(n, d) * 1e-2).to(out)
    s["dtable"] = (normal(v, d) * 1e-2).to(_TYPES[case["grad"]])
    return s


def _plain_ce(s):
    x, w, t = s["x"].float(), s["w"].float(), s["targets"]
    counted = t >= 0
    at = t.clamp(min=0).unsqueeze(1)
    weights = counted.float() if s["weights"] is None else s["weights"] * counted
    z = x @ w.T
    top = z.max(dim=1, keepdim=True).values
    zt = z.gather(1, at)
    e = (z - top).exp_()
    sums = e.sum(dim=1, keepdim=True)
    lse = top + sums.log()
    zero = torch.zeros((), device=x.device)
    loss = torch.where(counted, (lse - zt).squeeze(1), zero)
    lse = torch.where(counted, lse.squeeze(1), zero)
    if s["case"]["op"] == "ce_score":
        return {"loss": loss, "lse": lse}
    norm = weights.sum()
    coef = torch.where(norm > 0, weights / norm, zero).unsqueeze(1)
    total = (coef.squeeze(1) * loss).sum().reshape(1)
    dz = e.mul_(coef / sums)
    dz.scatter_add_(1, at, -coef)
    return {"loss": loss, "lse": lse, "total": total, "dx": (dz @ w).to(s["dx"].dtype), "dw": (dz.T @ x).to(s["dw"].dtype)}


def _plain_embed(s):
    ids = s["ids"]
    rows = s["table"][ids.clamp(min=0)].float() * s["case"]["scale"]
    return (rows * (ids >= 0).unsqueeze(1)).to(s["out"].dtype)


def _plain_embed_grad(s):
    ids, table = s["ids"], s["dtable"]
    rows = s["dout"].float() * (ids >= 0).unsqueeze(1)
    sums = torch.zeros(table.shape, device=table.device).index_add_(0, ids.clamp(min=0), rows) * s["case"]["scale"]
    if s["case"]["add"]:
        sums += table
    table.copy_(sums)
    return table


def run(state):
    op = state["case"]["op"]
    if not own:
        return {"ce_train": _plain_ce, "ce_score": _plain_ce, "embed": _plain_embed, "embed_grad": _plain_embed_grad}[op](state)
    ops, s = _ops(), state
    if op == "ce_score":
        ops.cross_entropy(s["x"], s["w"], s["targets"], loss=s["loss"], lse=s["lse"])
        return {"loss": s["loss"], "lse": s["lse"]}
    if op == "ce_train":
        ops.cross_entropy(s["x"], s["w"], s["targets"], weights=s["weights"], loss=s["loss"], lse=s["lse"],
                          total=s["total"], dx=s["dx"], dw=s["dw"])
        return {k: s[k] for k in ("loss", "lse", "total", "dx", "dw")}
    if op == "embed":
        ops.embed(s["ids"], s["table"], s["out"], scale=s["case"]["scale"])
        return s["out"]
    ops.embed_grad(s["ids"], s["dout"], s["dtable"], scale=s["case"]["scale"], accumulate=s["case"]["add"])
    return s["dtable"]


def work(case):
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    size = {"bf16": 2, "f32": 4}
    if case["op"].startswith("ce"):
        train = case["op"] == "ce_train"
        # Hidden states and head read, targets read, loss and log-sum written; gradients written as large as both.
        nbytes = 2 * (n + v) * d * (2 if train else 1) + 16 * n
        return {"bytes": nbytes, "flops": (6 if train else 2) * n * v * d}
    if case["op"] == "embed":
        # Rows read for each token, but not more than the table; rows written.
        return {"bytes": min(n, v) * d * size[case["table"]] + n * d * size[case["out"]] + 8 * n, "flops": n * d}
    rows = min(n, v) * 2 if case["add"] else v  # rows read and written, or the whole table written
    return {"bytes": n * d * size[case["out"]] + rows * d * size[case["grad"]] + 8 * n, "flops": n * d}


def exact(case, seed):
    """The definitions in 64 bits, token by token blocks."""
    n, v, d = case["tokens"], case["vocab"], case["dim"]
    s = prepare(case, seed)
    if case["op"] == "embed":
        out = torch.zeros(n, d, device="cuda", dtype=torch.float64)
        keep = (s["ids"] >= 0).nonzero().squeeze(1)
        out[keep] = case["scale"] * s["table"][s["ids"][keep]].double()
        return out
    if case["op"] == "embed_grad":
        keep = (s["ids"] >= 0).nonzero().squeeze(1)
        out = s["dtable"].double() if case["add"] else torch.zeros(v, d, device="cuda", dtype=torch.float64)
        return out.index_put_((s["ids"][keep],), case["scale"] * s["dout"][keep].double(), accumulate=True)
    if n * v * d > 2.0e12:
        return None
    train = case["op"] == "ce_train"
    w = s["w"].double()
    weight = torch.ones(n, device="cuda", dtype=torch.float64) if s["weights"] is None else s["weights"].double()
    weight = weight.masked_fill(s["targets"] < 0, 0.0)
    norm = float(weight.sum())
    loss, lse = torch.zeros(2, n, device="cuda", dtype=torch.float64)
    dx, dw = torch.zeros(n, d, device="cuda", dtype=torch.float64), torch.zeros(v, d, device="cuda", dtype=torch.float64)
    for block in (s["targets"] >= 0).nonzero().squeeze(1).split(1024):
        x, t = s["x"][block].double(), s["targets"][block]
        z = torch.mm(x, w.t())
        lse[block] = torch.logsumexp(z, dim=1)
        rows = torch.arange(t.numel(), device="cuda")
        loss[block] = lse[block] - z[rows, t]
        if train:
            p = torch.softmax(z, dim=1)
            p[rows, t] -= 1.0
            p *= (weight[block] / norm).unsqueeze(1)
            dx[block] = torch.mm(p, w)
            dw += torch.mm(p.t(), x)
    if not train:
        return {"loss": loss, "lse": lse}
    total = (weight * loss).sum() / norm if norm > 0 else torch.zeros((), device="cuda", dtype=torch.float64)
    return {"loss": loss, "lse": lse, "total": total.reshape(1), "dx": dx, "dw": dw}
